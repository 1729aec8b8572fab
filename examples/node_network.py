"""A small trained network on the nodes of a graph: species embedding, the
fused convolution over the edges, the gated feed-forward block, and the norm
that joins it to the residual stream, with their backwards and plain
gradient descent.

    python examples/node_network.py [--steps 30] [--dtype f32|bf16|f16]

Everything between the edge harmonics and the updated weights runs in the
library's kernels, except the convolution's features, which it takes in
float32, and the weight update.  Data: seeded random graph and targets.
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import segmented_polynomials_amd as sp

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SPECIES, DIM, HIDDEN = 10, 64, 192


def make_graph(n_nodes, degree, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    species = torch.randint(0, SPECIES, (n_nodes,), generator=g, device="cuda", dtype=torch.int32)
    dst = torch.arange(n_nodes, device="cuda", dtype=torch.int32).repeat_interleave(degree)
    src = torch.randint(0, n_nodes, (n_nodes * degree,), generator=g, device="cuda", dtype=torch.int32)
    vec = torch.randn(n_nodes * degree, 3, generator=g, device="cuda")
    target = torch.randn(n_nodes, DIM, generator=g, device="cuda")
    return species, src, dst, sp.sh_fwd(vec, 1), target


def make_weights(dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    ones = torch.ones(DIM, device="cuda")
    return dict(table=normal(SPECIES, DIM, std=DIM ** -0.5), w_gate=normal(HIDDEN, DIM, std=DIM ** -0.5),
                w_up=normal(HIDDEN, DIM, std=DIM ** -0.5), w_down=normal(DIM, HIDDEN, std=HIDDEN ** -0.5),
                w_post=ones.clone(), res_scale=0.5 * ones, w_pre=ones.clone())


def step(conv, graph, p):
    """Loss and gradients of one pass: the last norm's output is fitted to
    the targets."""
    species, src, dst, sh, target = graph
    dtype = p["table"].dtype
    n = species.shape[0]
    edge_w = torch.full((src.shape[0], conv.weight_numel), 0.5, device="cuda")
    perm = torch.argsort(src, stable=True).int()

    x = sp.embedding_fwd(p["table"], species, scale=DIM ** 0.5)
    near = sp.tp_conv_fwd(conv, x.float(), sh, edge_w, src, dst, n_nodes=n).to(dtype)
    f = sp.gated_ffn_fwd(near, p["w_gate"], p["w_up"], p["w_down"])
    norm = dict(f=f, w_post=p["w_post"], res_scale=p["res_scale"], w_pre=p["w_pre"], kind="layer")
    y, h = sp.block_norm_fwd(x, **norm)

    off = h.float() - target
    loss = 0.5 * (off * off).mean()
    grad_h = (off / off.numel() * 1024).to(dtype)  # scaled up: float16 keeps small gradients
    grads = {}
    dx, df, _, grads["w_post"], grads["res_scale"], grads["w_pre"] = sp.block_norm_bwd(
        y, torch.zeros_like(y), grad_h, **norm)
    dnear, grads["w_gate"], grads["w_up"], grads["w_down"] = sp.gated_ffn_bwd(
        near, p["w_gate"], p["w_up"], p["w_down"], df)
    dconv = sp.tp_conv_bwd(conv, x.float(), sh, edge_w, dnear.float(), src, dst, perm, n_nodes=n)[0]
    grads["table"] = sp.embedding_bwd((dx.float() + dconv).to(dtype), species, SPECIES, scale=DIM ** 0.5)
    return loss, {k: v.float() / 1024 for k, v in grads.items()}


def train(steps=30, dtype="f32", n_nodes=2000, degree=8, rate=10.0, seed=0):
    conv = sp.tp_create(f"{DIM}x0e", "0e+1o", "0e", layout="ir_mul")
    graph = make_graph(n_nodes, degree, seed)
    p = make_weights(DTYPES[dtype], seed + 1)
    master = {k: v.float() for k, v in p.items()}
    losses = []
    for _ in range(steps):
        loss, grads = step(conv, graph, p)
        losses.append(loss.item())
        for k in p:
            master[k] -= rate * grads[k]
            p[k].copy_(master[k])
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--dtype", choices=sorted(DTYPES), default="f32")
    a = ap.parse_args()
    for i, loss in enumerate(train(a.steps, a.dtype)):
        print(f"step {i:3d} loss {loss:.5f}")
