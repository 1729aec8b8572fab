"""A small trained message-passing layer with an edge network and a mixture of
experts on its nodes:

    edge network   two dense layers make the convolution's weight rows from
                   a radial basis of the edge lengths
    convolution    the fused tensor product of node features and harmonics
    router         a dense layer scores the experts, each node takes two
    experts        rows sorted by expert, one linear layer with a weight per
                   expert, rows back with the router's weights
    residual       dropout of the branch, added to the node features

    python examples/expert_network.py [--steps 20]

The five steps run in the library's kernels, forward and backward.  PyTorch's are
the choice of the experts (top-k, the softmax of their scores and its gradient), the
order of the edges by source, the sums of gradients of one tensor, the loss and the
weight update.  Float32 (the class-indexed linear layer's type); data: seeded random
graph and targets.
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import segmented_polynomials_amd as sp

SPECIES, DIM, BASIS, HIDDEN, EXPERTS, CHOICES = 10, 64, 8, 48, 6, 2
DROP, SEED = 0.2, 11


def make_graph(n_nodes, degree, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    species = torch.randint(0, SPECIES, (n_nodes,), generator=g, device="cuda", dtype=torch.int32)
    dst = torch.arange(n_nodes, device="cuda", dtype=torch.int32).repeat_interleave(degree)
    src = torch.randint(0, n_nodes, (n_nodes * degree,), generator=g, device="cuda", dtype=torch.int32)
    vec = torch.randn(n_nodes * degree, 3, generator=g, device="cuda")
    centres = torch.linspace(0.0, 3.0, BASIS, device="cuda")
    basis = torch.exp(-4 * (vec.norm(dim=1, keepdim=True) - centres) ** 2)
    target = torch.randn(n_nodes, DIM, generator=g, device="cuda")
    return species, src, dst, sp.sh_fwd(vec, 1), basis, target


def make_layers():
    conv = sp.tp_create(f"{DIM}x0e", "0e+1o", "0e", layout="ir_mul")
    experts = sp.linear_create(f"{DIM}x0e", f"{DIM}x0e")
    return conv, experts


def make_weights(conv, experts, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    return dict(table=normal(SPECIES, DIM), w1=normal(HIDDEN, BASIS, std=BASIS ** -0.5), b1=normal(HIDDEN, std=0.1),
                w2=normal(conv.weight_numel, HIDDEN, std=0.3 * HIDDEN ** -0.5), router=normal(EXPERTS, DIM, std=DIM ** -0.5),
                router_bias=normal(EXPERTS, std=0.1), experts=normal(EXPERTS, experts.weight_numel))


def step(layers, graph, p, count):
    """Loss, gradients and the chosen experts of one pass; ``count`` is the
    step's number, the dropout's offset."""
    conv, experts = layers
    species, src, dst, sh, basis, target = graph
    n = species.shape[0]
    perm = torch.argsort(src, stable=True).int()

    x = sp.embedding_fwd(p["table"], species)
    hidden = sp.dense_fwd(basis, p["w1"], bias=p["b1"], act="silu")
    edge_w = sp.dense_fwd(hidden, p["w2"])
    near = sp.tp_conv_fwd(conv, x, sh, edge_w, src, dst, n_nodes=n)
    scores, chosen = sp.dense_fwd(near, p["router"], bias=p["router_bias"]).topk(CHOICES, dim=1)
    share = torch.softmax(scores, 1)
    order, place, offsets, ids = sp.expert_sort(chosen, EXPERTS)
    rows = sp.expert_dispatch_fwd(near, place, offsets)
    made = sp.linear_fwd(experts, rows, p["experts"], classes=ids)
    branch = sp.expert_combine_fwd(made, place, offsets, share, residual=near)
    y = sp.dropout_fwd(branch, DROP, SEED, offset=count, residual=x)

    off = y - target
    loss = 0.5 * (off * off).mean()
    grad_y = off / off.numel()
    grads = {}
    dbranch = sp.dropout_bwd(grad_y, DROP, SEED, offset=count)
    dmade, dshare = sp.expert_combine_bwd(dbranch, made, place, offsets, share)
    drows, grads["experts"] = sp.linear_bwd(experts, rows, p["experts"], dmade, classes=ids)
    dscores = share * (dshare - (share * dshare).sum(1, keepdim=True))
    dlogits = torch.zeros(n, EXPERTS, device="cuda").scatter_(1, chosen, dscores)
    drouted, grads["router"], grads["router_bias"] = sp.dense_bwd(near, p["router"], dlogits, bias=p["router_bias"])
    dnear = dbranch + sp.expert_dispatch_bwd(drows, place, offsets) + drouted
    dx, _, dedge = sp.tp_conv_bwd(conv, x, sh, edge_w, dnear, src, dst, perm, n_nodes=n)
    dhidden, grads["w2"], _ = sp.dense_bwd(hidden, p["w2"], dedge)
    _, grads["w1"], grads["b1"] = sp.dense_bwd(basis, p["w1"], dhidden, bias=p["b1"], act="silu", need_dx=False)
    grads["table"] = sp.embedding_bwd(grad_y + dx, species, SPECIES)
    return loss, grads, chosen


def train(steps=20, n_nodes=2000, degree=8, rate=2.0, seed=0):
    layers = make_layers()
    graph = make_graph(n_nodes, degree, seed)
    p = make_weights(*layers, seed + 1)
    losses = []
    for count in range(steps):
        loss, grads, _ = step(layers, graph, p, count)
        losses.append(loss.item())
        for k in p:
            p[k] -= rate * grads[k]
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--steps", type=int, default=20)
    for i, loss in enumerate(train(ap.parse_args().steps)):
        print(f"step {i:3d} loss {loss:.5f}")
