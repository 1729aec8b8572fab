"""The example network with an edge network and experts: it runs, and its
gradients agree with automatic differentiation of the same network in plain
float64 operations."""

import math

import numpy as np
import pytest
import torch

from tests._gpu import announce, need_gpu
from tests._philox import kept

pytestmark = pytest.mark.gpu


def test_gradients():
    need_gpu()
    import segmented_polynomials_amd as sp
    from examples import expert_network as net
    announce("expert network: gradients")
    n, count = 300, 5
    layers = conv, experts = net.make_layers()
    graph = net.make_graph(n, 5, 3)
    p = net.make_weights(conv, experts, 4)
    loss, grads, chosen = net.step(layers, graph, p, count)
    species, src, dst, sh, basis, target = graph
    # the one path 0e x 0e -> 0e is a product with sh[:, 0]; its constant from one edge of ones
    one = torch.ones(1, net.DIM, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    e0 = torch.zeros(1, sh.shape[1], device="cuda")
    e0[0, 0] = 1
    c = sp.tp_conv_fwd(conv, one, e0, one[:, :conv.weight_numel], zero, zero, n_nodes=1)[0, 0].item()
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    x = q["table"][species.long()]
    hidden = torch.nn.functional.silu(basis.double() @ q["w1"].T + q["b1"])
    edge_w = hidden @ q["w2"].T
    msg = x[src.long()] * edge_w * (c * sh[:, :1].double())
    near = torch.zeros(n, net.DIM, dtype=torch.float64, device="cuda").index_add(0, dst.long(), msg)
    scores = (near @ q["router"].T + q["router_bias"]).gather(1, chosen)
    share = torch.softmax(scores, 1)
    w = q["experts"].reshape(net.EXPERTS, net.DIM, net.DIM) / math.sqrt(net.DIM)  # [in, out], unit-variance outputs
    made = torch.stack([(near[:, None] @ w[chosen[:, j]])[:, 0] for j in range(net.CHOICES)], 1)
    branch = near + (share[:, :, None] * made).sum(1)
    keep = torch.from_numpy(np.array(kept(n, net.DIM, net.DROP, net.SEED, count))).cuda()
    y = x + torch.where(keep, branch / (1 - net.DROP), 0.0)
    ref = 0.5 * ((y - target.double()) ** 2).mean()
    ref.backward()
    # each gradient is a sum over n rows of values that a few hundred float32
    # operations made: 2^-24 times a few hundred, of the largest gradient
    assert abs(loss.item() - ref.item()) <= 512 * 2.0 ** -24 * ref.item()
    for k in p:
        off = (grads[k].double() - q[k].grad).abs().max().item()
        worst = off / q[k].grad.abs().max().item()
        print(f"[parity] {k}: {worst:.2e} of the largest gradient", flush=True)
        assert worst <= 512 * 2.0 ** -24, k


def test_runs():
    need_gpu()
    from examples import expert_network as net
    announce("expert network: training")
    losses = net.train(steps=4, n_nodes=400, degree=4)
    assert len(losses) == 4 and all(math.isfinite(v) for v in losses)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_experts_of_dense_layers(dtype):
    """The sorted rows of each expert through a dense layer of its own, forward
    and backward, against the same layers on gathered rows."""
    need_gpu()
    import segmented_polynomials_amd as sp
    announce(f"experts of dense layers {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    n, k, num, d, hidden = 400, 2, 5, 72, 40
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)
    x, w, b = r(n, d), r(num, hidden, d) * 0.1, r(num, hidden)
    chosen = torch.randint(-1, num - 1, (n, k), generator=g, device="cuda")  # the last has no row
    order, place, offsets, ids = sp.expert_sort(chosen, num)
    xs = sp.expert_dispatch_fwd(x, place, offsets)
    ends = offsets.tolist()
    assert ends[num - 1] == ends[num]
    ys, gy = torch.zeros(n * k, hidden, dtype=dtype, device="cuda"), r(n * k, hidden)
    dxs = torch.zeros_like(xs)
    for e in range(num):
        rows = slice(ends[e], ends[e + 1])
        sp.dense_fwd(xs[rows], w[e], bias=b[e], act="gelu", out=ys[rows])
        dxs[rows], dw, db = sp.dense_bwd(xs[rows], w[e], gy[rows], bias=b[e], act="gelu")
        at = torch.nonzero(chosen.reshape(-1) == e)[:, 0]
        alone = x[at // k].contiguous()
        assert torch.equal(ys[rows], sp.dense_fwd(alone, w[e], bias=b[e], act="gelu"))
        same = sp.dense_bwd(alone, w[e], gy[rows], bias=b[e], act="gelu")
        assert torch.equal(dxs[rows], same[0]) and torch.equal(dw, same[1]) and torch.equal(db, same[2])
    share = torch.rand(n, k, generator=g, device="cuda")
    out = sp.expert_combine_fwd(ys, place, offsets, share)
    used = (chosen >= 0)
    ref = (ys.double()[place.long()] * (share * used).double()[:, :, None]).sum(1)
    assert ((out.double() - ref).abs() <= torch.finfo(dtype).eps * (ref.abs() + 1)).all()
