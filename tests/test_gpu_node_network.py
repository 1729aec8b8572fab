"""The example network: its gradients agree with automatic differentiation
of the same network in plain float64 operations, and it learns."""

import pytest
import torch

from tests._gpu import announce, need_gpu

pytestmark = pytest.mark.gpu


def test_gradients():
    need_gpu()
    import segmented_polynomials_amd as sp
    from examples import node_network as net
    announce("node network: gradients, float32")
    n = 300
    conv = sp.tp_create(f"{net.DIM}x0e", "0e+1o", "0e", layout="ir_mul")
    graph = net.make_graph(n, 5, 3)
    p = net.make_weights(torch.float32, 4)
    loss, grads = net.step(conv, graph, p)
    species, src, dst, sh, target = graph
    # the one path 0e x 0e -> 0e is a product with sh[:, 0]; its constant from one edge of ones
    one = torch.ones(1, net.DIM, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    e0 = torch.zeros(1, sh.shape[1], device="cuda")
    e0[0, 0] = 1
    c = sp.tp_conv_fwd(conv, one, e0, one[:, :conv.weight_numel], zero, zero, n_nodes=1)[0, 0].item()
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    x = q["table"][species.long()] * net.DIM ** 0.5
    msg = x[src.long()] * (c * 0.5 * sh[:, :1].double())
    near = torch.zeros(n, net.DIM, dtype=torch.float64, device="cuda").index_add(0, dst.long(), msg)
    f = (torch.nn.functional.silu(near @ q["w_gate"].T) * (near @ q["w_up"].T)) @ q["w_down"].T

    def norm(v):
        v = v - v.mean(1, keepdim=True)
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)

    y = x + q["res_scale"] * q["w_post"] * norm(f)
    ref = 0.5 * ((norm(y) * q["w_pre"] - target.double()) ** 2).mean()
    ref.backward()
    # each gradient is a sum over n rows of values that a few hundred float32
    # operations made: 2^-24 times a few hundred, of the largest gradient
    assert abs(loss.item() - ref.item()) <= 512 * 2.0 ** -24 * ref.item()
    for k in p:
        off = (grads[k].double() - q[k].grad).abs().max().item()
        worst = off / q[k].grad.abs().max().item()
        print(f"[parity] {k}: {worst:.2e} of the largest gradient", flush=True)
        assert worst <= 512 * 2.0 ** -24, k


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_learns(dtype):
    need_gpu()
    from examples import node_network as net
    announce(f"node network: training, {dtype}")
    losses = net.train(steps=12, dtype=dtype, n_nodes=400, degree=4)
    print(losses)
    assert losses[-1] < 0.97 * losses[0]
