"""What the gated feed-forward block's accuracy is measured by: its value in
float64, its value with chosen roundings in between, and the root mean square
error that float32 arithmetic explains."""

import math

import torch

NAMES = ("out", "grad_x", "grad_w_gate", "grad_w_up", "grad_w_down")


def same(t):
    return t


def block(x, wg, wu, wd, gy, product=torch.mm, hidden=same, dh_held=same, activation=None):
    """out and the gradients, silu: ``product`` for every product, ``hidden``
    applied to h, dg and du, ``dh_held`` to dh."""
    g, u = product(x, wg.T), product(x, wu.T)
    s = torch.sigmoid(g)
    a, da = g * s, s * (1 + g * (1 - s))
    h = hidden(a * u)
    dh = dh_held(product(gy, wd))
    dg, du = hidden(dh * u * da), hidden(dh * a)
    return (product(h, wd.T), product(dg, wg) + product(du, wu), product(dg.T, x), product(du.T, x), product(gy.T, h))


def planes_product(pairs):
    """A product of float32 matrices as the products of some pairs of their bf16
    planes, summed in float64."""
    def planes(t):
        out, rest = [], t.float()
        for _ in range(3):
            out.append(rest.bfloat16().float())
            rest = rest - out[-1]
        return [p.double() for p in out]

    def product(a, b):
        pa, pb = planes(a), planes(b)
        return sum(pa[i] @ pb[j] for i, j in pairs)

    return product


ALL_PAIRS = [(0, 0), (0, 1), (1, 0), (1, 1), (0, 2), (2, 0)]


def float32_rms(n, di, F, do):
    """Root mean square errors, relative to the outputs' root mean square, that
    float32 sums explain.  One addition is off by 0.41 2^-24 of its result, root
    mean square; a sum of K random terms one after another by 0.29 sqrt(K) 2^-24 of
    its own size, its partial sums being sqrt(k / K) of it.  Per sum in the chain that
    leads to an output half sqrt(K) 2^-24 is allowed, and 6 2^-24 for the activation,
    the products and the roundings of what is held."""
    r = lambda *sums: 2.0 ** -24 * (6 + 0.5 * sum(math.sqrt(k) for k in sums))
    return dict(zip(NAMES, (r(di, F), r(di, do, 2 * F), r(di, do, n), r(di, do, n), r(di, n))))


def rms_error(got, ref):
    return ((got.double() - ref).square().mean().sqrt() / ref.square().mean().sqrt()).item()


def unequal(got, ref, dtype):
    """Share of the elements that are not the reference's rounded value."""
    return (got.to(dtype) != ref.to(dtype)).double().mean().item()


# sums in float32 leave a value within 2^-7 of a step of where it rounds, a few
# steps of the hidden values that round the other way move an output by less than a
# step of its own
UNEQUAL = 0.1

SHAPES_F32 = [(33, 2048, 96, 2048), (5, 333, 1001, 77), (64, 64, 1500, 200), (130, 322, 853, 257), (300, 512, 512, 512),
              (700, 1500, 96, 1030)]
SHAPES_16 = [(70, 200, 520, 65), (130, 322, 853, 257), (700, 64, 64, 64), (300, 512, 512, 512)]


def inputs(n, di, F, do, seed, device, dtype=torch.float32):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=device) * std).to(dtype)
    return r(n, di), r(F, di, std=di ** -0.5), r(F, di, std=di ** -0.5), r(do, F, std=F ** -0.5), r(n, do)
