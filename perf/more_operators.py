"""The dense layer, dropout and the routing of rows to experts at real sizes:
inputs, the plain PyTorch form of each, the calls a user makes of the library,
the float64 value, and the work of one pass.

``own`` selects what :func:`run` does: the plain form (elementary operations
in float32, rounded once at the end) or this package's calls.
"""

import math

import torch

own = False

_T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # three rows through one layer with all of its epilogue: the weights are read once, latency counts
        dict(name="dense fwd few rows", op="dense", dir="fwd", dtype="bf16", n=3, d_in=1024, d_out=4096, act="gelu",
             bias=True, residual=True),
        # hidden layer of the edge network over the 600,000 edges of the large graph workload
        dict(name="dense fwd edges", op="dense", dir="fwd", dtype="f32", n=600000, d_in=64, d_out=64, act="silu",
             bias=True, residual=False),
        # its gradient, each weight a sum over all edges
        dict(name="dense bwd edges", op="dense", dir="bwd", dtype="f32", n=600000, d_in=64, d_out=64, act="silu",
             bias=True),
        # ragged everything: rows, widths that are no multiple of 8
        dict(name="dense bwd ragged", op="dense", dir="bwd", dtype="f16", n=1357, d_in=322, d_out=853, act="gelu",
             bias=True),
        # a training step of a wide network's first layer
        dict(name="dense bwd training", op="dense", dir="bwd", dtype="bf16", n=8192, d_in=2048, d_out=5632, act="gelu",
             bias=True),
        # the end of a residual branch in a training step
        dict(name="dropout fwd training", op="dropout", dir="fwd", dtype="bf16", n=16384, dim=2048, p=0.1,
             mode="element", residual=True),
        # gradient on the invariant channels of the 20,000-node graph
        dict(name="dropout bwd nodes", op="dropout", dir="bwd", dtype="f32", n=20000, dim=128, p=0.2, mode="element"),
        # a serving step of a few rows: ordering and copies are latency only
        dict(name="route fwd few rows", op="route", dir="fwd", dtype="f16", idx="i64", n=5, k=2, experts=8, dim=1000),
        # many small experts, a training step's rows
        dict(name="route fwd training", op="route", dir="fwd", dtype="bf16", idx="i64", n=16384, k=8, experts=128,
             dim=2048),
        # gradient of the nodes of the 20,000-node graph, each by one expert of every two of its four
        dict(name="route bwd nodes", op="route", dir="bwd", dtype="f32", idx="i32", n=20000, k=2, experts=4, dim=128),
        # back to the rows' order in half precision, two experts a row, odd sizes
        dict(name="combine fwd ragged", op="combine", dir="fwd", dtype="f16", idx="i32", n=7001, k=2, experts=16,
             dim=1030, residual=True),
        # gradient of the training step's weighted sum
        dict(name="combine bwd training", op="combine", dir="bwd", dtype="bf16", idx="i64", n=16384, k=4, experts=64,
             dim=2048),
    ]


def _size(rng, lo, hi, multiple=1):
    """A size spread over the logarithm of [lo, hi], a multiple of `multiple` above it."""
    v = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    if multiple > 1 and v >= multiple:
        v -= v % multiple
    return v


def _width(rng, lo, hi):
    """Widths: multiples of 64 and of 8 mostly, any number (odd ones too) in a third of the cases."""
    return _size(rng, lo, hi, rng.choice([64, 8, 1]))


def draw(rng):
    op = rng.choice(["dense", "dense", "dropout", "route", "combine"])
    case = dict(op=op, dir=rng.choice(["fwd", "bwd"]), dtype=rng.choice(["f32", "bf16", "f16"]))
    fwd = case["dir"] == "fwd"
    if op == "dense":
        while True:
            case.update(n=_size(rng, 1, 600000), d_in=_width(rng, 8, 8192), d_out=_width(rng, 8, 8192),
                        act=rng.choice(["none", "silu", "gelu", "relu", "sigmoid"]), bias=rng.random() < 0.8)
            if fwd:
                case["residual"] = rng.random() < 0.4
            w = work(case)
            # in float32 and float64 alike no more than the largest listed cases
            if w["flops"] <= 5.6e11 and w["bytes"] <= 5.0e8:
                return case
    if op == "dropout":
        case.update(dim=_width(rng, 16, 8192), p=rng.choice([0.0, 0.05, 0.1, 0.3, 0.5]),
                    mode=rng.choice(["element", "element", "row"]))
        if fwd:
            case["residual"] = rng.random() < 0.5
        case["n"] = _size(rng, 1, max(16, min(600000, (1 << 25) // case["dim"])))
        return case
    case.update(idx=rng.choice(["i32", "i64"]), k=rng.choice([1, 2, 2, 3, 4, 6, 8]), experts=_size(rng, 2, 512),
                dim=_width(rng, 16, 8192))
    if op == "combine" and fwd:
        case["residual"] = rng.random() < 0.5
    case["n"] = _size(rng, 1, max(16, min(200000, (1 << 27) // (case["dim"] * (2 * case["k"] + 1)))))
    return case


def _chosen(case, gen):
    """k different experts a row, the low numbers more often; one entry in fifty without an expert (-1)."""
    n, k, e = case["n"], case["k"], case["experts"]
    if k <= e:
        liked = torch.linspace(0.0, 1.5, e, device="cuda")
        noise = -torch.log(-torch.log(torch.rand(n, e, generator=gen, device="cuda").clamp_(1e-9, 1 - 1e-7)))
        chosen = (noise - liked).topk(k, dim=1).indices
    else:
        chosen = torch.randint(0, e, (n, k), generator=gen, device="cuda")
    none = torch.rand(n, k, generator=gen, device="cuda") < 0.02
    chosen = torch.where(none, torch.full_like(chosen, -1), chosen)
    return chosen.to(torch.int32 if case["idx"] == "i32" else torch.int64).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = _T[case["dtype"]]

    def normal(*shape, std=1.0, dtype=t):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    s = dict(case=case)
    n, fwd = case["n"], case["dir"] == "fwd"
    if case["op"] == "dense":
        s["x"] = normal(n, case["d_in"])
        s["w"] = normal(case["d_out"], case["d_in"], std=1.0 / math.sqrt(case["d_in"]))
        s["bias"] = normal(case["d_out"], std=0.2) if case["bias"] else None
        if fwd:
            s["residual"] = normal(n, case["d_out"]) if case["residual"] else None
        else:
            s["grad_out"] = normal(n, case["d_out"])
    elif case["op"] == "dropout":
        s["seed"] = torch.randint(0, 1 << 62, (2,), generator=gen, device="cuda")
        s["x" if fwd else "grad_out"] = normal(n, case["dim"])
        if fwd:
            s["residual"] = normal(n, case["dim"]) if case["residual"] else None
    else:
        k, d = case["k"], case["dim"]
        s["experts"] = _chosen(case, gen)
        if case["op"] == "route" and fwd:
            s["x"] = normal(n, d)
            return s
        # what the forward pass left: the place of every entry in the order by expert, and each expert's range
        _, s["place"], s["offsets"], _ = _sorted(s["experts"], case["experts"])
        if case["op"] == "route":
            s["grad_xs"] = normal(n * k, d)
            return s
        s["weights"] = torch.rand(n, k, generator=gen, device="cuda") + 0.1
        s["weights"] /= s["weights"].sum(1, keepdim=True)
        s["ys"] = normal(n * k, d)
        if fwd:
            s["residual"] = normal(n, d) if case["residual"] else None
        else:
            s["grad_out"] = normal(n, d)
    return s


# ------------------------------------------------------------ the library's calls

def _run_own(s):
    import segmented_polynomials_amd as sp
    c = s["case"]
    fwd = c["dir"] == "fwd"
    if c["op"] == "dense":
        if fwd:
            return {"out": sp.dense_fwd(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"])}
        dx, dw, db = sp.dense_bwd(s["x"], s["w"], s["grad_out"], bias=s["bias"], act=c["act"])
        return {"grad_x": dx, "grad_w": dw, "grad_bias": db}
    if c["op"] == "dropout":
        if fwd:
            return {"out": sp.dropout_fwd(s["x"], c["p"], s["seed"], residual=s["residual"], mode=c["mode"])}
        return {"grad_x": sp.dropout_bwd(s["grad_out"], c["p"], s["seed"], mode=c["mode"])}
    if c["op"] == "route":
        if fwd:
            order, place, offsets, ids = sp.expert_sort(s["experts"], c["experts"])
            return {"order": order, "place": place, "offsets": offsets, "ids": ids,
                    "xs": sp.expert_dispatch_fwd(s["x"], place, offsets)}
        return {"grad_x": sp.expert_dispatch_bwd(s["grad_xs"], s["place"], s["offsets"])}
    if fwd:
        return {"out": sp.expert_combine_fwd(s["ys"], s["place"], s["offsets"], s["weights"], residual=s["residual"])}
    dys, dw = sp.expert_combine_bwd(s["grad_out"], s["ys"], s["place"], s["offsets"], s["weights"])
    return {"grad_ys": dys, "grad_weights": dw}


# ------------------------------------------------------------ the plain forms

def _act(z, act):
    """The activation and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * p, p + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "relu":
        m = (z > 0).to(z.dtype)
        return z * m, m
    s = 1 / (1 + torch.exp(-z))
    return s, s * (1 - s)


_M32 = 0xFFFFFFFF


def _philox(c, key):
    """Four words of Philox 4x32-10 in int64, whose products keep their low 64 bits."""
    k0, k1 = key
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & _M32) ^ c[1] ^ k0, b & _M32, ((a >> 32) & _M32) ^ c[3] ^ k1, a & _M32]
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    return c


def _kept(seed, n, columns, p):
    """keep[row, col]: the word col % 4 of the counter (col / 4, row, offset) is not below p 2^32."""
    row = torch.arange(n, device="cuda")[:, None].expand(n, (columns + 3) // 4)
    col = torch.arange((columns + 3) // 4, device="cuda")[None].expand_as(row)
    lo, hi = seed & _M32, (seed >> 32) & _M32
    words = _philox([col, row, lo[1], hi[1]], (lo[0], hi[0]))
    return torch.stack(words, 2).reshape(n, -1)[:, :columns] >= round(p * 2.0 ** 32)


def _sorted(experts, num):
    """Entries in the order of their expert, those without one last: order, its inverse, ranges, sorted numbers."""
    flat = experts.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < num), flat, torch.full_like(flat, num))
    ids, order = torch.sort(flat, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device="cuda")
    count = torch.zeros(num + 1, dtype=torch.int64, device="cuda").index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([torch.zeros_like(count[:1]), torch.cumsum(count[:num], 0)])
    ids = torch.where(ids < num, ids, torch.full_like(ids, -1))
    return order.int(), place.reshape(experts.shape).int(), offsets.int(), ids.int()


def _run_plain(s):
    c = s["case"]
    t = _T[c["dtype"]]
    fwd = c["dir"] == "fwd"
    if c["op"] == "dense":
        x, w = s["x"].float(), s["w"].float()
        z = x @ w.T
        if s["bias"] is not None:
            z = z + s["bias"].float()
        a, da = _act(z, c["act"])
        if fwd:
            return {"out": (a if s["residual"] is None else a + s["residual"].float()).to(t)}
        d = s["grad_out"].float() * da
        return {"grad_x": (d @ w).to(t), "grad_w": (d.T @ x).to(t),
                "grad_bias": None if s["bias"] is None else d.sum(0).to(t)}
    if c["op"] == "dropout":
        v = s["x" if fwd else "grad_out"]
        keep = _kept(s["seed"], c["n"], c["dim"] if c["mode"] == "element" else 1, c["p"])
        v = torch.where(keep, v.float() * (1 / (1 - c["p"])), torch.zeros((), device="cuda"))
        if fwd:
            return {"out": (v if s["residual"] is None else v + s["residual"].float()).to(t)}
        return {"grad_x": v.to(t)}
    n, k, d = c["n"], c["k"], c["dim"]
    if c["op"] == "route" and fwd:
        order, place, offsets, ids = _sorted(s["experts"], c["experts"])
        xs = s["x"].float()[order.long() // k] * (ids >= 0)[:, None]
        return {"order": order, "place": place, "offsets": offsets, "ids": ids, "xs": xs.to(t)}
    place = s["place"].long()
    used = place < s["offsets"][-1]
    if c["op"] == "route":
        return {"grad_x": (s["grad_xs"].float()[place] * used[:, :, None]).sum(1).to(t)}
    w = s["weights"] * used
    if fwd:
        out = (s["ys"].float()[place] * w[:, :, None]).sum(1)
        return {"out": (out if s["residual"] is None else out + s["residual"].float()).to(t)}
    g = s["grad_out"].float()
    dys = torch.empty(n * k, d, device="cuda")
    dys[place.reshape(-1)] = (g[:, None] * w[:, :, None]).reshape(n * k, d)
    return {"grad_ys": dys.to(t), "grad_weights": (s["ys"].float()[place] * g[:, None]).sum(2) * used}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------ the value in 64 bits

def _high_low(a, m):
    """The two halves of the 64-bit product of 32-bit numbers, from products of 16-bit digits."""
    a1, a0, m1, m0 = a >> 16, a & 0xFFFF, m >> 16, m & 0xFFFF
    low = a0 * m0
    middle = a1 * m0 + (low >> 16)
    cross = a0 * m1 + (middle & 0xFFFF)
    return a1 * m1 + (middle >> 16) + (cross >> 16), ((cross & 0xFFFF) << 16) | (low & 0xFFFF)


def _exact_kept(seed, n, columns, p):
    key0, key1 = int(seed[0]) % 2 ** 32, int(seed[0]) >> 32 & 0xFFFFFFFF
    offset = int(seed[1]) % 2 ** 64
    rows, cols = torch.meshgrid(torch.arange(n, device="cuda"), torch.arange((columns + 3) // 4, device="cuda"),
                                indexing="ij")
    x, y = cols.clone(), rows.clone()
    z = torch.full_like(x, offset % 2 ** 32)
    u = torch.full_like(x, offset >> 32)
    for r in range(10):
        h0, l0 = _high_low(x, 0xD2511F53)
        h1, l1 = _high_low(z, 0xCD9E8D57)
        x, y, z, u = (h1 ^ y ^ ((key0 + r * 0x9E3779B9) % 2 ** 32), l1,
                      h0 ^ u ^ ((key1 + r * 0xBB67AE85) % 2 ** 32), l0)
    word = torch.empty(n, (columns + 3) // 4, 4, dtype=torch.int64, device="cuda")
    for i, v in enumerate((x, y, z, u)):
        word[:, :, i] = v
    return word.view(n, -1)[:, :columns] >= round(p * 2.0 ** 32)


def _exact_order(experts, num):
    """Entry numbers as the low digits of a key: all keys differ, any sort will do."""
    flat = experts.reshape(-1).to(torch.int64)
    flat = flat.masked_fill((flat < 0) | (flat >= num), num)
    m = flat.numel()
    order = torch.sort(flat * m + torch.arange(m, device="cuda"))[0] % m
    place = torch.argsort(order)
    ids = flat.index_select(0, order)
    offsets = torch.searchsorted(ids, torch.arange(num + 1, device="cuda"))
    return order, place.view(experts.shape), offsets, ids.masked_fill(ids == num, -1)


def exact(case, seed):
    """The definition in float64; gradients by automatic differentiation of it."""
    s = prepare(case, seed)
    fwd = case["dir"] == "fwd"
    leaf = {k: s[k].double().requires_grad_(not fwd) for k in ("x", "w", "bias", "ys", "weights")
            if isinstance(s.get(k), torch.Tensor)}
    res = s.get("residual")
    if case["op"] == "dense":
        import torch.nn.functional as F
        act = {"none": lambda v: v, "silu": F.silu, "gelu": F.gelu, "relu": F.relu, "sigmoid": torch.sigmoid}[case["act"]]
        out = act(F.linear(leaf["x"], leaf["w"], leaf.get("bias")))
        if fwd:
            return {"out": out if res is None else res.double() + out}
        keys = [k for k in ("x", "w", "bias") if k in leaf]
        g = dict(zip(keys, torch.autograd.grad(out, [leaf[k] for k in keys], s["grad_out"].double())))
        return {"grad_x": g["x"], "grad_w": g["w"], "grad_bias": g.get("bias")}
    if case["op"] == "dropout":
        keep = _exact_kept(s["seed"], case["n"], case["dim"] if case["mode"] == "element" else 1, case["p"])
        if fwd:
            out = leaf["x"].masked_fill(~keep, 0.0) / (1.0 - case["p"])
            return {"out": out if res is None else res.double() + out}
        return {"grad_x": s["grad_out"].double().masked_fill(~keep, 0.0) / (1.0 - case["p"])}
    n, k, d = case["n"], case["k"], case["dim"]
    order, place, offsets, ids = _exact_order(s["experts"], case["experts"])
    row = torch.div(order, k, rounding_mode="floor")
    kept = int(offsets[-1])
    if case["op"] == "route":
        if fwd:
            xs = leaf["x"].index_select(0, row)
            xs[kept:] = 0
            return {"order": order, "place": place, "offsets": offsets, "ids": ids, "xs": xs}
        gx = torch.zeros(n, d, dtype=torch.float64, device="cuda")
        return {"grad_x": gx.scatter_add_(0, row[:kept, None].expand(-1, d), s["grad_xs"][:kept].double())}
    # as sums over the sorted entries
    share = leaf["weights"].reshape(-1).index_select(0, order[:kept])
    out = torch.zeros(n, d, dtype=torch.float64, device="cuda")
    out = out.scatter_add(0, row[:kept, None].expand(-1, d), leaf["ys"][:kept] * share[:, None])
    if fwd:
        return {"out": out if res is None else res.double() + out}
    g = torch.autograd.grad(out, (leaf["ys"], leaf["weights"]), s["grad_out"].double())
    return {"grad_ys": g[0], "grad_weights": g[1]}


# ------------------------------------------------------------ the work of one pass

def work(case):
    e = _BYTES[case["dtype"]]
    n, fwd = case["n"], case["dir"] == "fwd"
    if case["op"] == "dense":
        di, do = case["d_in"], case["d_out"]
        bias = do if case["bias"] else 0
        if fwd:
            return {"bytes": e * (n * (di + do * (2 if case["residual"] else 1)) + di * do + bias),
                    "flops": 2 * n * di * do}
        # the product again unless there is no activation, then the two gradients
        return {"bytes": e * (n * (2 * di + do) + 2 * (di * do + bias)),
                "flops": 2 * n * di * do * (2 if case["act"] == "none" else 3)}
    if case["op"] == "dropout":
        d = case["dim"]
        return {"bytes": e * n * d * (3 if fwd and case["residual"] else 2) + 16, "flops": 2 * n * d}
    k, d, num = case["k"], case["dim"], case["experts"]
    idx = 4 if case["idx"] == "i32" else 8
    if case["op"] == "route":
        if fwd:
            return {"bytes": n * k * (idx + 12) + 4 * (num + 1) + e * n * d * (1 + k), "flops": n * k}
        return {"bytes": n * k * 4 + 4 + e * n * d * (1 + k), "flops": n * k * d}
    if fwd:
        return {"bytes": n * k * 8 + 4 + e * n * d * (k + (2 if case["residual"] else 1)), "flops": 2 * n * k * d}
    return {"bytes": n * k * 12 + 4 + e * n * d * (1 + 2 * k), "flops": 3 * n * k * d}
