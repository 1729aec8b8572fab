"""The invariant-channel operators (embedding, block norm, gated feed-forward)
at real sizes: inputs, the plain PyTorch form of each, the calls a user makes
of the library, the float64 value, and the work of one pass.

``own`` selects what :func:`run` does: the plain form (elementary operations
in float32, rounded once at the end) or this package's calls.
"""

import math

import torch

own = False

_T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
# a size no drawn case takes
_SKIP = 3072


def listed():
    return [
        # the species embedding of the 20,000-node graph workload, 128 channels
        dict(name="embed fwd species", op="embedding", dir="fwd", dtype="f32", idx="i32", n=20000, rows=10, dim=128,
             scale=1.0),
        # a token table of a language model, rows scaled by sqrt(dim), a batch of 8 x 4096 tokens
        dict(name="embed fwd vocabulary", op="embedding", dir="fwd", dtype="bf16", idx="i64", n=32768, rows=65536,
             dim=2048, scale=math.sqrt(2048)),
        # gradient of the species embedding over 50,000 atoms: 10 rows, each a sum of thousands
        dict(name="embed bwd species", op="embedding", dir="bwd", dtype="f32", idx="i32", n=50000, rows=10, dim=128,
             scale=1.0),
        # gradient of a token table, most rows without a token, a few with hundreds
        dict(name="embed bwd vocabulary", op="embedding", dir="bwd", dtype="bf16", idx="i64", n=16384, rows=32768,
             dim=1024, scale=32.0),
        # a serving step of a few sequences, a width that is no multiple of a wave
        dict(name="norm fwd few rows", op="block_norm", dir="fwd", dtype="f16", n=5, dim=1000, kind="rms", gate="none",
             gate_act="none", res_scale=True, next_norm=True),
        # between two blocks of a training step, elementwise sigmoid gate
        dict(name="norm fwd training", op="block_norm", dir="fwd", dtype="bf16", n=16384, dim=2048, kind="rms",
             gate="element", gate_act="sigmoid", res_scale=True, next_norm=True),
        # invariant channels of the 20,000-node graph, layer norm, one gate per node
        dict(name="norm bwd nodes", op="block_norm", dir="bwd", dtype="f32", n=20000, dim=128, kind="layer", gate="row",
             gate_act="none", res_scale=True, next_norm=True),
        # backward of the training step at a larger width
        dict(name="norm bwd training", op="block_norm", dir="bwd", dtype="bf16", n=8192, dim=4096, kind="rms",
             gate="element", gate_act="sigmoid", res_scale=True, next_norm=True),
        # three sequences, one token each: the weights are read once, latency counts
        dict(name="ffn fwd few rows", op="gated_ffn", dir="fwd", dtype="bf16", n=3, d_in=1024, hidden=4096, d_out=1024,
             act="silu"),
        # node update of the 20,000-node graph in the framework's own type
        dict(name="ffn fwd nodes", op="gated_ffn", dir="fwd", dtype="f32", n=20000, d_in=128, hidden=512, d_out=128,
             act="silu"),
        # ragged everything: rows, widths that are no multiple of 8, another output width
        dict(name="ffn bwd ragged", op="gated_ffn", dir="bwd", dtype="f16", n=1357, d_in=322, hidden=853, d_out=257,
             act="gelu"),
        # a training step of a language model's block
        dict(name="ffn bwd training", op="gated_ffn", dir="bwd", dtype="bf16", n=8192, d_in=2048, hidden=5632,
             d_out=2048, act="silu"),
    ]


def _size(rng, lo, hi, multiple=1):
    """A size spread over the logarithm of [lo, hi], a multiple of `multiple` above it."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        v = max(lo, min(hi, v))
        if multiple > 1 and v >= multiple:
            v -= v % multiple
        if v != _SKIP:
            return v


def _width(rng, lo, hi):
    """Widths: multiples of 64 and of 8 mostly, any number (odd ones too) in a third of the cases."""
    return _size(rng, lo, hi, rng.choice([64, 8, 1]))


def draw(rng):
    op = rng.choice(["embedding", "block_norm", "gated_ffn"])
    case = dict(op=op, dir=rng.choice(["fwd", "bwd"]), dtype=rng.choice(["f32", "bf16", "f16"]))
    if op == "embedding":
        case.update(idx=rng.choice(["i32", "i64"]), rows=_size(rng, 4, 65536), dim=_width(rng, 32, 2048),
                    scale=rng.choice([1.0, 0.5, 11.3]))
        case["n"] = _size(rng, 1, max(16, min(131072, (1 << 25) // case["dim"])))
    elif op == "block_norm":
        case.update(dim=_width(rng, 32, 8192), kind=rng.choice(["rms", "layer"]),
                    gate=rng.choice(["none", "row", "element"]), gate_act=rng.choice(["none", "sigmoid"]),
                    res_scale=rng.random() < 0.7, next_norm=rng.random() < 0.8)
        case["n"] = _size(rng, 1, max(16, min(65536, (1 << 24) // case["dim"])))
    else:
        while True:
            case.update(n=_size(rng, 1, 16384), d_in=_width(rng, 48, 2048), hidden=_width(rng, 64, 8192),
                        d_out=_width(rng, 48, 2048), act=rng.choice(["silu", "gelu", "relu", "sigmoid"]))
            # in float32 and float64 alike no more than the largest listed case
            if work(case)["flops"] <= 1.0e12:
                break
    return case


def _tokens(case, gen):
    """Token ids with the spread of a text (a few frequent ones) and 3 % padding (-1) over large tables;
    the even spread of elements over small ones."""
    n, rows = case["n"], case["rows"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    if rows > 256:
        t = (torch.exp(u * math.log(rows)) - 1).long().clamp_(0, rows - 1)
        pad = torch.rand(n, generator=gen, device="cuda") < 0.03
        t = torch.where(pad, torch.full_like(t, -1), t)
    else:
        t = (u * rows).long().clamp_(0, rows - 1)
    return t.to(torch.int32 if case["idx"] == "i32" else torch.int64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = _T[case["dtype"]]

    def normal(*shape, std=1.0, dtype=t):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    s = dict(case=case)
    if case["op"] == "embedding":
        s["tokens"] = _tokens(case, gen)
        if case["dir"] == "fwd":
            s["table"] = normal(case["rows"], case["dim"], std=1.0 / math.sqrt(case["dim"]))
        else:
            s["grad_out"] = normal(case["n"], case["dim"])
    elif case["op"] == "block_norm":
        n, d = case["n"], case["dim"]
        s["f"] = normal(n, d, std=0.7)
        s["gate"] = None if case["gate"] == "none" else normal(n, 1 if case["gate"] == "row" else d)
        s["w_post"] = 1 + normal(d, std=0.1, dtype=torch.float32)
        s["res_scale"] = 0.3 + normal(d, std=0.05, dtype=torch.float32) if case["res_scale"] else None
        s["w_pre"] = 1 + normal(d, std=0.1, dtype=torch.float32) if case["next_norm"] else None
        s["x"] = normal(n, d, std=1.5)  # the residual stream: x of the forward, y of the backward
        if case["dir"] == "bwd":
            s["grad_y"] = normal(n, d)
            s["grad_h"] = normal(n, d) if case["next_norm"] else None
    else:
        n, di, f, do = case["n"], case["d_in"], case["hidden"], case["d_out"]
        s["x"] = normal(n, di)
        s["w_gate"] = normal(f, di, std=1.0 / math.sqrt(di))
        s["w_up"] = normal(f, di, std=1.0 / math.sqrt(di))
        s["w_down"] = normal(do, f, std=1.0 / math.sqrt(f))
        if case["dir"] == "bwd":
            s["grad_out"] = normal(n, do)
    return s


# ------------------------------------------------------------ the library's calls

def _run_own(s):
    import segmented_polynomials_amd as sp
    c = s["case"]
    if c["op"] == "embedding":
        if c["dir"] == "fwd":
            return {"out": sp.embedding_fwd(s["table"], s["tokens"], scale=c["scale"])}
        return {"grad_table": sp.embedding_bwd(s["grad_out"], s["tokens"], c["rows"], scale=c["scale"])}
    if c["op"] == "block_norm":
        kw = dict(f=s["f"], gate=s["gate"], w_post=s["w_post"], res_scale=s["res_scale"], w_pre=s["w_pre"],
                  kind=c["kind"], gate_act=c["gate_act"], eps=1e-6)
        if c["dir"] == "fwd":
            y, h = sp.block_norm_fwd(s["x"], **kw)
            return {"y": y, "h": h}
        dx, df, dgate, dpost, dscale, dpre = sp.block_norm_bwd(s["x"], s["grad_y"], s["grad_h"], **kw)
        return {"grad_x": dx, "grad_f": df, "grad_gate": dgate, "grad_w_post": dpost, "grad_res_scale": dscale,
                "grad_w_pre": dpre}
    w = (s["w_gate"], s["w_up"], s["w_down"])
    if c["dir"] == "fwd":
        return {"out": sp.gated_ffn_fwd(s["x"], *w, act=c["act"])}
    dx, dg, du, dd = sp.gated_ffn_bwd(s["x"], *w, s["grad_out"], act=c["act"])
    return {"grad_x": dx, "grad_w_gate": dg, "grad_w_up": du, "grad_w_down": dd}


# ------------------------------------------------------------ the plain forms

def _norm(v, kind, eps=1e-6):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
    return v * r, r


def _norm_vjp(g, nv, r, kind):
    d = g - nv * (g * nv).mean(-1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(-1, keepdim=True)
    return d * r


def _act(g, act):
    """The activation and its derivative."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    if act == "relu":
        m = (g > 0).to(g.dtype)
        return g * m, m
    s = 1 / (1 + torch.exp(-g))
    return s, s * (1 - s)


def _run_plain(s):
    c = s["case"]
    t = _T[c["dtype"]]
    if c["op"] == "embedding":
        tok = s["tokens"].long()
        ok = (tok >= 0) & (tok < c["rows"])
        tok = tok.clamp(0, c["rows"] - 1)
        if c["dir"] == "fwd":
            return {"out": (s["table"][tok].float() * (c["scale"] * ok[:, None])).to(t)}
        g = s["grad_out"].float() * ok[:, None]
        d = torch.zeros(c["rows"], c["dim"], device=g.device).index_add_(0, tok, g)
        return {"grad_table": (d * c["scale"]).to(t)}
    if c["op"] == "block_norm":
        kind, f, x = c["kind"], s["f"].float(), s["x"].float()
        nf, rf = _norm(f, kind)
        v = nf * s["w_post"]
        if s["gate"] is None:
            gate, dact = torch.ones((), device=f.device), None
        else:
            gate = s["gate"].float()
            dact = torch.ones_like(gate)
            if c["gate_act"] == "sigmoid":
                gate = 1 / (1 + torch.exp(-gate))
                dact = gate * (1 - gate)
        rs = s["res_scale"] if s["res_scale"] is not None else torch.ones((), device=f.device)
        if c["dir"] == "fwd":
            y = x + rs * gate * v
            h = None if s["w_pre"] is None else (_norm(y, kind)[0] * s["w_pre"]).to(t)
            return {"y": y.to(t), "h": h}
        dy = s["grad_y"].float()
        dpre = None
        if s["w_pre"] is not None:
            ny, ry = _norm(x, kind)
            dh = s["grad_h"].float()
            dpre = (dh * ny).sum(0)
            dy = dy + _norm_vjp(dh * s["w_pre"], ny, ry, kind)
        dv = dy * rs * gate
        dgate = None
        if s["gate"] is not None:
            dgate = dy * rs * v
            if c["gate"] == "row":
                dgate = dgate.sum(-1, keepdim=True)
            dgate = (dgate * dact).to(t)
        drs = None if s["res_scale"] is None else (dy * gate * v).sum(0)
        return {"grad_x": dy.to(t), "grad_f": _norm_vjp(dv * s["w_post"], nf, rf, kind).to(t), "grad_gate": dgate,
                "grad_w_post": (dv * nf).sum(0), "grad_res_scale": drs, "grad_w_pre": dpre}
    x, wg, wu, wd = (s[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
    g, u = x @ wg.T, x @ wu.T
    a, da = _act(g, c["act"])
    if c["dir"] == "fwd":
        return {"out": ((a * u) @ wd.T).to(t)}
    dy = s["grad_out"].float()
    dh = dy @ wd
    dwd = dy.T @ (a * u)
    dg, du = dh * u * da, dh * a
    return {"grad_x": (dg @ wg + du @ wu).to(t), "grad_w_gate": (dg.T @ x).to(t), "grad_w_up": (du.T @ x).to(t),
            "grad_w_down": dwd.to(t)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------ the value in 64 bits

def _exact_norm(v, w, kind):
    mean = v.mean(1, keepdim=True) if kind == "layer" else 0
    var = ((v - mean) ** 2).sum(1, keepdim=True) / v.shape[1]
    return w * (v - mean) / torch.sqrt(var + 1e-6)


def exact(case, seed):
    """The definition in float64; gradients by automatic differentiation of it."""
    s = prepare(case, seed)
    leaf = {k: v.double().requires_grad_(case["dir"] == "bwd") for k, v in s.items()
            if isinstance(v, torch.Tensor) and k not in ("tokens", "grad_out", "grad_y", "grad_h")}
    if case["op"] == "embedding":
        tok = s["tokens"].long()
        keep = torch.nonzero((tok >= 0) & (tok < case["rows"]))[:, 0]
        if case["dir"] == "fwd":
            out = torch.zeros(case["n"], case["dim"], dtype=torch.float64, device="cuda")
            out[keep] = case["scale"] * leaf["table"].index_select(0, tok[keep])
            return {"out": out}
        d = torch.zeros(case["rows"], case["dim"], dtype=torch.float64, device="cuda")
        src = s["grad_out"].index_select(0, keep).double() * case["scale"]
        return {"grad_table": d.scatter_add_(0, tok[keep][:, None].expand(-1, case["dim"]), src)}
    if case["op"] == "block_norm":
        gate = leaf.get("gate")
        if gate is not None and case["gate_act"] == "sigmoid":
            gate = torch.sigmoid(gate)
        b = _exact_norm(leaf["f"], leaf["w_post"], case["kind"])
        b = b if gate is None else b * gate
        b = b if s["res_scale"] is None else b * leaf["res_scale"]
        if case["dir"] == "fwd":
            y = leaf["x"] + b
            return {"y": y, "h": None if s["w_pre"] is None else _exact_norm(y, leaf["w_pre"], case["kind"])}
        # the backward's x is the stored sum: its gradient is the branch's too
        y = leaf["x"]
        dy = s["grad_y"].double()
        dpre = None
        if s["w_pre"] is not None:
            h = _exact_norm(y, leaf["w_pre"], case["kind"])
            gy, dpre = torch.autograd.grad(h, (y, leaf["w_pre"]), s["grad_h"].double())
            dy = dy + gy
        keys = [k for k in ("f", "gate", "w_post", "res_scale") if k in leaf]
        g = dict(zip(keys, torch.autograd.grad(b, [leaf[k] for k in keys], dy)))
        return {"grad_x": dy, "grad_f": g["f"], "grad_gate": g.get("gate"), "grad_w_post": g["w_post"],
                "grad_res_scale": g.get("res_scale"), "grad_w_pre": dpre}
    import torch.nn.functional as F
    act = {"silu": F.silu, "gelu": F.gelu, "relu": F.relu, "sigmoid": torch.sigmoid}[case["act"]]
    x, wg, wu, wd = (leaf[k] for k in ("x", "w_gate", "w_up", "w_down"))
    out = torch.mm(act(torch.mm(x, wg.t())) * torch.mm(x, wu.t()), wd.t())
    if case["dir"] == "fwd":
        return {"out": out}
    g = torch.autograd.grad(out, (x, wg, wu, wd), s["grad_out"].double())
    return dict(zip(("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down"), g))


# ------------------------------------------------------------ the work of one pass

def work(case):
    e = _BYTES[case["dtype"]]
    n = case["n"]
    if case["op"] == "embedding":
        d, rows, idx = case["dim"], case["rows"], 4 if case["idx"] == "i32" else 8
        if case["dir"] == "fwd":
            return {"bytes": n * idx + (n + min(n, rows)) * d * e, "flops": n * d}
        return {"bytes": n * idx + (n + rows) * d * e, "flops": n * d}
    if case["op"] == "block_norm":
        d = case["dim"]
        gate = {"none": 0, "row": 1, "element": d}[case["gate"]]
        nxt = 1 if case["next_norm"] else 0
        params = 4 * d * (1 + nxt + (1 if case["res_scale"] else 0))
        if case["dir"] == "fwd":
            return {"bytes": n * e * (3 * d + gate + nxt * d) + params, "flops": n * d * (8 + 6 * nxt)}
        # y is read only for the following norm; gate and its gradient
        return {"bytes": n * e * (4 * d + 2 * gate + nxt * 2 * d) + 2 * params, "flops": n * d * (18 + 12 * nxt)}
    di, f, do = case["d_in"], case["hidden"], case["d_out"]
    weights = (2 * di + do) * f
    if case["dir"] == "fwd":
        return {"bytes": e * (weights + n * (di + do)), "flops": 2 * n * weights}
    # three products again (gate, up, and the hidden gradient), then grad_x and the three weight gradients
    return {"bytes": e * (2 * weights + n * (2 * di + do)), "flops": 2 * n * (weights + 2 * di * f + weights)}
