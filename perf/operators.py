"""The normalisation, activation and 8-bit checkpoint operators around the block-scaled linear layers: what a pass
of each is, in elementary torch operations and through the library.

  norm_fwd   layer norm or RMS norm of a residual stream's rows (with the residual addition, the 8-bit checkpoint of
             the normalised input and the output's absolute maximum, where the case asks for them)
  norm_bwd   its gradients: dx, and the reductions over all rows for the weight and the bias, from the kept input or
             from its checkpoint
  act_fwd    h = act(gate) * up (or act(gate)), with the checkpoints of gate and up and the maximum of |h|
  act_bwd    its gradients, from the kept inputs or from their checkpoints
  act8       a checkpoint on its own: saved, then restored

A checkpoint holds E4M3 codes and, for each 32 columns of a row (the last group may be shorter), one byte e + 127: e is
the smallest integer with max|x| 2^-e <= 448 over the group, no less than -127, and 0 for a group of zeros.  A value
stands for code * 2^e.  Passes return it as its two factors, the codes as float8 values and the exponent bytes as
whole numbers, so that no restoring pass is timed with the operator that wrote it.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
def _norm_fwd(name, rows, cols, kind="layer", stream="bf16", out="bf16", residual=False, save=False, amax=False,
              stats=True):
    return {"name": name, "op": "norm_fwd", "rows": rows, "cols": cols, "kind": kind, "stream": stream, "out": out,
            "residual": residual, "save": save, "amax": amax, "stats": stats}


def _norm_bwd(name, rows, cols, kind="layer", stream="bf16", out="bf16", from8=False, dres=False):
    return {"name": name, "op": "norm_bwd", "rows": rows, "cols": cols, "kind": kind, "stream": stream, "out": out,
            "from8": from8, "dres": dres}


def _act_fwd(name, rows, cols, act="silu", gated=True, dtype="bf16", save=False, amax=False):
    return {"name": name, "op": "act_fwd", "rows": rows, "cols": cols, "act": act, "gated": gated, "dtype": dtype,
            "save": save, "amax": amax}


def _act_bwd(name, rows, cols, act="silu", gated=True, dtype="bf16", from8=False, amax=False):
    return {"name": name, "op": "act_bwd", "rows": rows, "cols": cols, "act": act, "gated": gated, "dtype": dtype,
            "from8": from8, "amax": amax}


def _act8(name, rows, cols, dtype="bf16"):
    return {"name": name, "op": "act8", "rows": rows, "cols": cols, "dtype": dtype}


def listed():
    return [
        # one new token in serving: the norm before a projection, latency only
        _norm_fwd("norm_fwd_token", 1, 4096, kind="rms", residual=True, stats=False),
        # the norm before a layer's first linear in training: 8192 tokens, hidden size 4096, everything asked for
        _norm_fwd("norm_fwd_train", 8192, 4096, residual=True, save=True, amax=True),
        # rows that start at odd addresses: a stream kept in 32 bits, a hidden size that no vector width divides
        _norm_fwd("norm_fwd_odd", 1021, 4099, stream="f32"),
        # a small batch's gradients, 32 bits throughout
        _norm_bwd("norm_bwd_small", 32, 1024, stream="f32", out="f32"),
        # the training norm's backward pass from the 8-bit checkpoint, joined with the residual path's gradient
        _norm_bwd("norm_bwd_train", 8192, 4096, from8=True, dres=True),
        # a ragged batch with an odd hidden size, from the kept input
        _norm_bwd("norm_bwd_odd", 4097, 1531, kind="rms"),
        # one new token through the gated MLP's activation
        _act_fwd("act_fwd_token", 1, 14336),
        # the training MLP's activation: 8192 tokens, both halves checkpointed, the maximum for the next quantization
        _act_fwd("act_fwd_train", 8192, 14336, save=True, amax=True),
        # its backward pass from the checkpoints; the largest case
        _act_bwd("act_bwd_train", 8192, 14336, from8=True, amax=True),
        # an ungated GELU in 32 bits with an odd width, from the kept input
        _act_bwd("act_bwd_odd", 1023, 11009, act="gelu", gated=False, dtype="f32"),
        # a small activation saved and restored
        _act8("act8_small", 16, 4096),
        # a training batch's MLP input saved and restored
        _act8("act8_train", 4096, 11008),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "act_fwd", "act_bwd", "act8"])
    rows = _log(rng, 1, 16384)
    cols = _log(rng, 32, 16384)
    if rng.random() < 0.5:  # half of the widths are what a model would have, the other half anything
        cols = max(32, cols // 64 * 64 if cols >= 64 else cols)
    while rows * cols > (1 << 26):
        rows = max(1, rows // 2 - rng.randrange(2))
    t, u, flag = rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]), lambda: rng.random() < 0.5
    kind, act = rng.choice(["layer", "rms"]), rng.choice(["silu", "gelu", "gelu_tanh"])
    if op == "norm_fwd":
        c = _norm_fwd("", rows, cols, kind, t, u, flag(), flag(), flag(), flag())
    elif op == "norm_bwd":
        c = _norm_bwd("", rows, cols, kind, t, u, flag(), flag())
    elif op == "act_fwd":
        c = _act_fwd("", rows, cols, act, flag(), t, flag(), flag())
    elif op == "act_bwd":
        c = _act_bwd("", rows, cols, act, flag(), t, flag(), flag())
    else:
        c = _act8("", rows, cols, t)
    del c["name"]
    return c


def work(case):
    n, rows, cols = case["rows"] * case["cols"], case["rows"], case["cols"]
    groups = rows * -(-cols // 32)
    saved = n + groups  # bytes of one checkpoint
    op = case["op"]
    if op == "norm_fwd":
        s = SIZE[case["stream"]]
        b = n * (s + SIZE[case["out"]]) + (2 * n * s if case["residual"] else 0) + (saved if case["save"] else 0)
        b += 4 * cols * (2 if case["kind"] == "layer" else 1) + (8 * rows if case["stats"] else 0)
        return {"bytes": b, "flops": 8 * n}
    if op == "norm_bwd":
        s = SIZE[case["stream"]]
        b = n * (SIZE[case["out"]] + s) + (saved if case["from8"] else n * s) + (n * s if case["dres"] else 0)
        return {"bytes": b + 12 * cols + 8 * rows, "flops": 16 * n}
    if op == "act8":
        return {"bytes": 2 * (n * SIZE[case["dtype"]] + saved), "flops": 4 * n}
    halves, s = (2 if case["gated"] else 1), SIZE[case["dtype"]]
    if op == "act_fwd":
        return {"bytes": n * s * (halves + 1) + (halves * saved if case["save"] else 0), "flops": 8 * n}
    return {"bytes": n * s * (halves + 1) + halves * (saved if case["from8"] else n * s), "flops": 16 * n}


# ------------------------------------------------------------------ inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _stream(g, rows, cols, dtype):
    """Activations: a level and a spread of each column's own, a few columns far larger than the rest."""
    spread = torch.exp(0.5 * _normal(g, 1, cols))
    spread[:, :: max(1, cols // 4)] *= 20.0
    return (_normal(g, rows, cols) * spread + 0.2 * _normal(g, 1, cols)).to(dtype)


def _gradient(g, rows, cols, dtype):
    """Gradients: Student-t with three degrees of freedom, a thousandth."""
    chi2 = _normal(g, rows, cols).square_()
    for _ in range(2):
        chi2 += _normal(g, rows, cols).square_()
    return (_normal(g, rows, cols) / chi2.div_(3.0).sqrt_() * 1e-3).to(dtype)


def _encode(x):
    """(codes uint8 [rows, 32 G], exponent bytes uint8 [rows, G]) of x's checkpoint."""
    rows, cols = x.shape
    groups = -(-cols // 32)
    xf = x.float()
    if groups * 32 != cols:
        xf = torch.nn.functional.pad(xf, (0, groups * 32 - cols))
    xg = xf.view(rows, groups, 32)
    m, e = torch.frexp(xg.abs().amax(-1))  # the largest is m 2^e with 0.5 <= m < 1, and 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, torch.zeros_like(e), e).clamp(min=-127)
    down = ((127 - e) << 23).to(torch.int32).view(torch.float32)  # 2^-e
    codes = (xg * down[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(rows, groups * 32), (e + 127).to(torch.uint8)


def _decode(codes, sf, cols):
    """fp32 values that a checkpoint stands for."""
    rows, groups = sf.shape
    e = sf.to(torch.int32)
    up = torch.where(e > 0, e << 23, torch.full_like(e, 1 << 22)).view(torch.float32)  # 2^(byte - 127)
    v = codes.view(torch.float8_e4m3fn).float().view(rows, groups, 32) * up[..., None]
    return v.view(rows, groups * 32)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    rows, cols, op = case["rows"], case["cols"], case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        t, o = TYPES[case["stream"]], TYPES[case["out"]]
        s["w"] = 1.0 + 0.1 * _normal(g, cols)
        s["b"] = 0.1 * _normal(g, cols) if case["kind"] == "layer" else None
        x = _stream(g, rows, cols, t)
        if op == "norm_fwd":
            s["x"] = x
            s["r"] = _stream(g, rows, cols, t) if case["residual"] else None
            return s
        s["dy"] = _gradient(g, rows, cols, o)
        s["dres"] = _gradient(g, rows, cols, t) if case["dres"] else None
        xf = x.float()
        s["mean"] = xf.mean(1) if case["kind"] == "layer" else None
        d = xf - s["mean"][:, None] if case["kind"] == "layer" else xf
        s["rstd"] = torch.rsqrt(d.square().mean(1) + EPS)
        if case["from8"]:
            s["codes"], s["sf"] = _encode(x)
        else:
            s["x"] = x
        return s
    t, halves = TYPES[case["dtype"]], (2 if case.get("gated") else 1)
    if op == "act8":
        s["x"] = _stream(g, rows, cols, t)
        return s
    x = _normal(g, rows, halves * cols) * torch.exp(0.3 * _normal(g, 1, halves * cols))
    x = x.to(t)  # a gate_up projection's output: the gate in the first half of a row, up in the second
    if op == "act_bwd":
        s["dh"] = _gradient(g, rows, cols, t)
    if op == "act_bwd" and case["from8"]:
        s["gate8"] = _encode(x[:, :cols])
        s["up8"] = _encode(x[:, cols:]) if case["gated"] else None
    else:
        s["x"] = x
    return s


# ------------------------------------------------------------------ the passes
def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _codes(codes, cols):
    return codes[:, :cols].view(torch.float8_e4m3fn)


def _plain_norm_fwd(s):
    x, out = s["x"].float(), {}
    if s["residual"]:
        out["sum"] = (x + s["r"].float()).to(s["x"].dtype)
        x = out["sum"].float()
    n = s["cols"]
    if s["kind"] == "layer":
        mean = x.sum(1) / n
        d = x - mean[:, None]
    else:
        mean, d = None, x
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / n + EPS)
    y = d * rstd[:, None] * s["w"]
    if s["kind"] == "layer":
        y = y + s["b"]
    y = out["y"] = y.to(TYPES[s["out"]])
    if s["stats"]:
        out["rstd"] = rstd
        if mean is not None:
            out["mean"] = mean
    if s["save"]:
        codes, out["sf"] = _encode(out["sum"] if s["residual"] else s["x"])
        out["codes"] = _codes(codes, n)
    if s["amax"]:
        out["amax"] = y.float().abs().max().reshape(1)
    return out


def _plain_norm_bwd(s):
    n, t = s["cols"], TYPES[s["stream"]]
    x = _decode(s["codes"], s["sf"], n) if s["from8"] else s["x"].float()
    rstd, dy = s["rstd"][:, None], s["dy"].float()
    xh = (x - s["mean"][:, None]) * rstd if s["kind"] == "layer" else x * rstd
    g = dy * s["w"]
    dx = g - xh * ((g * xh).sum(1, keepdim=True) / n)
    if s["kind"] == "layer":
        dx = dx - g.sum(1, keepdim=True) / n
    dx = dx * rstd
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    out = {"dx": dx.to(t), "dw": (dy * xh).sum(0)}
    if s["kind"] == "layer":
        out["db"] = dy.sum(0)
    return out


_C0, _C1 = math.sqrt(2.0 / math.pi), 0.044715


def _act_and_slope(z, act):
    """act(z) and its derivative."""
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * p, p + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    th = torch.tanh(_C0 * (z + _C1 * z * z * z))
    return 0.5 * z * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * _C0 * (1.0 + 3.0 * _C1 * z * z)


def _plain_act_fwd(s):
    n, t = s["cols"], TYPES[s["dtype"]]
    gate = s["x"][:, :n]
    h = _act_and_slope(gate.float(), s["act"])[0]
    if s["gated"]:
        h = h * s["x"][:, n:].float()
    h = h.to(t)
    out = {"h": h}
    if s["save"]:
        codes, out["gate_sf"] = _encode(gate)
        out["gate"] = _codes(codes, n)
        if s["gated"]:
            codes, out["up_sf"] = _encode(s["x"][:, n:])
            out["up"] = _codes(codes, n)
    if s["amax"]:
        out["amax"] = h.float().abs().max().reshape(1)
    return out


def _plain_act_bwd(s):
    n, t = s["cols"], TYPES[s["dtype"]]
    gate = _decode(*s["gate8"], n) if s["from8"] else s["x"][:, :n].float()
    dh = s["dh"].float()
    a, slope = _act_and_slope(gate, s["act"])
    if s["gated"]:
        up = _decode(*s["up8"], n) if s["from8"] else s["x"][:, n:].float()
        out = {"dgate": (dh * up * slope).to(t), "dup": (dh * a).to(t)}
    else:
        out = {"dgate": (dh * slope).to(t)}
    if s["amax"]:
        top = out["dgate"].float().abs().max()
        out["amax"] = (torch.maximum(top, out["dup"].float().abs().max()) if s["gated"] else top).reshape(1)
    return out


def _plain_act8(s):
    codes, sf = _encode(s["x"])
    return {"codes": _codes(codes, s["cols"]), "sf": sf, "restored": _decode(codes, sf, s["cols"]).to(s["x"].dtype)}


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "act_fwd": _plain_act_fwd,
          "act_bwd": _plain_act_bwd, "act8": _plain_act8}


def _own_norm_fwd(s):
    import fp4_precision_gemms_gb300 as mx

    x = s["x"]
    amax = torch.empty(1, dtype=torch.float32, device=x.device) if s["amax"] else None
    r = mx.norm_fwd(x, s["w"], s["b"], kind=s["kind"], eps=EPS, residual=s["r"], save=s["save"], amax_out=amax,
                    out_dtype=TYPES[s["out"]], need_stats=s["stats"])
    out = {"y": r.y}
    if s["residual"]:
        out["sum"] = r.sum
    if s["stats"]:
        out["rstd"] = r.rstd
        if s["kind"] == "layer":
            out["mean"] = r.mean
    if s["save"]:
        out["codes"], out["sf"] = _codes(r.saved.codes, s["cols"]), r.saved.sf
    if s["amax"]:
        out["amax"] = amax
    return out


def _own_norm_bwd(s):
    import fp4_precision_gemms_gb300 as mx

    x = mx.Act8(s["codes"], s["sf"], s["cols"]) if s["from8"] else s["x"]
    dx, dw, db = mx.norm_bwd(s["dy"], x, s["rstd"], s["mean"], s["w"], kind=s["kind"], dres=s["dres"],
                             dx_dtype=TYPES[s["stream"]])
    out = {"dx": dx, "dw": dw}
    if s["kind"] == "layer":
        out["db"] = db
    return out


def _own_act_fwd(s):
    import fp4_precision_gemms_gb300 as mx

    x, n = s["x"], s["cols"]
    gate, up = (x[:, :n], x[:, n:]) if s["gated"] else (x, None)
    amax = torch.empty(1, dtype=torch.float32, device=x.device) if s["amax"] else None
    r = mx.act_fwd(gate, up, act=s["act"], save=s["save"], amax_out=amax)
    out = {"h": r.h}
    if s["save"]:
        out["gate"], out["gate_sf"] = _codes(r.gate.codes, n), r.gate.sf
        if s["gated"]:
            out["up"], out["up_sf"] = _codes(r.up.codes, n), r.up.sf
    if s["amax"]:
        out["amax"] = amax
    return out


def _own_act_bwd(s):
    import fp4_precision_gemms_gb300 as mx

    dh, n = s["dh"], s["cols"]
    if s["from8"]:
        gate = mx.Act8(*s["gate8"], n)
        up = mx.Act8(*s["up8"], n) if s["gated"] else None
    else:
        gate, up = (s["x"][:, :n], s["x"][:, n:]) if s["gated"] else (s["x"], None)
    amax = torch.empty(1, dtype=torch.float32, device=dh.device) if s["amax"] else None
    dgate, dup = mx.act_bwd(dh, gate, up, act=s["act"], amax_out=amax)
    out = {"dgate": dgate}
    if s["gated"]:
        out["dup"] = dup
    if s["amax"]:
        out["amax"] = amax
    return out


def _own_act8(s):
    import fp4_precision_gemms_gb300 as mx

    a = mx.act8_save(s["x"])
    return {"codes": _codes(a.codes, s["cols"]), "sf": a.sf, "restored": mx.act8_restore(a, out_dtype=s["x"].dtype)}


_OWN = {"norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd, "act_fwd": _own_act_fwd, "act_bwd": _own_act_bwd,
        "act8": _own_act8}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_code(x):
    """(value of each code, value that the checkpoint stands for) of float64 x: the E4M3 grid written out."""
    rows, cols = x.shape
    groups = (cols + 31) // 32
    b = torch.zeros(rows, groups * 32, dtype=torch.float64, device=x.device)
    b[:, :cols] = x.abs()
    b = b.reshape(rows, groups, 32).max(dim=2).values
    e = torch.ceil(torch.log2(torch.clamp(b, min=2.0 ** -200)) - math.log2(448.0))
    for _ in range(2):  # the logarithm may be off by its last bit next to a power of two
        e = torch.where(b * torch.exp2(-e) > 448.0, e + 1, e)
        e = torch.where(b * torch.exp2(1 - e) <= 448.0, e - 1, e)
    e = torch.where(b == 0, torch.zeros_like(e), e).clamp(min=-127.0)
    scale = torch.exp2(e).repeat_interleave(32, dim=1)[:, :cols]
    v = x / scale
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)  # three bits after the first, from 2^-6 up
    code = torch.round(v / step) * step  # ties to even
    return code, code * scale


def _exact_act(z, act):
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    inner = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    p = torch.sigmoid(2 * inner)  # (1 + tanh(inner)) / 2
    return z * p, p + z * 2 * p * (1 - p) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    n, op = case["cols"], case["op"]
    if op == "norm_fwd":
        t, out, x = TYPES[case["stream"]], {}, s["x"].double()
        if case["residual"]:
            out["sum"] = x + s["r"].double()
            x = out["sum"].to(t).double()  # the norm and the checkpoint read the stream as it is stored
        mean = x.mean(dim=1, keepdim=True) if case["kind"] == "layer" else torch.zeros_like(x[:, :1])
        rstd = ((x - mean).pow(2).mean(dim=1, keepdim=True) + EPS).rsqrt()
        y = out["y"] = (x - mean) * rstd * s["w"].double() + (s["b"].double() if case["kind"] == "layer" else 0.0)
        if case["stats"]:
            out["rstd"] = rstd[:, 0]
            if case["kind"] == "layer":
                out["mean"] = mean[:, 0]
        if case["save"]:
            out["codes"], out["sf"] = _exact_code(x)[0], None
        if case["amax"]:
            out["amax"] = y.to(TYPES[case["out"]]).double().abs().max().reshape(1)
        return out
    if op == "norm_bwd":
        x = _value64(s["codes"], s["sf"], n) if case["from8"] else s["x"].double()
        dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
        xh = (x - (s["mean"].double()[:, None] if case["kind"] == "layer" else 0.0)) * rstd
        g = dy * s["w"].double()
        back = g - xh * (g * xh).mean(dim=1, keepdim=True)
        if case["kind"] == "layer":
            back = back - g.mean(dim=1, keepdim=True)
        out = {"dx": back * rstd + (s["dres"].double() if case["dres"] else 0.0), "dw": (dy * xh).sum(dim=0)}
        if case["kind"] == "layer":
            out["db"] = dy.sum(dim=0)
        return out
    if op == "act8":
        code, value = _exact_code(s["x"].double())
        return {"codes": code, "sf": None, "restored": value}
    t, out = TYPES[case["dtype"]], {}
    if op == "act_fwd":
        gate = s["x"][:, :n].double()
        h = _exact_act(gate, case["act"])[0]
        if case["gated"]:
            up = s["x"][:, n:].double()
            h = h * up
        out["h"] = h
        if case["save"]:
            out["gate"], out["gate_sf"] = _exact_code(gate)[0], None
            if case["gated"]:
                out["up"], out["up_sf"] = _exact_code(up)[0], None
        if case["amax"]:
            out["amax"] = h.to(t).double().abs().max().reshape(1)
        return out
    gate = _value64(*s["gate8"], n) if case["from8"] else s["x"][:, :n].double()
    value, slope = _exact_act(gate, case["act"])
    dh = s["dh"].double()
    if case["gated"]:
        up = _value64(*s["up8"], n) if case["from8"] else s["x"][:, n:].double()
        out["dup"] = dh * value
        out["dgate"] = dh * slope * up
    else:
        out["dgate"] = dh * slope
    if case["amax"]:
        out["amax"] = torch.stack([v.to(t).double().abs().max() for v in out.values()]).max().reshape(1)
    return out


def _value64(codes, sf, cols):
    """What a checkpoint stands for: sign, exponent and fraction of each code taken apart."""
    c = codes[:, :cols].to(torch.int64)
    exponent, fraction = (c >> 3) & 15, (c & 7).double()
    size = torch.where(exponent > 0, (1 + fraction / 8) * torch.exp2((exponent - 7).double()), fraction * 2.0 ** -9)
    scale = torch.exp2(sf.double() - 127).repeat_interleave(32, dim=1)[:, :cols]
    return torch.where(c >= 128, -size, size) * scale
