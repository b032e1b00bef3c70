"""The gated feed-forward block, the AdamW step and the gradient norm: what a pass of each is, in elementary torch
operations and through the library.

  gated      h = act(X Wg^T) * (X Wu^T) with X and W = [Wg; Wu] in a block-scaled format.  Serving: the weights are
             quantized beforehand, X within the pass.  Training: both within the pass, which then goes back from dh,
             with the projections' outputs kept as 8-bit checkpoints and the gradients quantized like the inputs
  adamw      one step over many tensors, the moments in 32 bits, or in 8: E4M3 codes of m and of sqrt(v) with one byte
             e + 127 for each 32 values, as the 8-bit checkpoints have them (e the smallest integer with
             max 2^-e <= 448, 0 for zeros); a root that is not zero keeps the smallest code above zero
  grad_norm  the norm over all tensors' gradients, and the factor that brings it down to a given one

Formats (blocks run along the product's inner dimension):
  mxfp8   E4M3, 2^e per 32 values, e = floor(log2 max) - 8
  mxfp4   E2M1, 2^e per 32, e = floor(log2 max) - 2
  moss    E4M3, ts = fl32(max of all / 448), y = fl32(x / ts), 2^e per 32 of y, e the smallest with max 2^-e <= 448
  nvfp4   E2M1, ts = fl32(max of all / 2688), per 16: s = E4M3(fl32(max / fl32(6 ts))), code of fl32(x / fl32(s ts))

Stochastic rounding of value L of tensor i takes the 16-bit half (L & 1) of word (L & 7) >> 1 of Philox4x32-10 with key
`seed` and counter (L >> 3, L >> 35, t, 4 i + k), k = 0, 1, 2 for m, sqrt(v) and a bf16 parameter, and goes up where
that number is below 2^16 times the value's place between its two neighbours.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
BETAS, EPS, LR, DECAY = (0.9, 0.999), 1e-8, 3e-4, 0.1
WEIGHT_BYTES = {"mxfp8": 1 + 1 / 32, "moss": 1 + 1 / 32, "mxfp4": 0.5 + 1 / 32, "nvfp4": 0.5 + 1 / 16}


# ------------------------------------------------------------------ cases
def _gated(name, tokens, hidden, ffn, fmt, act="silu", train=False):
    return {"name": name, "op": "gated", "tokens": tokens, "hidden": hidden, "ffn": ffn, "fmt": fmt, "act": act,
            "train": train}


def _adamw(name, shape, a, b, bits=32, param="f32", grad="f32", copy=False, amax=False, rounding="rne", scale=False,
           t=100):
    return {"name": name, "op": "adamw", "shape": shape, "a": a, "b": b, "bits": bits, "param": param, "grad": grad,
            "copy": copy, "amax": amax, "rounding": rounding, "scale": scale, "t": t}


def _grad_norm(name, shape, a, b, grad="f32"):
    return {"name": name, "op": "grad_norm", "shape": shape, "a": a, "b": b, "grad": grad}


def listed():
    return [
        # one new token in serving: the weights' bytes and latency
        _gated("gated_token", 1, 4096, 14336, "mxfp8"),
        # a batch of decoding sequences, four-bit weights
        _gated("gated_decode", 48, 4096, 14336, "nvfp4"),
        # a prompt of odd length, four-bit weights
        _gated("gated_prompt", 4001, 4096, 14336, "nvfp4"),
        # the training MLP's first half, forward and backward, at 8192 tokens; the largest of its kind
        _gated("gated_train", 8192, 4096, 14336, "mxfp8", train=True),
        # a small model's, with an inner width that no tile divides
        _gated("gated_train_odd", 1152, 1280, 3392, "mxfp8", act="gelu_tanh", train=True),
        # the norms' weights of a model: many small tensors, latency
        _adamw("adamw_norms", "vectors", 65, 4096),
        # the four linears and two norms of a layer: fp32 weights, their bf16 copies, the next quantization's maxima
        _adamw("adamw_layer", "layer", 4096, 14336, copy=True, amax=True, scale=True),
        # the same with moments in 8 bits and bf16 gradients
        _adamw("adamw8_layer", "layer", 4096, 14336, bits=8, grad="bf16", copy=True, amax=True, scale=True),
        # tensors of odd sizes, bf16 weights without a 32-bit copy, moments and weights rounded stochastically
        _adamw("adamw8_odd", "ragged", 37, 400000, bits=8, param="bf16", grad="bf16", rounding="sr", t=3),
        # gradients of a model's norms: latency
        _grad_norm("norm_small", "vectors", 12, 4096, "bf16"),
        # gradients of a layer
        _grad_norm("norm_layer", "layer", 4096, 14336),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    flag = lambda: rng.random() < 0.5  # noqa: E731
    op = rng.choice(["gated", "gated", "adamw", "adamw", "grad_norm"])
    if op == "gated":
        train = flag()
        # a tensor scale rests on one value: where that is itself computed (training), its last bit moves every code
        fmt = rng.choice(["mxfp8", "mxfp4"] if train else ["mxfp8", "mxfp4", "nvfp4", "moss"])
        hidden = 256 * max(1, _log(rng, 256, 8192) // 256)
        # training multiplies along the tokens and along both halves too: whole steps of the product's inner dimension
        of, least = ((256, 128) if fmt == "mxfp4" else (128, 64)) if train else (1, 32)
        tokens = of * max(1, _log(rng, of, 8192) // of)
        ffn = least * max(1, _log(rng, 64, 14336) // least)
        if flag() and ffn >= 128:
            ffn = ffn // 128 * 128
        act = rng.choice(["silu", "silu", "gelu", "gelu_tanh"])
        while tokens * hidden * ffn > 8192 * 4096 * 14336:
            tokens = of * max(1, tokens // 2 // of)
        c = _gated("", tokens, hidden, ffn, fmt, act, train)
    else:
        shape = rng.choice(["vectors", "layer", "ragged"])
        if shape == "layer":
            a = 16 * max(1, _log(rng, 64, 4096) // 16)
            b = 16 * max(1, int(a * rng.uniform(2.0, 3.5)) // 16)
        else:
            a, b = _log(rng, 1, 100), _log(rng, 1, 400000)
        if op == "grad_norm":
            c = _grad_norm("", shape, a, b, rng.choice(["bf16", "f32"]))
        else:
            bits, param = rng.choice([32, 8]), rng.choice(["f32", "f32", "bf16"])
            rounding = rng.choice(["rne", "sr"]) if bits == 8 or param == "bf16" else "rne"
            c = _adamw("", shape, a, b, bits, param, rng.choice(["bf16", "f32"]), param == "f32" and flag(), flag(),
                       rounding, flag(), _log(rng, 1, 100000))
    del c["name"]
    return c


def _shapes(case):
    """The tensors' shapes: a layer's linears and norms (a hidden, b inner width), a vectors of b values, or a tensors
    of up to b values, odd sizes among them."""
    a, b = case["a"], case["b"]
    if case["shape"] == "layer":
        return [(a + a // 2, a), (a, a), (2 * b, a), (a, b), (a,), (a,)]
    if case["shape"] == "vectors":
        return [(b,)] * a
    return [(1 + (b * ((37 * i * i + 11 * i + 5) % 101)) // 101,) for i in range(a)]


def work(case):
    if case["op"] == "gated":
        t, k, f = case["tokens"], case["hidden"], case["ffn"]
        if case["train"]:
            return {"bytes": 4 * t * k + 8 * f * k + 4 * t * f, "flops": 12 * t * k * f}  # x, dx; w, dw; h, dh
        return {"bytes": int(2 * t * k + 2 * f * k * WEIGHT_BYTES[case["fmt"]] + 2 * t * f), "flops": 4 * t * k * f}
    n = sum(math.prod(s) for s in _shapes(case))
    if case["op"] == "grad_norm":
        return {"bytes": n * SIZE[case["grad"]], "flops": 2 * n}
    each = 2 * SIZE[case["param"]] + SIZE[case["grad"]] + (16 if case["bits"] == 32 else 4 + 4 / 32) + 2 * case["copy"]
    return {"bytes": int(n * each), "flops": 16 * n}


# ------------------------------------------------------------------ block-scaled values
def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _e4m3(y):
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()


def _e2m1(y):
    a = y.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), y)


def _ceil_exponent(b):
    """The smallest e with b 2^-e <= 448 = 0.875 2^9, 0 for b = 0."""
    m, e = torch.frexp(b)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(b == 0, torch.zeros_like(e), e).clamp(-127, 127)


def _quantized(x, fmt):
    """(codes times block scales in fp32, exactly, and the tensor scale) of a matrix quantized along its rows."""
    rows, k = x.shape
    xf = x.float()
    top = xf.abs().max()
    if fmt == "nvfp4":
        ts = torch.where(top > 0, top / torch.full_like(top, 2688.0), torch.ones_like(top))  # a quotient
        xb = xf.view(rows, k // 16, 16)
        s = _e4m3(xb.abs().amax(-1) / (ts * 6.0))
        d = s * ts
        q = torch.where(d[..., None] > 0, _e2m1(xb / torch.where(d > 0, d, 1.0)[..., None]), 0.0) * s[..., None]
        return q.view(rows, k), ts
    ts = torch.ones_like(top)
    if fmt == "moss":
        ts = torch.where(top > 0, top / torch.full_like(top, 448.0), ts)
        xf = xf / ts
    xb = xf.view(rows, k // 32, 32)
    b = xb.abs().amax(-1)
    if fmt == "moss":
        e = _ceil_exponent(b)
    else:
        e = torch.frexp(b)[1] - 1 - (8 if fmt == "mxfp8" else 2)
        e = torch.where(b == 0, torch.zeros_like(e), e).clamp(-127, 127)
    y = xb * _pow2(-e)[..., None]
    q = (_e2m1(y) if fmt == "mxfp4" else _e4m3(y)) * _pow2(e)[..., None]
    return q.view(rows, k), ts


def _act8(x):
    """The values that the 8-bit checkpoint of x (columns a multiple of 32) stands for."""
    xb = x.view(x.shape[0], -1, 32)
    e = _ceil_exponent(xb.abs().amax(-1))[..., None]
    return (_e4m3(xb * _pow2(-e)) * _pow2(e)).view(x.shape)


def _times(a, b):
    """a b^T of two quantized operands."""
    return (a[0] @ b[0].t()) * (a[1] * b[1])


# ------------------------------------------------------------------ inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _gradient(g, *shape):
    """Gradients: Student-t with three degrees of freedom, a thousandth."""
    chi2 = _normal(g, *shape).square_()
    for _ in range(2):
        chi2 += _normal(g, *shape).square_()
    return _normal(g, *shape).div_(chi2.div_(3.0).sqrt_()).mul_(1e-3)


def _encode(x, root):
    """(codes uint8 [1, 32 G], bytes uint8 [1, G]) of a flat moment."""
    n = x.numel()
    groups = -(-n // 32)
    xb = torch.nn.functional.pad(x, (0, groups * 32 - n)).view(groups, 32)
    e = _ceil_exponent(xb.abs().amax(-1))
    v = _e4m3(xb * _pow2(-e)[:, None])
    if root:
        v = torch.where((v == 0) & (xb > 0), 2.0 ** -9, v)
    return v.to(torch.float8_e4m3fn).view(torch.uint8).view(1, -1), (e + 127).to(torch.uint8).view(1, -1)


def _put(state, at, pair):
    """Writes a tensor's codes and bytes to their place."""
    codes, sf = pair
    state[0][0, at:at + codes.numel()] = codes[0]
    state[1][0, at // 32:at // 32 + sf.numel()] = sf[0]


def _decode(state, at, n):
    groups = -(-n // 32)
    codes, sf = state[0][0, at:at + 32 * groups], state[1][0, at // 32:at // 32 + groups]
    v = codes.view(torch.float8_e4m3fn).float().view(-1, 32) * _pow2(sf.view(-1, 1).int() - 127)
    return v.view(-1)[:n]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    s["seed"] = int(seed)
    if case["op"] == "gated":
        t, k, f = case["tokens"], case["hidden"], case["ffn"]
        x = _normal(g, t, k)  # a norm's output, some columns larger than the rest
        x *= torch.exp(0.3 * _normal(g, 1, k))
        x[:, :: max(1, k // 4)] *= 8.0
        s["x"] = x.bfloat16()
        s["w"] = (_normal(g, 2 * f, k) / math.sqrt(k)).bfloat16()
        if case["train"]:
            s["dh"] = _gradient(g, t, f).bfloat16()
        elif own:
            import fp4_precision_gemms_gb300 as mx

            s["weights"] = mx.gated_weights(s["w"], case["fmt"])
        else:
            s["weights"] = _quantized(s["w"], case["fmt"])
        return s
    shapes = _shapes(case)
    s["grads"] = [_gradient(g, *shape).to(TYPES[case["grad"]]) for shape in shapes]
    if case["op"] == "grad_norm":
        total = sum(math.prod(shape) for shape in shapes)
        s["max_norm"] = 1e-3 * math.sqrt(total)  # some way below the norm, as in a step that is clipped
        return s
    dt, sizes = TYPES[case["param"]], [math.prod(shape) for shape in shapes]
    s["flat"] = torch.empty(sum(sizes), dtype=dt, device="cuda")  # the parameters one behind another, at any offset
    s["params"] = [p.view(shape) for p, shape in zip(s["flat"].split(sizes), shapes)]
    groups = [-(-n // 32) for n in sizes]  # the moments' places: each tensor starts a group of 32
    s["places"] = [(32 * sum(groups[:i]), n) for i, n in enumerate(sizes)]
    total = sum(groups)
    if case["bits"] == 8:
        s["m"], s["v"] = ((torch.zeros(1, 32 * total, dtype=torch.uint8, device="cuda"),
                           torch.zeros(1, total, dtype=torch.uint8, device="cuda")) for _ in range(2))
    else:
        s["m"], s["v"] = (torch.zeros(32 * total, device="cuda") for _ in range(2))
    for shape, grad, p, (at, n) in zip(shapes, s["grads"], s["params"], s["places"]):
        p.copy_(_normal(g, *shape) * 0.02 if len(shape) == 2 else 1.0 + 0.1 * _normal(g, *shape))
        flat = grad.float().reshape(-1)
        m = 0.3 * flat + 3e-4 * _normal(g, n)
        r = 0.5 * flat.abs() + 1e-3 * (0.1 + _normal(g, n).abs())  # the second moment's root
        if case["bits"] == 8:
            for state, x, root in ((s["m"], m, False), (s["v"], r, True)):
                _put(state, at, _encode(x, root))
        else:
            s["m"][at:at + n] = m
            s["v"][at:at + n] = r.square()
    s["decay"] = [DECAY if len(shape) == 2 else 0.0 for shape in shapes]
    s["copy_flat"] = torch.empty_like(s["flat"], dtype=torch.bfloat16)
    s["copies"] = [c.view(shape) for c, shape in zip(s["copy_flat"].split(sizes), shapes)] if case["copy"] else None
    s["factor"] = 0.25 + 0.5 * torch.rand(1, generator=g, device="cuda") if case["scale"] else None
    s["amax_out"] = torch.empty(len(shapes), device="cuda") if case["amax"] else None
    if own:
        import fp4_precision_gemms_gb300 as mx

        s["opt"] = opt = mx.AdamW(s["params"], lr=LR, betas=BETAS, eps=EPS, weight_decay=s["decay"],
                                  state="8bit" if case["bits"] == 8 else "fp32", copies=s["copies"],
                                  rounding=case["rounding"], seed=int(seed))
        for mine, given in ((opt.m_all, s["m"]), (opt.v_all, s["v"])):
            if case["bits"] == 8:
                mine.codes.copy_(given[0])
                mine.sf.copy_(given[1])
            else:
                mine.copy_(given)
    return s


# ------------------------------------------------------------------ the passes
def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


_C0, _C1 = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act):
    """(value, slope)"""
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    t = torch.tanh(_C0 * (z + _C1 * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C0 * (1.0 + 3.0 * _C1 * z * z)


def _plain_gated(s):
    fmt, f, act = s["fmt"], s["ffn"], s["act"]
    w = _quantized(s["w"], fmt) if s["train"] else s["weights"]
    gu = _times(_quantized(s["x"], fmt), w)
    gate, up = gu[:, :f], gu[:, f:]
    h = (_act(gate, act)[0] * up).bfloat16()
    if not s["train"]:
        return {"h": h}
    gate, up = _act8(gate.contiguous()), _act8(up.contiguous())
    dh = s["dh"].float()
    value, slope = _act(gate, act)
    d = torch.cat([(dh * up * slope).bfloat16(), (dh * value).bfloat16()], 1)
    dx = _times(_quantized(d, fmt), _quantized(s["w"].t().contiguous(), fmt)).bfloat16()
    dw = _times(_quantized(d.t().contiguous(), fmt), _quantized(s["x"].t().contiguous(), fmt)).bfloat16()
    return {"h": h, "dx": dx, "dw": dw}


def _mul_wide(a, b):
    """(high, low) 32-bit words of the product of 32-bit numbers, in int64."""
    low, high = (a & 0xFFFF) * b, (a >> 16) * b
    return (high + (low >> 16)) >> 16, (((high & 0xFFFF) << 16) + low) & 0xFFFFFFFF


def _random16(seed, n, t, word):
    """The 16-bit numbers of values 0 .. n - 1."""
    i = torch.arange(-(-n // 8), device="cuda", dtype=torch.int64)
    c = [i & 0xFFFFFFFF, i >> 32, torch.full_like(i, t & 0xFFFFFFFF), torch.full_like(i, word)]
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        h0, l0 = _mul_wide(c[0], 0xD2511F53)
        h1, l1 = _mul_wide(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack(c, 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).view(-1)[:n]


def _moment8(x, root, bits):
    """A moment's codes and bytes, rounded to nearest or by 16-bit numbers; returns views like _encode's."""
    if bits is None:
        return _encode(x, root)
    n = x.numel()
    groups = -(-n // 32)
    pad = groups * 32 - n
    xb = torch.nn.functional.pad(x, (0, pad)).view(groups, 32)
    u = torch.nn.functional.pad(bits, (0, pad)).view(groups, 32)
    e = _ceil_exponent(xb.abs().amax(-1))
    y = (xb * _pow2(-e)[:, None]).abs()
    step = _pow2((torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
    q = y / step
    low = torch.floor(q)
    v = ((low + (u < (q - low) * 65536.0)) * step).clamp(max=448.0)
    if root:
        v = torch.where((v == 0) & (xb > 0), 2.0 ** -9, v)
    v = torch.copysign(v, xb)
    return v.to(torch.float8_e4m3fn).view(torch.uint8).view(1, -1), (e + 127).to(torch.uint8).view(1, -1)


def _adamw_outputs(s, m, v, amax):
    """The parameters, and moments of 8 bits as their two factors: the codes' values and the exponents' bytes."""
    out = {"p": s["flat"]}
    if s["bits"] == 8:
        out["m"], out["m_sf"] = m[0].view(torch.float8_e4m3fn), m[1]
        out["root"], out["root_sf"] = v[0].view(torch.float8_e4m3fn), v[1]
    else:
        out["m"], out["v"] = m, v
    if s["copy"]:
        out["copy"] = s["copy_flat"]
    if s["amax"]:
        out["amax"] = amax
    return out


def _plain_adamw(s):
    b1, b2 = BETAS
    t, sr = s["t"], s["rounding"] == "sr"
    c1, c2 = 1.0 - b1 ** t, math.sqrt(1.0 - b2 ** t)
    top = []
    for i, (p, grad, (at, n)) in enumerate(zip(s["params"], s["grads"], s["places"])):
        g = grad.float().reshape(-1)
        if s["scale"]:
            g = g * s["factor"]
        if s["bits"] == 8:
            m, r = _decode(s["m"], at, n), _decode(s["v"], at, n)
            v = r * r
        else:
            m, v = s["m"][at:at + n], s["v"][at:at + n]
        m = m * b1 + g * (1.0 - b1)
        v = v * b2 + g * g * (1.0 - b2)
        r = torch.sqrt(v)
        new = p.float().view(-1) * (1.0 - LR * s["decay"][i]) - (LR / c1) * (m / (r / c2 + EPS))
        if s["bits"] == 8:
            for k, (state, x) in enumerate(((s["m"], m), (s["v"], r))):
                _put(state, at, _moment8(x, k == 1, _random16(s["seed"], n, t, 4 * i + k) if sr else None))
        else:
            s["m"][at:at + n] = m
            s["v"][at:at + n] = v
        if s["param"] == "bf16" and sr:
            bits = new.view(torch.int32)
            up = _random16(s["seed"], n, t, 4 * i + 2) < (bits & 0xFFFF)
            new = ((bits & -65536) + (up.int() << 16)).view(torch.float32)
        p.view(-1).copy_(new)
        if s["copy"]:
            s["copies"][i].copy_(p)
        if s["amax"]:
            top.append((s["copies"][i] if s["copy"] else p).abs().max().float())
    return _adamw_outputs(s, s["m"], s["v"], torch.stack(top) if top else None)


def _plain_grad_norm(s):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for g in s["grads"]:
        total = total + (g.double() * g.double()).sum()
    norm = torch.sqrt(total)
    return torch.stack([norm, torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)]).float()


_PLAIN = {"gated": _plain_gated, "adamw": _plain_adamw, "grad_norm": _plain_grad_norm}


def _own_gated(s):
    import fp4_precision_gemms_gb300 as mx

    if not s["train"]:
        return {"h": mx.gated_fwd(s["x"], s["weights"], s["fmt"], act=s["act"])}
    kept = mx.gated_fwd_save(s["x"], s["w"], s["fmt"], act=s["act"])
    dx, dw = mx.gated_bwd(s["dh"], kept, s["hidden"], s["fmt"], act=s["act"], dw_dtype=torch.bfloat16)
    return {"h": kept.h, "dx": dx, "dw": dw}


def _own_adamw(s):
    opt = s["opt"]
    opt.step(s["grads"], grad_scale=s["factor"], amax_out=s["amax_out"], t=s["t"])
    m, v = ((a.codes, a.sf) if s["bits"] == 8 else a for a in (opt.m_all, opt.v_all))
    return _adamw_outputs(s, m, v, s["amax_out"])


def _own_grad_norm(s):
    import fp4_precision_gemms_gb300 as mx

    return mx.grad_norm(s["grads"], max_norm=s["max_norm"])


_OWN = {"gated": _own_gated, "adamw": _own_adamw, "grad_norm": _own_grad_norm}


# ------------------------------------------------------------------ the definitions in 64 bits
def _grid(a, bits, least):
    """|a| to nearest, ties to even, on the numbers with `bits` after the first and no finer than 2^(least - bits)."""
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** least))) - bits)
    return torch.round(a / step) * step


def _scale_exponent(b, largest, rule):
    """floor(log2 b) less that of the largest code, or the smallest e with b 2^-e <= the largest code."""
    e = torch.floor(torch.log2(b.clamp(min=2.0 ** -200))) - math.floor(math.log2(largest))
    low = torch.exp2(e + math.floor(math.log2(largest)))  # the logarithm may be off next to a power of two
    e = torch.where(low > b, e - 1, torch.where(2 * low <= b, e + 1, e))
    if rule == "ceil":
        e = torch.where(b * torch.exp2(-e) > largest, e + 1, e)
    return torch.where(b == 0, torch.zeros_like(e), e).clamp(-127.0, 127.0)


def _fl32(x):
    return x.float().double()


def _exact_quantized(x, fmt):
    """float64 values of a matrix quantized along its rows, tensor scale included."""
    x = x.double()
    size = 16 if fmt == "nvfp4" else 32
    blocks = x.reshape(x.shape[0], -1, size)
    top = x.abs().max()
    if fmt == "nvfp4":
        ts = _fl32(top / 2688.0) if top > 0 else torch.ones_like(top)
        s = _grid(_fl32(blocks.abs().max(dim=2, keepdim=True).values / _fl32(6.0 * ts)), 3, -6).clamp(max=448.0)
        d = _fl32(s * ts)
        v = _fl32(blocks / torch.where(d == 0, torch.ones_like(d), d))
        code = torch.where(d == 0, torch.zeros_like(v), _grid(v.abs(), 1, 0).clamp(max=6.0) * torch.sign(v))
        return (code * s * ts).reshape(x.shape)
    ts = torch.ones_like(top)
    if fmt == "moss" and top > 0:
        ts = _fl32(top / 448.0)
        blocks = _fl32(blocks / ts)
    largest, bits, least = (6.0, 1, 0) if fmt == "mxfp4" else (448.0, 3, -6)
    e = _scale_exponent(blocks.abs().max(dim=2, keepdim=True).values, largest, "ceil" if fmt == "moss" else "floor")
    v = blocks * torch.exp2(-e)
    return (torch.sign(v) * _grid(v.abs(), bits, least).clamp(max=largest) * torch.exp2(e) * ts).reshape(x.shape)


def _exact_act8(x):
    b = x.reshape(x.shape[0], -1, 32)
    up = torch.exp2(_scale_exponent(b.abs().max(dim=2, keepdim=True).values, 448.0, "ceil"))
    return (torch.sign(b) * _grid((b / up).abs(), 3, -6) * up).reshape(x.shape)


def _exact_act(z, act):
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    p = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))  # (1 + tanh) / 2
    return z * p, p + z * 2 * p * (1 - p) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)


def _exact_gated(case, s):
    fmt, f = case["fmt"], case["ffn"]
    gu = _exact_quantized(s["x"], fmt) @ _exact_quantized(s["w"], fmt).T
    h = _exact_act(gu[:, :f], case["act"])[0] * gu[:, f:]
    if not case["train"]:
        return {"h": h}
    gate, up = _exact_act8(gu[:, :f]), _exact_act8(gu[:, f:])
    value, slope = _exact_act(gate, case["act"])
    dh = s["dh"].double()
    d = torch.cat([dh * slope * up, dh * value], dim=1).bfloat16()  # bf16 between the activation and the products
    return {"h": h, "dx": _exact_quantized(d, fmt) @ _exact_quantized(s["w"].T, fmt).T,
            "dw": _exact_quantized(d.T, fmt) @ _exact_quantized(s["x"].T, fmt).T}


def _exact_random16(seed, n, t, word):
    """Philox in numpy's wrapping 64-bit integers, on the host."""
    import numpy as np

    count = (n + 7) // 8
    x = np.zeros((4, count), dtype=np.uint64)
    x[0], x[1] = np.arange(count) % 2 ** 32, np.arange(count) // 2 ** 32
    x[2], x[3] = t % 2 ** 32, word
    low = np.uint64(2 ** 32 - 1)
    for r in range(10):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        k0 = np.uint64((seed + r * 0x9E3779B9) % 2 ** 32)
        k1 = np.uint64(((seed >> 32) + r * 0xBB67AE85) % 2 ** 32)
        x = np.stack([(b >> np.uint64(32)) ^ x[1] ^ k0, b & low, (a >> np.uint64(32)) ^ x[3] ^ k1, a & low])
    halves = x.T.astype(np.uint32).copy().view(np.uint16)  # the low half of a word comes first
    return torch.from_numpy(halves.reshape(-1)[:n].astype(np.int64)).cuda()


def _exact_code(x, root, random):
    """float64 code values of a flat moment."""
    n = x.numel()
    x = torch.cat([x, x.new_zeros(-n % 32)]).reshape(-1, 32)
    v = x * torch.exp2(-_scale_exponent(x.abs().max(dim=1, keepdim=True).values, 448.0, "ceil"))
    if random is None:
        code = _grid(v.abs(), 3, -6)
    else:
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        low = torch.floor(v.abs() / step)
        place = (v.abs() / step - low) * 65536.0
        random = torch.cat([random, random.new_zeros(-n % 32)]).reshape(-1, 32)
        code = torch.clamp((low + (random.double() < place).double()) * step, max=448.0)
    if root:
        code = torch.where((x > 0) & (code == 0), torch.full_like(code, 2.0 ** -9), code)
    return (code * torch.sign(x)).reshape(-1)[:n]


def _exact_moment(state, at, n):
    """What a moment's codes stand for: sign, exponent and fraction of each taken apart."""
    c = state[0].reshape(-1)[at:at + n].to(torch.int64)
    exponent, fraction = (c >> 3) & 15, (c & 7).double()
    size = torch.where(exponent > 0, (1 + fraction / 8) * torch.exp2((exponent - 7).double()), fraction * 2.0 ** -9)
    scale = torch.exp2(state[1].reshape(-1)[at // 32:(at + n + 31) // 32].double() - 127)
    return torch.where(c >= 128, -size, size) * scale.repeat_interleave(32)[:n]


def _exact_adamw(case, s):
    b1, b2 = BETAS
    t, sr = case["t"], case["rounding"] == "sr"
    eight = case["bits"] == 8
    new_p, top = s["flat"].double(), []
    new_m, new_v = ((x[0].view(-1) if eight else x).double().zero_() for x in (s["m"], s["v"]))
    for i, (p, (at, n)) in enumerate(zip(new_p.split([n for _, n in s["places"]]), s["places"])):
        g = s["grads"][i].double().reshape(-1) * (s["factor"].double() if case["scale"] else 1.0)
        if eight:
            m, v = _exact_moment(s["m"], at, n), _exact_moment(s["v"], at, n).pow(2)
        else:
            m, v = s["m"][at:at + n].double(), s["v"][at:at + n].double()
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g.pow(2)
        step = m / (1 - b1 ** t) / ((v / (1 - b2 ** t)).sqrt() + EPS)
        new = p * (1 - LR * s["decay"][i]) - LR * step
        if eight:
            random = [_exact_random16(s["seed"], n, t, 4 * i + k) if sr else None for k in range(2)]
            m, v = _exact_code(m, False, random[0]), _exact_code(v.sqrt(), True, random[1])
        new_m[at:at + n], new_v[at:at + n] = m, v
        if case["param"] == "bf16" and sr:
            unit = torch.exp2(torch.floor(torch.log2(new.abs().clamp(min=2.0 ** -126))) - 7)
            low = torch.floor(new.abs() / unit)
            up = _exact_random16(s["seed"], n, t, 4 * i + 2).double() < (new.abs() / unit - low) * 65536.0
            new = torch.sign(new) * (low + up.double()) * unit
        p.copy_(new)
        read = new.to(TYPES[case["param"]])
        top.append((read.to(torch.bfloat16) if case["copy"] else read).double().abs().max())
    out = {"p": new_p}
    if eight:
        out["m"], out["m_sf"], out["root"], out["root_sf"] = new_m.view(1, -1), None, new_v.view(1, -1), None
    else:
        out["m"], out["v"] = new_m, new_v
    if case["copy"]:
        out["copy"] = new_p
    if case["amax"]:
        out["amax"] = torch.stack(top)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gated":
        return _exact_gated(case, s)
    if case["op"] == "adamw":
        return _exact_adamw(case, s)
    norm = math.sqrt(sum(float(torch.dot(g.double().reshape(-1), g.double().reshape(-1))) for g in s["grads"]))
    return torch.tensor([norm, min(1.0, s["max_norm"] / (norm + 1e-6))], dtype=torch.float64, device="cuda")
