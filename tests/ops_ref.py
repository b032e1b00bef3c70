"""Plain 64-bit forms of the norm, activation and 8-bit checkpoint calls, and
the error bounds that their tests use.

Bounds are first-order rounding analyses with u = 2^-24 (fp32) on the values
themselves, never fitted: a sum of n terms in which no value passes through more
than k additions is off by at most k u sum|terms|; an output rounded to bf16 is
off by half a spacing, at most 2^-8 |value| with the doubled last place that an
error of the unrounded value can cost.
"""
import numpy as np
import torch

U = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -118}


def out_rounding(v, dtype):
    return v.abs() * (2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -23) + TINY[dtype]


def layout(t, how):
    """The same values as t in rows of another stride or alignment: "dense";
    "wide" (16-byte aligned rows with a gap); "odd" (rows that start anywhere)."""
    if how == "dense":
        return t.contiguous()
    rows, cols = t.shape
    ld, at = ((cols + 7) // 8 * 8 + 16, 8) if how == "wide" else (cols + 5 + cols % 2, 1)
    base = torch.full((rows, ld), float("nan"), dtype=t.dtype, device=t.device)
    v = base[:, at:at + cols]
    v.copy_(t)
    return v


# ------------------------------------------------------------------ 8-bit checkpoints
def encode(x):
    """(codes uint8 [rows, 32 G], sf uint8 [rows, G]) of a float matrix, by search
    over the 256 codes' values (numpy, 64 bits)."""
    x = x.detach().cpu().double().numpy()
    rows, cols = x.shape
    groups = -(-cols // 32)
    xp = np.zeros((rows, groups * 32))
    xp[:, :cols] = x
    xg = xp.reshape(rows, groups, 32)
    fin = np.isfinite(xg)
    b = np.where(fin, np.abs(xg), 0.0).max(-1)
    m, ex = np.frexp(b)  # b = m 2^ex; 448 = 0.875 2^9
    e = np.where(m <= 0.875, ex - 9, ex - 8)
    e = np.maximum(np.where(b == 0, 0, e), -127)
    v = np.where(fin, xg, 0.0) * np.exp2(-e.astype(np.float64))[..., None]
    grid = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(a == grid[hi], hi, code)
    code = code + 128 * np.signbit(np.where(fin, xg, 0.0))
    codes = code.astype(np.uint8).reshape(rows, groups * 32)
    nan = np.zeros((rows, groups * 32), dtype=bool)
    nan[:, :cols] = ~np.isfinite(x)
    return codes, (e + 127).astype(np.uint8), nan


def decode(codes, sf, cols):
    """float64 torch values of codes / sf given as uint8 tensors."""
    c = codes[:, :cols].to(torch.int64)
    ex, fr = (c >> 3) & 15, (c & 7).double()
    v = torch.where(ex > 0, (1 + fr / 8) * torch.exp2((ex - 7).double()), fr * 2.0 ** -9)
    v = torch.where((c & 127) == 127, torch.full_like(v, float("nan")), v)
    s = torch.exp2(sf.double() - 127).repeat_interleave(32, dim=1)[:, :cols]
    return torch.where(c >= 128, -v, v) * s


# ------------------------------------------------------------------ norm
def norm_fwd(s, w, b, kind, eps):
    s = s.double()
    mean = s.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(s[:, :1])
    rstd = 1 / torch.sqrt(((s - mean) ** 2).mean(1, keepdim=True) + eps)
    y = (s - mean) * rstd
    y = y * w.double() if w is not None else y
    y = y + b.double() if b is not None else y
    return y, mean[:, 0], rstd[:, 0]


def norm_fwd_bounds(s, w, b, kind, eps, y_dtype):
    """(bound of y, of mean, of rstd)."""
    s = s.double()
    C = s.shape[1]
    k = C / 128 + 32  # additions that a value passes through
    y, mean, rstd = norm_fwd(s, w, b, kind, eps)
    dm = k * U * s.abs().mean(1) if kind == "layer" else torch.zeros_like(mean)
    var = 1 / rstd ** 2
    rel = (k + 4) * U / 2 + 3 * U + dm ** 2 / (2 * var)
    c = (s - mean[:, None])
    ww = w.double().abs() if w is not None else 1.0
    bb = b.double().abs() if b is not None else 0.0
    by = ww * rstd[:, None] * (dm[:, None] + c.abs() * (rel[:, None] + 4 * U)) + 2 * U * (bb + y.abs())
    return by + out_rounding(y, y_dtype), dm + U * mean.abs(), rstd * rel


def norm_bwd(dy, s, mean, rstd, w, kind, dres):
    """(dx, dw, db) by the formulas, from 64-bit values."""
    dy, rstd = dy.double(), rstd.double()[:, None]
    h = (s.double() - (mean.double()[:, None] if kind == "layer" else 0.0)) * rstd
    g = dy * w.double() if w is not None else dy
    dx = g - h * (g * h).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * rstd
    if dres is not None:
        dx = dx + dres.double()
    return dx, (dy * h).sum(0), dy.sum(0)


def norm_bwd_bounds(dy, s, mean, rstd, w, kind, dres, dx_dtype):
    rows, C = dy.shape
    k = C / 128 + 32
    kr = rows / 128 + 128
    dy, rs = dy.double(), rstd.double()[:, None]
    h = ((s.double() - (mean.double()[:, None] if kind == "layer" else 0.0)) * rs).abs()
    g = (dy * w.double() if w is not None else dy).abs()
    dx, _, _ = norm_bwd(dy, s, mean, rstd, w, kind, dres)
    c1 = (g * h).mean(1, keepdim=True)
    c2 = g.mean(1, keepdim=True) if kind == "layer" else 0.0
    b = rs * (4 * U * g + h * c1 * (k + 12) * U + c2 * (k + 6) * U) + 2 * U * dx.abs()
    if dres is not None:
        b = b + U * dres.double().abs()
    return b + out_rounding(dx, dx_dtype), (kr + 4) * U * (dy.abs() * h).sum(0) + 2.0 ** -126, \
        kr * U * dy.abs().sum(0) + 2.0 ** -126


# ------------------------------------------------------------------ activation
K_TANH, C_TANH = float(np.sqrt(2 / np.pi)), 0.044715


def activation(z, act):
    """(a(z), a'(z), p, t): p the weight that multiplies z, t the argument of its exponential."""
    z = z.double()
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z), p, z.abs()
    if act == "gelu":
        p = 0.5 * torch.erfc(-z * 0.5 ** 0.5)
        return z * p, p + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5, p, z * z
    t = 2 * K_TANH * (z + C_TANH * z ** 3)
    p = torch.sigmoid(t)
    return z * p, p + z * p * torch.sigmoid(-t) * 2 * K_TANH * (1 + 3 * C_TANH * z ** 2), p, t.abs()


def activation_bounds(z, act):
    """Bounds of a(z) and a'(z) before the output's rounding.  The exponential's
    argument t is off by a few u |t|, which its result carries as a relative
    error, and the exponential itself by at most (2 + 1.2 |t|) last places."""
    z = z.double()
    a, s, p, t = activation(z, act)
    rel = (8 * t + 24) * U
    value = a.abs() * rel
    if act == "gelu":
        slope = p * rel + z.abs() * torch.exp(-z * z / 2) * rel + U * s.abs()
    else:
        inner = 2 * K_TANH * (1 + 3 * C_TANH * z ** 2) if act == "gelu_tanh" else 1.0
        q = p * (1 - p)
        slope = p * rel + z.abs() * inner * (2 * q * rel + 4 * U * p) + U * s.abs()
    return value + z.abs() * 2.0 ** -120, slope + (1 + z.abs()) * 2.0 ** -120


def assert_within(got, ref, bound, what=""):
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    err = (got - ref).abs()
    bad = (err > bound).nonzero()
    if bad.numel():
        i = tuple(bad[0].tolist())
        raise AssertionError(f"{what}: {bad.shape[0]} of {got.numel()} out of bounds; first at {i}: got {got[i].item()!r} "
                             f"expected {ref[i].item()!r} bound {bound[i].item()!r}")
