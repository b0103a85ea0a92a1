"""Plain 64-bit implementations of the 8-bit pool, of attention with a window
and of normalised heads, straight from the formulas; no code of the library."""
import math

import torch

import step_util as su

U = 2.0 ** -24


def scale_of(amax):
    """Least power of two s, within 2^-100 .. 2^119, with amax <= 448 s (a float)."""
    e = -100
    while e < 119 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def scales_of(x, dims):
    """scale_of the largest finite magnitude over dims."""
    a = x.double().abs()
    a = torch.where(torch.isfinite(a), a, torch.zeros_like(a)).amax(dims)
    return torch.tensor([scale_of(v) for v in a.flatten().tolist()], dtype=torch.float64).view(a.shape)


def e4m3(x):
    """x rounded to the nearest e4m3 value, ties to even, saturating; NaN for what is not finite (64 bits)."""
    x = x.double()
    y = x.clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    y = torch.round(y / step) * step
    return torch.where(torch.isfinite(x), y, torch.full_like(y, math.nan))


def to_bytes(y):
    """The bytes of e4m3 values (exact)."""
    return y.float().to(torch.float8_e4m3fn).view(torch.uint8)


def values(b8, scales):
    """What bytes [..., page, heads, dim] under scales [..., heads] stand for, 64 bits."""
    return b8.view(torch.float8_e4m3fn).float().double() * scales.double()[..., None, :, None]


class Batch8(su.Batch):
    """A Batch whose pool is held in 8 bits: bytes8, scales, and pool as the bf16 values that they stand for.  Bytes
    that no token is in are NaN, scales of blocks that hold nothing are too."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.quantise()

    def quantise(self):
        x = self.pool.double()
        s = scales_of(x, (3, 5))
        none = ~torch.isfinite(x).any(5).any(3)
        self.bytes8 = to_bytes(e4m3(x / s[:, :, :, None, :, None]))
        self.scales = torch.where(none, torch.full_like(s, math.nan), s).float()
        self.pool = values(self.bytes8, s).bfloat16()


def attend_window64(b, q, scale, window=None, sinks=0, layer=0):
    """(out, lse, bound of out, bound of lse) as su.attend64, of rows that see the tokens t <= p with t > p - window or
    t < sinks, p counted from the start of the prefix.  A row without a slot of its own stands on the prefix's last token.

    The bounds are derived there.  An 8-bit pool's values are exact in bf16, and in fp16 beside each other; its weights go
    into the second product as fp16 (or, more exactly, as two bf16): half a step of 2^-11, so 2^-12 of each, and half of
    fp16's least step, 2^-25, for one below 2^-14, relative to the row's largest weight, which is 1 or more before the
    division by their sum, itself 1 or more."""
    rows, hq, D = q.shape
    rep = hq // b.heads
    out = torch.full((rows, hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((rows, hq), math.nan, dtype=torch.float64)
    eo, el = torch.zeros_like(out), torch.zeros_like(lse)
    for s, (n, m) in enumerate(zip(b.lens, b.new)):
        k, v = b.cached(0, s, layer), b.cached(1, s, layer)
        pre = k.shape[0] - n
        for i in range(m):
            r = b.q_start[s] + i
            p = pre + max(-1, n - m + i)
            t = [x for x in range(p + 1) if window is None or x > p - window or x < sinks]
            if not t:
                out[r], lse[r] = 0.0, -math.inf
                continue
            kt, vt = k[t], v[t]
            for h in range(hq):
                kk, vv, x = kt[:, h // rep], vt[:, h // rep], q[r, h].double()
                sc = (kk @ x) * scale
                lse[r, h] = torch.logsumexp(sc, 0)
                if float(lse[r, h]) == -math.inf:
                    out[r, h] = 0.0
                    continue
                w = torch.exp(sc - lse[r, h])
                out[r, h] = w @ vv
                # an infinite score has no error of its own: the bounds are those of the finite ones
                size = ((kk.abs() @ x.abs()) * scale)[torch.isfinite(sc)]
                S = float(size.max()) if size.numel() else 0.0
                rel = (D + 4) * U * S + (len(t) + 12) * U
                if math.isfinite(float(lse[r, h])):
                    el[r, h] = rel + 4 * U * (abs(float(lse[r, h])) + S)
                    part = (2 * rel + 2.0 ** -16) * (w @ vv.abs())
                    if isinstance(b, Batch8):
                        part = (2 * rel + 2.0 ** -12) * (w @ vv.abs()) + 2.0 ** -25 * vv.abs().sum(0)
                    eo[r, h] = part * (1 + 2.0 ** -8) + 2.0 ** -8 * out[r, h].abs() + 2.0 ** -133
    return out, lse, eo, el


def norm64(x, weight, eps, centered):
    """(normalised heads, bound of their error in float32), x [rows, heads, dim].

    With A = max |x| of a head and s its sqrt(mean + eps): the mean is off by e = (D + 2) u A (0 where none is
    subtracted), x - c by that and u |x - c|, the mean of squares by 2 e s + e^2 and (D + 4) u of itself, the root and
    the quotient by half of it and 4 u, the products with the weight by 2 u more."""
    D = x.shape[-1]
    x = x.double()
    w = 1.0 if weight is None else weight.double()
    c = x.mean(-1, keepdim=True) if centered else torch.zeros_like(x[..., :1])
    e = (D + 2) * U * x.abs().amax(-1, keepdim=True) if centered else torch.zeros_like(c)
    d = x - c
    s = (d.square().mean(-1, keepdim=True) + eps).sqrt()
    y = d / s * w
    wa = w if isinstance(w, float) else w.abs()
    rel = (2 * e * s + e * e) / (s * s) + (D + 4) * U
    return y, wa / s * (e + U * d.abs()) + y.abs() * (rel / 2 + 6 * U)


def rotated64(x, ex, positions, f, gain, rot, interleaved):
    """(rotated, bound): su.rope64, with 2^-20 of |x| + |y| for float32 angles and sums, and the operands' own errors."""
    y, size = su.rope64(x, positions, f, gain, rot, interleaved)
    err = ex.clone()
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        err[..., a] = err[..., b] = (ex[..., a] + ex[..., b]) * gain
    return y, err * (1 + 2.0 ** -20) + size * 2.0 ** -20


def rounded(want, err, dtype):
    """Bound after one rounding to dtype of a value that may be off by err."""
    info = torch.finfo(dtype)
    return err + (want.abs() + err) * info.eps / 2 + info.smallest_normal * info.eps
