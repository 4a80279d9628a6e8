"""Plain 64-bit implementations of the training operators, on the CPU, and the
error bounds their tests use.

u(t) is the largest relative error of one rounding to t (half a step)."""
import math

import torch

MAX8 = {"e4m3": 448.0, "e5m2": 57344.0}
#: mantissa bits and the exponent of the smallest normal value
SHAPE8 = {"e4m3": (3, -6), "e5m2": (2, -14)}
TYPE8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def u(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the spacing of the subnormals: the absolute error of a rounding there."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def pitch_of(cols):
    return (cols + 31) // 32 * 32


def encode(x, fmt):
    """(values, exponents + 127) of the checkpoint of x (any float type): values rows x cols in 64 bits, exponents
    rows x blocks, from the definition."""
    rows, cols = x.shape
    pitch = pitch_of(cols)
    wide = torch.zeros(rows, pitch, dtype=torch.float64)
    wide[:, :cols] = x.double()
    blocks = wide.view(rows, pitch // 32, 32)
    finite = torch.where(torch.isfinite(blocks), blocks.abs(), torch.zeros(()))
    amax = finite.amax(2)
    e = torch.full_like(amax, -127.0)
    for k in range(-126, 129):  # the smallest e with amax <= MAX 2^e, by trying each
        e = torch.where(amax > MAX8[fmt] * 2.0 ** (k - 1), float(k), e)
    scale = torch.exp2(e)[:, :, None]
    bits, least = SHAPE8[fmt]
    y = blocks / scale
    level = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** (least - 1)))).clamp(min=least)
    step = torch.exp2(level - bits)
    values = torch.round(y / step) * step * scale  # torch.round: ties to even
    if fmt == "e4m3":
        values = torch.where(torch.isinf(blocks), torch.full_like(values, math.nan), values)
    else:
        values = torch.where(torch.isinf(blocks), blocks, values)
    return values.view(rows, pitch)[:, :cols], (e + 127).to(torch.uint8)


def parts(buf, rows, cols):
    """(codes rows x pitch, scale bytes rows x blocks) of a checkpoint buffer."""
    pitch = pitch_of(cols)
    at = (rows * pitch + 255) // 256 * 256
    buf = buf.cpu()
    return buf[: rows * pitch].view(rows, pitch), buf[at: at + rows * (pitch // 32)].view(rows, pitch // 32)


def decode(buf, rows, cols, fmt):
    codes, bytes_ = parts(buf, rows, cols)
    v = codes.contiguous().view(TYPE8[fmt]).double().view(rows, pitch_of(cols) // 32, 32)
    return (v * torch.exp2(bytes_.double() - 127)[:, :, None]).reshape(rows, pitch_of(cols))[:, :cols]


def buffer_of(codes, bytes_):
    """A checkpoint buffer with the given codes and scale bytes."""
    rows, pitch = codes.shape
    at = (rows * pitch + 255) // 256 * 256
    buf = torch.zeros(at + bytes_.numel(), dtype=torch.uint8)
    buf[: rows * pitch] = codes.reshape(-1)
    buf[at:] = bytes_.reshape(-1)
    return buf


def act(x, name):
    """a(x), a'(x) and the size of the terms a' is the sum of."""
    if name == "silu":
        q, dq = x, torch.ones_like(x)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        q, dq = c * (x + 0.044715 * x ** 3), c * (1 + 3 * 0.044715 * x * x)
    s = torch.sigmoid(q)
    # s (1 - s), from the smaller of the two, which the difference would lose
    both = torch.exp(-q.abs()) / (1 + torch.exp(-q.abs())) ** 2
    term = x * both * dq
    return x * s, s + term, s + term.abs()


#: Relative error of the activation's float arithmetic (a, and each of the terms of a'), in units of 2^-24: q of gelu is
#: four rounded operations and enters an exponent, which multiplies its relative error by |q|; |q| is kept within 88 by
#: the exponent's range and beyond 20 the result no longer depends on it to that accuracy, except through
#: s = exp(q) for negative q, where the relative error of s is |q| 4 2^-24.  The exponential, the sum, the reciprocal
#: and two products add one to two units each.
def act_error(x, name):
    if name == "silu":
        q = x.abs()
        return 12 * 2.0 ** -24 * torch.ones_like(q)
    q = (1.5957691216057308 * (x + 0.044715 * x ** 3)).abs().clamp(max=130)
    return (12 + 5 * q) * 2.0 ** -24


def xent(h, w, target, weight, ignore, scale):
    """loss, lse, dh, dw in 64 bits, and G, p."""
    h, w = h.double(), w.double()
    rows, vocab = h.shape[0], w.shape[0]
    keep = target != ignore
    h = torch.where(keep[:, None], h, torch.zeros(()))
    z = h @ w.t()
    lse = torch.logsumexp(z, 1)
    at = torch.where(keep, target, torch.zeros_like(target))
    wt = torch.ones(rows, dtype=torch.float64) if weight is None else torch.where(keep, weight.double(), 0.0)
    wt = torch.where(keep, wt, torch.zeros(()))
    loss = torch.where(keep, wt * (lse - z.gather(1, at[:, None])[:, 0]), torch.zeros(()))
    p = torch.exp(z - lse[:, None])
    hot = torch.zeros(rows, vocab, dtype=torch.float64).scatter_(1, at[:, None], 1.0)
    g = wt[:, None] * (p - hot)
    lse = torch.where(keep, lse, torch.zeros(()))
    return dict(loss=loss, lse=lse, dh=scale * (g @ w), dw=scale * (g.t() @ h), g=g, p=p, h=h, w=w, weight=wt, z=z)


def xent_bounds(r, dtype, scale, g_error=None):
    """Error bounds of loss, lse, dh and dw before the outputs' rounding (r: xent()'s result).

    A float sum of n products of 16-bit numbers is off by at most (n + 8) 2^-23 of the sum of their magnitudes (each
    product is exact in the sum's 24 bits, each addition rounds or truncates).  With dz that bound of a logit's, taken
    over the row: lse moves by at most max dz, plus the exponentials' and the sum's own error: each exponential is off
    by 2^-16 relative at most, where its argument's rounding counts (|x| <= 88: 88 * 1.45 * 2^-24 < 2^-16), the sum by
    (vocab + 16) 2^-24.  p moves by dz + dlse relative; E rounds to 11 bits (2^-11), or by 2^-40 of its own piece's
    maximum (at most 1 as a probability) where it is subnormal; G rounds to its type (and fp16, held times 256, by
    2^-33 where subnormal).  g_error: the relative error of G's rounding, where it is not one rounding to dtype."""
    vocab, hidden = r["w"].shape
    dz = (hidden + 8) * 2.0 ** -23 * (r["h"].abs() @ r["w"].abs().t()).amax(1)
    sum_error = 2.0 ** -16 + (vocab + 16) * 2.0 ** -24
    dlse = dz + sum_error + r["lse"].abs() * 2.0 ** -22
    at = r["weight"].abs()
    dloss = at * (dz + dlse + (r["lse"].abs() + r["z"].abs().amax(1)) * 2.0 ** -22)
    rel = (dz + dlse + 2.0 ** -16 + 2.0 ** -11)[:, None]
    # fp16's subnormals are 2^-24 apart: G times 256 is off by at most 2^-25 there, G by 2^-33, whatever the weight
    floor = 2.0 ** -33 if dtype == torch.float16 else 0.0
    # p's error, then G's rounding; the target's entry, weight * (p - 1), comes from float logits: its error is p's too
    g_error = 1.01 * u(dtype) if g_error is None else g_error
    dg = at[:, None] * (r["p"] * rel + 2.0 ** -39) + r["g"].abs() * (g_error + 2.0 ** -22)
    dg = dg + floor * (at > 0)[:, None]
    g = r["g"].abs()
    w, h = r["w"].abs(), r["h"].abs()
    rows = h.shape[0]
    dh = abs(scale) * (dg @ w + (vocab + 300) * 2.0 ** -23 * (g @ w))
    dw = abs(scale) * (dg.t() @ h + (rows + 300) * 2.0 ** -23 * (g.t() @ h))
    return dict(loss=dloss, lse=dlse, dh=dh, dw=dw)
