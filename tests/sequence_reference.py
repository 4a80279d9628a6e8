"""Plain 64-bit implementations of the embedding and of attention over packed
documents, on the CPU, and the error bounds their tests use."""
import math

import torch

from train_reference import tiny, u


def embed(token, w, scale, ignore):
    y = torch.zeros(len(token), w.shape[1], dtype=torch.float64)
    for i, t in enumerate(token.tolist()):
        if t == ignore:
            continue
        y[i] = scale * w[t].double() if 0 <= t < w.shape[0] else math.nan
    return y


def embed_gradient(token, dy, vocab, scale, ignore):
    """(gradient, sum of the magnitudes, number of rows) of each row of the weight."""
    dw = torch.zeros(vocab, dy.shape[1], dtype=torch.float64)
    size, count = torch.zeros_like(dw), torch.zeros(vocab, 1, dtype=torch.float64)
    keep = (token != ignore) & (token >= 0) & (token < vocab)
    rows, at = dy[keep].double(), token[keep]
    dw.index_add_(0, at, rows * scale)
    size.index_add_(0, at, rows.abs() * abs(scale))
    count.index_add_(0, at, torch.ones(len(at), 1, dtype=torch.float64))
    return dw, size, count


def visible(rows, offsets, prefix, causal, window):
    """Which keys each query sees, from the definition, pair by pair."""
    see = torch.zeros(rows, rows, dtype=torch.bool)
    for d, (a, b) in enumerate(zip(offsets, offsets[1:])):
        for i in range(a, b):
            for j in range(a, b):
                if not causal:
                    see[i, j] = True
                elif j <= i:
                    see[i, j] = window == 0 or i - j < window
                else:
                    see[i, j] = prefix is not None and j < a + prefix[d]
    return see


def attention(q, k, v, see, scale, cap=0.0, slopes=None, dout=None):
    """o, lse (and dq, dk, dv) in 64 bits, and the bounds of their errors, all before any rounding of the outputs.

    With u the relative error of a rounding to the 16-bit type, and float sums of n products of 16-bit numbers off by
    at most (n + 8) 2^-23 of the sum of their magnitudes (each product exact, each addition rounds or truncates):
    a score moves by dz = that bound of its product (times scale), 2^-22 of its own size for the scaling, the exponent's
    units and the bias, and with a cap by cap 2^-21 (1 - 2 / (1 + e): the exponential, the reciprocal and the sum are
    off by 2^-23 each, of numbers up to 2).  lse moves by the row's largest dz, the sum's (n + 8) 2^-23 and 2^-21 of
    itself and of the row's largest score (its own rounding, and the change of units).  A weight p moves by
    dz + dlse + 2^-21 (the exponential; the units of its argument are in dz and dlse) relative, then rounds by u."""
    rows, heads, dim = q.shape
    group = heads // k.shape[1]
    half = q.dtype
    e = u(half)
    names = ["o", "lse"] + (["dq", "dk", "dv"] if dout is not None else [])
    like = dict(o=q, lse=torch.zeros(heads, rows), dq=q, dk=k, dv=v)
    out = {n: torch.zeros(like[n].shape, dtype=torch.float64) for n in names}
    bound = {n: torch.zeros(like[n].shape, dtype=torch.float64) for n in names}
    has = see.any(1)
    distance = (torch.arange(rows)[:, None] - torch.arange(rows)[None, :]).abs().double()
    for h in range(heads):
        g = h // group
        a, b, c = (torch.where(torch.isfinite(x), x, 0.0) for x in (q[:, h].double(), k[:, g].double(), v[:, g].double()))
        raw = scale * (a @ b.t())
        z = raw if not cap else cap * torch.tanh(raw / cap)
        factor = torch.ones_like(z) if not cap else 1 - (z / cap) ** 2
        dz = scale * (dim + 8) * 2.0 ** -23 * (a.abs() @ b.abs().t()) + raw.abs() * 2.0 ** -22
        if cap:
            dz = dz * factor.clamp(min=2.0 ** -10) + cap * 2.0 ** -21
        if slopes is not None:
            z = z - slopes[h].double() * distance
            dz = dz + 2.0 ** -22 * slopes[h].double().abs() * distance
        dz = dz + z.abs() * 2.0 ** -22
        z = torch.where(see, z, -math.inf)
        lse = torch.where(has, torch.logsumexp(torch.where(has[:, None], z, 0.0), 1), 0.0)
        p = torch.where(see, torch.exp(z - lse[:, None]), 0.0)
        top = torch.where(see, z.abs(), 0.0).amax(1)
        n = see.sum(1).double()
        dlse = torch.where(see, dz, 0.0).amax(1) + (n + 8) * 2.0 ** -23 + (lse.abs() + top) * 2.0 ** -21
        rel = dz + dlse[:, None] + 2.0 ** -21  # of an unrounded weight
        o = p @ c
        size = p @ c.abs()
        out["o"][:, h], out["lse"][h] = o, lse
        bound["o"][:, h] = (p * (rel + 1.01 * e)) @ c.abs() + (n[:, None] + 16) * 2.0 ** -22 * size
        bound["lse"][h] = dlse
        if dout is None:
            continue
        d = torch.where(has[:, None] & torch.isfinite(dout[:, h]), dout[:, h].double(), 0.0)
        dp = d @ c.t()
        ddp = (dim + 8) * 2.0 ** -23 * (d.abs() @ c.abs().t())
        delta = (p * dp).sum(1, keepdim=True)
        # delta: from the rounded o in long rows; the sum of p dp elsewhere
        ddelta = (d.abs() * (bound["o"][:, h] + o.abs() * 1.01 * e)).sum(1, keepdim=True)
        ddelta = ddelta + (p * (dp.abs() * rel + ddp)).sum(1, keepdim=True) + (n[:, None] + 8) * 2.0 ** -22 * (p * dp.abs()).sum(1, keepdim=True)
        ds = p * (dp - delta) * factor
        # 1 - tanh^2 moves by twice the error of the tanh, 2^-21 and that of its argument
        dfactor = 2 * (2.0 ** -20 + rel / max(cap, 1.0)) if cap else 0.0
        dds = ds.abs() * (rel + 1.01 * e + 2.0 ** -21) + p * (ddp + ddelta + dfactor * (dp - delta).abs())
        # fp16: units of the own row's largest, subnormals 2^-25 / 2^13 of it apart
        dds = dds + 2.0 ** -36 * torch.maximum(ds.abs().amax(1, keepdim=True), ds.abs().amax(0, keepdim=True)) * see
        dpw = p * (rel + 1.01 * e)
        out["dq"][:, h] = scale * ds @ b
        bound["dq"][:, h] = scale * (dds @ b.abs() + (n[:, None] + 16) * 2.0 ** -22 * (ds.abs() @ b.abs()))
        out["dk"][:, g] += scale * ds.t() @ a
        out["dv"][:, g] += p.t() @ d
        m = (group * see.sum(0).double() + 16)[:, None] * 2.0 ** -22
        bound["dk"][:, g] += scale * (dds.t() @ a.abs() + m * (ds.abs().t() @ a.abs()))
        # (and fp16's subnormal weights: 2^-25)
        bound["dv"][:, g] += dpw.t() @ d.abs() + m * (p.t() @ d.abs()) + 2.0 ** -25 * see.double().t() @ d.abs()
    for n in names:
        if n != "lse":
            bound[n] = bound[n] * 1.02 + out[n].abs() * 1.01 * e + tiny(half)
    return out, bound
