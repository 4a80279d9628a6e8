"""The training operators on the GPU at values and sizes near the ends of their
ranges, against the definitions in 64 bits: cross entropy with logits of any
finite magnitude and row weights of any, the widest rows, rows that end inside a
16-byte chunk, the largest sizes."""
import math

import pytest
import torch

import adamw_optimizer_step_tensor_amd as A
import train_reference as R
from test_gpu_train import BF16, DEV, F16, F32, Guarded, close, gen, wgrad_case

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Cross entropy: large finite logits
# ---------------------------------------------------------------------------
#
# The logits are exact in float: each is one large term plus a small multiple of two of its float's units, or small
# multiples of 1/8 alone, so the products' sums round nothing and every error comes from what follows them.

LEVELS = {BF16: [2.0 ** k for k in (19, 20, 21, 24, 25, 27, 30, 33, 37, 40, 57, 70, 99, 100, 101, 120)],
          F16: [2.0 ** k for k in (19, 20, 21, 24, 25, 27, 30, 32)]}
ONE = {BF16: 2.0 ** 60, F16: 2.0 ** 15}  # most that one factor holds here
MASK = slice(128, 390)  # one part of 128 whole, one in part, across a tile's border


def factors(level, dtype):
    """level as a sum of at most four equal products."""
    terms = 4 if level > ONE[dtype] ** 2 else 1
    a = min(ONE[dtype], 2.0 ** (math.frexp(level / terms)[1] // 2))
    return terms, a, level / terms / a


def large_case(kind, level, dtype, rows, hidden, vocab=700, seed=0):
    """h, w and targets.  masked: a range of the vocabulary at -level, the others ordinary; mixed: that range at +level,
    the others ordinary; live, low: all logits at +level or -level, apart by multiples of two units."""
    g = gen(seed)
    h, w = torch.zeros(rows, hidden), torch.zeros(vocab, hidden)
    terms, a, b = factors(level, dtype)
    j = torch.randint(0, 8, (vocab,), generator=g).float()
    h[:, :terms] = a
    h[:, 8] = torch.arange(rows) % 3
    at = torch.randint(0, vocab, (rows,), generator=g)
    if kind in ("masked", "mixed"):
        w[MASK, :terms] = b if kind == "mixed" else -b
        w[:, 8] = j / 8
        w[MASK, 8] = 0
    else:
        w[:, :terms] = b if kind == "live" else -b
        w[:, 8] = j * level * 2.0 ** -23 * (2 if kind == "live" else 1)
    return h.to(dtype), w.to(dtype), at


def large_reference(h, w, at, weight, scale, dtype):
    """Outputs in 64 bits, and their bounds: train_reference.xent_bounds' terms without the logits' error.  An entry
    whose logit lies 200 below the row's largest has probability 0 exactly (e^-200 is below every float)."""
    h, w, weight = h.double(), w.double(), weight.double()
    vocab, rows = w.shape[0], h.shape[0]
    z = h @ w.t()
    assert torch.equal(z, z.float().double())  # exact in float
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1)
    below = (z.gather(1, at[:, None]) - top)[:, 0] - torch.log(total)
    p = e / total[:, None]
    hot = torch.zeros_like(z).scatter_(1, at[:, None], 1.0)
    g = weight[:, None] * (p - hot)
    r = dict(lse=top[:, 0] + torch.log(total), loss=-weight * below, dh=scale * (g @ w), dw=scale * (g.t() @ h))
    sums = 2.0 ** -16 + (vocab + 16) * 2.0 ** -24
    live = (z > top - 200).double()
    dg = weight[:, None] * (p * (sums + 2.0 ** -16 + 2.0 ** -11) + 2.0 ** -39 * live)
    dg = dg + g.abs() * (1.01 * R.u(dtype) + 2.0 ** -22) + (2.0 ** -33 * live if dtype == F16 else 0)
    g = g.abs()
    b = dict(lse=sums + r["lse"].abs() * 2.0 ** -22, loss=weight * (sums + below.abs() * 2.0 ** -22),
             dh=scale * (dg @ w.abs() + (vocab + 300) * 2.0 ** -23 * (g @ w.abs())),
             dw=scale * (dg.t() @ h.abs() + (rows + 300) * 2.0 ** -23 * (g.t() @ h.abs())))
    return r, b


def check_large(h, w, at, dtype, what, scale=1.0):
    rows, hidden = h.shape
    vocab = w.shape[0]
    weight = (torch.arange(rows) % 4 + 1).float() / 4
    r, b = large_reference(h, w, at, weight, scale, dtype)
    loss, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    hd, wd, td, wt = h.to(DEV), w.to(DEV), at.to(DEV), weight.to(DEV)
    A.adam_xent(hd, wd, td, loss, lse=lse, weight=wt)
    close(lse.cpu(), r["lse"], b["lse"], what + " lse alone")
    close(loss.cpu(), r["loss"], b["loss"], what + " loss alone")
    dh, dw = Guarded(rows, hidden, dtype), Guarded(vocab, hidden, F32)
    A.adam_xent(hd, wd, td, loss, lse=lse, weight=wt, dh=dh.view, dw=dw.view,
                d_loss_scale=torch.tensor([scale], device=DEV))
    close(lse.cpu(), r["lse"], b["lse"], what + " lse")
    close(loss.cpu(), r["loss"], b["loss"], what + " loss")
    close(dh.check(), r["dh"], b["dh"] + r["dh"].abs() * R.u(dtype) * 1.01 + R.tiny(dtype), what + " dh")
    close(dw.check(), r["dw"], b["dw"] + r["dw"].abs() * R.u(F32) * 1.01 + R.tiny(F32), what + " dw")


@pytest.mark.parametrize("rows,hidden", [(5, 16), (140, 16), (5, 2048)])  # 2048: the logits' product is split over it
@pytest.mark.parametrize("kind", ["masked", "mixed", "live", "low"])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_xent_large_logits(dtype, kind, rows, hidden):
    for k, level in enumerate(LEVELS[dtype]):
        h, w, at = large_case(kind, level, dtype, rows, hidden, seed=k)
        check_large(h, w, at, dtype, f"{kind} {level:g} {rows}x{hidden}")


@pytest.mark.parametrize("value", [-1e6, -3e7, -1e9, -1e10, -1e12, -1e20, -1e30, -2e30, -1e31, torch.finfo(BF16).min])
def test_xent_vocabulary_masked_by_a_large_value(value):
    """Weights of any large negative value in a range of the vocabulary: those entries have probability 0, the others are
    as they would be without them."""
    g = gen(3)
    h, w = torch.randint(-8, 9, (40, 16), generator=g).float() / 8, torch.randint(-8, 9, (600, 16), generator=g).float() / 8
    h[:, 0] = 1
    w[MASK] = 0
    w[MASK, 0] = value
    at = torch.randint(0, 128, (40,), generator=g)
    check_large(h.to(BF16), w.to(BF16), at, BF16, f"masked by {value:g}")


def test_xent_lowest_values_in_both_directions():
    """Rows whose logits are all 0 or the type's lowest value, or all 0 or its largest."""
    h = torch.full((2, 8), 1.0, dtype=BF16)
    h[1] = -1.0
    w = torch.zeros(200, 8, dtype=BF16)
    w[100:, 0] = torch.finfo(BF16).min
    for t in ([4, 150], [3, 20], [190, 150]):
        check_large(h, w, torch.tensor(t), BF16, f"targets {t}", scale=2.0 ** -10)


# ---------------------------------------------------------------------------
# Streaming calls: the widest rows
# ---------------------------------------------------------------------------

def test_widest_rows():
    """Rows of 2^31 - 1 columns, whose last group of 8 ends at column 2^31: the last block of each row is stored, decoded
    and activated as it is alone, and nothing behind a row is read or written."""
    rows, cols, last = 2, (1 << 31) - 1, 31
    g = gen(9)
    x = torch.zeros(rows * cols + 64, dtype=BF16, device=DEV)
    x[rows * cols:] = math.nan
    x = x[: rows * cols].view(rows, cols)
    x[:, -last:] = torch.randn(rows, last, generator=g).to(BF16).to(DEV)
    x[1, :8] = 3.0  # behind the first row
    n8 = A.adam_act8_bytes(rows, cols)
    buf = torch.full((n8 + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    A.adam_act8_store(x, buf[:n8])
    codes = buf[: rows << 31].view(rows, 1 << 31)
    tail = x[:, -last:].contiguous()
    alone = torch.empty(A.adam_act8_bytes(rows, last), dtype=torch.uint8, device=DEV)
    A.adam_act8_store(tail, alone)
    assert torch.equal(codes[:, -32:].cpu(), R.parts(alone, rows, last)[0])  # the padding's code, 0, among them
    assert bool((buf[n8:] == 0xA5).all())
    out = torch.full((rows * cols + 64,), 7.0, dtype=BF16, device=DEV)
    view = out[: rows * cols].view(rows, cols)
    A.adam_act8_load(buf[:n8], view)
    want = torch.empty_like(tail)
    A.adam_act8_load(alone, want)
    assert torch.equal(view[:, -last:], want)
    assert bool((view[1, :8] == 3.0).all()) and bool((out[rows * cols:] == 7.0).all())
    del buf, codes
    A.adam_glu_forward(x, x, view)
    A.adam_glu_forward(tail, tail, want)
    assert torch.equal(view[:, -last:], want)
    assert bool((out[rows * cols:] == 7.0).all()) and float(view[0, -last - 1]) == 0.0
    assert torch.equal(view[1, :8], view[1, :1].expand(8)) and float(view[1, 0]) > 8.5  # silu(3) * 3


# ---------------------------------------------------------------------------
# Weight gradient: rows read where they lie whose last 16 bytes are not all theirs
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [33, 95, 96, 223, 224, 225, 352, 480])
@pytest.mark.parametrize("n,pad", [(3, 5), (100, 4), (257, 7), (262, 2)])
def test_wgrad_of_rows_that_end_inside_a_chunk(rows, n, pad):
    """dy with an aligned stride and a width that is no multiple of 8; its padding is NaN."""
    for dtype in (BF16, F16):
        wgrad_case(rows, n, 300, dtype, F32, "e4m3", pad=pad, seed=rows)


# ---------------------------------------------------------------------------
# Cross entropy: row weights of any magnitude
# ---------------------------------------------------------------------------

def weighted_case(rows, hidden, vocab, dtype, weight, scale, logit_std=0.5, piece_rows=0, seed=0):
    """G's rounding may cost an entry u(dtype) of itself, or in fp16 2^-39 of the largest weight; never more."""
    g = gen(seed)
    h = torch.randn(rows, hidden, generator=g).to(dtype)
    w = (torch.randn(vocab, hidden, generator=g) * (logit_std / math.sqrt(hidden))).to(dtype)
    t = torch.randint(0, vocab, (rows,), generator=g)
    t[1::7] = -100
    weight = weight.clone()
    r = R.xent(h, w, t, weight, -100, scale)
    b = R.xent_bounds(r, BF16, scale, 1.01 * R.u(dtype))  # bf16: without an absolute floor
    kept = t != -100
    floor = 2.0 ** -39 * float(weight[kept].double().abs().max()) * scale if dtype == F16 else 0.0
    weight[~kept] = math.inf  # a weight that is not read
    loss, dh, dw = torch.empty(rows, device=DEV), Guarded(rows, hidden, dtype), Guarded(vocab, hidden, F32)
    A.adam_xent(h.to(DEV), w.to(DEV), t.to(DEV), loss, weight=weight.to(DEV), dh=dh.view, dw=dw.view,
                d_loss_scale=torch.tensor([scale], device=DEV), piece_rows=piece_rows)
    close(loss.cpu(), r["loss"], b["loss"] + R.tiny(F32), "loss")
    close(dh.check(), r["dh"], b["dh"] + floor * r["w"].abs().sum(0) + r["dh"].abs() * R.u(dtype) * 1.01 + R.tiny(dtype), "dh")
    close(dw.check(), r["dw"], b["dw"] + floor * r["h"].abs().sum(0) + r["dw"].abs() * R.u(F32) * 1.01 + R.tiny(F32), "dw")


@pytest.mark.parametrize("rows,vocab,piece_rows", [(20, 20000, 0), (140, 20000, 0), (600, 3001, 256), (1100, 3001, 0)])
@pytest.mark.parametrize("exponent", [-110, -60, -30, -20, -16, -13, -3, 0, 8, 9, 20, 100])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_xent_weights_of_one_magnitude(dtype, exponent, rows, vocab, piece_rows):
    """Weights between 1 and 2 times a power of two, and the loss scale that undoes it."""
    weight = (1 + torch.rand(rows, generator=gen(1))) * 2.0 ** exponent
    weighted_case(rows, 64, vocab, dtype, weight, 2.0 ** -exponent, piece_rows=piece_rows, seed=2)


@pytest.mark.parametrize("rows", [60, 300])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_xent_weights_of_many_magnitudes(dtype, rows):
    """Between 2^-12 and 2^12, of both signs, some zero; and all zero."""
    g = gen(4)
    weight = torch.exp2(24 * torch.rand(rows, generator=g) - 12) * (1 - 2 * (torch.rand(rows, generator=g) < 0.3).float())
    weight[::5] = 0
    weighted_case(rows, 64, 5000, dtype, weight, 1.0, seed=5)
    weighted_case(rows, 64, 5000, dtype, torch.zeros(rows), 1.0, seed=6)


@pytest.mark.parametrize("rows", [60, 1500])
def test_xent_weights_that_are_not_finite(rows):
    """An infinite or NaN weight spoils its own row's dh and the dw that it enters, and no other row's dh."""
    g = gen(7)
    h, w = torch.randn(rows, 32, generator=g).to(F16), (torch.randn(900, 32, generator=g) / 8).to(F16)
    t, weight = torch.randint(0, 900, (rows,), generator=g), torch.full((rows,), 2.0 ** -20)
    r = R.xent(h, w, t, weight, -100, 2.0 ** 20)
    b = R.xent_bounds(r, BF16, 2.0 ** 20, 1.01 * R.u(F16))
    weight[3], weight[9] = math.inf, math.nan
    loss, dh, dw = torch.empty(rows, device=DEV), torch.empty(rows, 32, dtype=F16, device=DEV), torch.empty(900, 32, device=DEV)
    A.adam_xent(h.to(DEV), w.to(DEV), t.to(DEV), loss, weight=weight.to(DEV), dh=dh, dw=dw,
                d_loss_scale=torch.tensor([2.0 ** 20], device=DEV))
    other = torch.ones(rows, dtype=torch.bool)
    other[[3, 9]] = False
    assert not bool(torch.isfinite(dh.cpu()[~other]).any()) and not bool(torch.isfinite(dw).any())
    assert float(loss[3]) == math.inf and bool(torch.isnan(loss[9]))
    bound = b["dh"] + 2.0 ** -39 * r["w"].abs().sum(0) + r["dh"].abs() * R.u(F16) * 1.01 + R.tiny(F16)
    close(dh.cpu()[other], r["dh"][other], bound[other], "dh")


# ---------------------------------------------------------------------------
# Gated activation: the derivative where it nears 1
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_glu_derivative_of_positive_gates(name):
    """float gates of every e4m3 mantissa between 2^-6 and 2^7, one a block, so that the checkpoint holds them exactly.
    s = 1 / (1 + e) is off by one unit of its float (2^-23) for the reciprocal and half a unit for each of the sum before
    it and the one behind it, and by e's own relative error times 1 - s; the other term by the arithmetic's
    (train_reference.act_error)."""
    gates = torch.tensor([(1 + k / 8) * 2.0 ** e for e in range(-6, 7) for k in range(8)])
    rows = len(gates)
    wide = torch.zeros(rows, 32)
    wide[:, 0] = gates
    buf_g, buf_u = (torch.empty(A.adam_act8_bytes(rows, 32), dtype=torch.uint8, device=DEV) for _ in range(2))
    A.adam_act8_store(wide.to(DEV), buf_g)
    A.adam_act8_store(torch.ones(rows, 32, device=DEV), buf_u)
    assert torch.equal(R.decode(buf_g, rows, 32, "e4m3"), wide.double())
    dg, du = torch.empty(rows, 32, device=DEV), torch.empty(rows, 32, device=DEV)
    A.adam_glu_backward(torch.ones(rows, 32, device=DEV), buf_g, buf_u, dg, du, name)
    x = gates.double()
    _, want, size = R.act(x, name)
    q = x if name == "silu" else 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    rest = 1 / (1 + torch.exp(q))  # 1 - s
    term = size - 1 / (1 + torch.exp(-q))
    bound = 2.0 ** -22 + R.act_error(x, name) * (rest + term)
    close(dg[:, 0].cpu(), want, bound, "dgate")


# ---------------------------------------------------------------------------
# Cross entropy: infinite logits
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("hidden", [16, 2048])
@pytest.mark.parametrize("rows", [12, 200])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_xent_rows_with_infinite_logits(dtype, rows, hidden):
    """lse, loss and gradient as their definitions say, in the rows that have them; the others as without those rows."""
    g = gen(11)
    vocab = 700
    h, w = torch.zeros(rows, hidden), torch.zeros(vocab, hidden)
    h[:, :4] = torch.randint(-8, 9, (rows, 4), generator=g) / 8
    w[:, :4] = torch.randint(-8, 9, (vocab, 4), generator=g) / 8
    # h of inf times column k: +inf where w is 1, -inf where it is -1, NaN where it is 0
    w[:, 8:12] = -1
    w[5, 8] = 1                # one logit of +inf, the others -inf
    w[[5, 200, 650], 9] = 1    # one in each of three tiles
    w[300, 10] = 0             # a NaN among -inf
    w[77, 11], w[78, 11] = 1, 0  # +inf and NaN in one part
    at = torch.randint(0, vocab, (rows,), generator=g)
    special = {1: (8, 9), 2: (8, 5), 3: (9, 201), 4: (9, 650), 6: (10, 5), 7: (11, 3), 8: (8, 6)}
    for row, (k, target) in special.items():
        h[row, k] = math.inf
        at[row] = target
    loss, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dh, dw = torch.empty(rows, hidden, dtype=dtype, device=DEV), torch.empty(vocab, hidden, device=DEV)
    hd, wd, td = h.to(dtype).to(DEV), w.to(dtype).to(DEV), at.to(DEV)
    bad = list(special)
    for grad in (False, True):
        A.adam_xent(hd, wd, td, loss, lse=lse, **(dict(dh=dh, dw=dw) if grad else {}))
        inf, nan = math.inf, math.nan
        want_lse = torch.tensor([inf, inf, inf, inf, nan, nan, inf])
        want_loss = torch.tensor([inf, nan, inf, nan, nan, nan, inf])
        assert torch.equal(torch.nan_to_num(lse.cpu()[bad], nan=-1.0), torch.nan_to_num(want_lse, nan=-1.0)), lse[bad]
        assert torch.equal(torch.nan_to_num(loss.cpu()[bad], nan=-1.0), torch.nan_to_num(want_loss, nan=-1.0)), loss[bad]
        others = torch.ones(rows, dtype=torch.bool)
        others[bad] = False
        assert bool(torch.isfinite(loss.cpu()[others]).all()) and bool(torch.isfinite(lse.cpu()[others]).all())
        z = h.double()[others] @ w.double().t()
        want = torch.logsumexp(z, 1)
        assert float((lse.cpu()[others] - want).abs().max()) < 1e-4
    assert bool(torch.isnan(dh[bad]).all()) and bool(torch.isfinite(dh.cpu()[others]).all())
    assert bool(torch.isnan(dw).all())


def test_xent_logits_that_overflow():
    """Products beyond the float range are infinite logits: of +inf as above, of -inf with probability 0."""
    h, w = torch.zeros(3, 16), torch.zeros(300, 16)
    h[:, 0], w[:, 0] = 1, torch.arange(300) % 5
    w[17, 1], w[40:200, 2] = 2.0 ** 60, -(2.0 ** 60)
    h[1, 1], h[2, 2] = 2.0 ** 100, 2.0 ** 100
    at = torch.tensor([3, 4, 39])
    loss, lse = torch.empty(3, device=DEV), torch.empty(3, device=DEV)
    A.adam_xent(h.to(BF16).to(DEV), w.to(BF16).to(DEV), at.to(DEV), loss, lse=lse)
    z = w[:, 0].double()
    assert abs(float(lse[0]) - float(torch.logsumexp(z, 0))) < 1e-4
    assert float(lse[1]) == math.inf and float(loss[1]) == math.inf
    z[40:200] = -math.inf
    assert abs(float(lse[2]) - float(torch.logsumexp(z, 0))) < 1e-4
    assert abs(float(loss[2]) - float(torch.logsumexp(z, 0) - z[39])) < 1e-4


# ---------------------------------------------------------------------------
# The largest sizes
# ---------------------------------------------------------------------------

def small_multiples(g, *shape):
    return torch.randint(-8, 9, shape, generator=g).float() / 8


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_xent_largest_hidden(dtype):
    """2^21 hidden elements, of which a few are not zero, so that the logits stay exact."""
    g = gen(20)
    h, w = torch.zeros(3, 1 << 21), torch.zeros(5, 1 << 21)
    at = [0, 7, 1000003, (1 << 21) - 2, (1 << 21) - 1]
    h[:, at], w[:, at] = small_multiples(g, 3, 5), small_multiples(g, 5, 5)
    check_large(h.to(dtype), w.to(dtype), torch.tensor([4, 0, 2]), dtype, "hidden 2^21")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_xent_largest_vocabulary(dtype):
    g = gen(21)
    vocab = (1 << 21) - 256
    h, w = small_multiples(g, 3, 8), small_multiples(g, vocab, 8)
    check_large(h.to(dtype), w.to(dtype), torch.tensor([vocab - 1, 0, 1000003]), dtype, "vocabulary 2^21 - 256")


def test_xent_more_rows_than_a_grid():
    """More rows than the gathering kernels' grids, in two pieces (with gradient) and 135 (without)."""
    g = gen(22)
    rows = 2200003
    h, w = small_multiples(g, rows, 8), small_multiples(g, 5, 8)
    check_large(h.to(BF16), w.to(BF16), torch.randint(0, 5, (rows,), generator=g), BF16, "2200003 rows")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_xent_of_rows_too_far_apart_to_read_in_place(dtype):
    """A stride of more than 2^21 elements: w is packed; with an odd one too."""
    g = gen(23)
    for stride in ((1 << 21) + 8, (1 << 21) + 3):
        far = torch.full((40 * stride,), math.nan, dtype=dtype, device=DEV).view(40, stride)
        h, w = small_multiples(g, 20, 24).to(dtype), small_multiples(g, 40, 24).to(dtype)
        t = torch.randint(0, 40, (20,), generator=g).to(DEV)
        far[:, :24] = w.to(DEV)
        outs = []
        for weight in (far[:, :24], w.to(DEV)):
            loss, dh, dw = torch.empty(20, device=DEV), torch.empty(20, 24, dtype=dtype, device=DEV), torch.empty(40, 24, device=DEV)
            A.adam_xent(h.to(DEV), weight, t, loss, dh=dh, dw=dw)
            outs.append((loss, dh, dw))
        assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("rows,n,k", [(40, 3, 1 << 21), (40, 8, 1 << 21), (40, 1 << 21, 33), (70, (1 << 21) - 5, 7)])
def test_wgrad_largest_sizes(rows, n, k):
    wgrad_case(rows, n, k, BF16, F32, "e4m3", seed=24)


def test_wgrad_of_rows_too_far_apart_to_read_in_place():
    wgrad_case(4, 8, 40, F16, F32, "e4m3", pad=1 << 21, seed=25)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name,lo,hi", [("silu", -88.7, -80.0), ("gelu", -10.06, -9.0)])
def test_glu_of_gates_whose_logistic_function_is_tiny(name, lo, hi, dtype):
    """exp(-q) up to the float range's end: 1 + exp(-q) beyond 2^126 has a reciprocal below the normal range, of at least
    21 bits.  Past the end, where the activation is below 3e-37 (silu) or 4e-38 (gelu), it may be 0."""
    x = torch.linspace(lo, hi, 992).view(31, 32).to(dtype)
    x = x.clamp(min=float(torch.tensor(lo).to(dtype)) if dtype == F32 else -88.5)
    h = torch.empty(31, 32, dtype=dtype, device=DEV)
    A.adam_glu_forward(x.to(DEV), torch.ones_like(x).to(DEV), h, name)
    a, _, _ = R.act(x.double(), name)
    within = a.abs() * (R.u(dtype) * 1.01 + R.act_error(x.double(), name) + 2.0 ** -21) + R.tiny(dtype)
    past = (x if name == "silu" else 2 * math.sqrt(2 / math.pi) * (x.double() + 0.044715 * x.double() ** 3)) < -88.7
    close(h.cpu(), a, torch.where(past, 3e-37, within), "h")


# ---------------------------------------------------------------------------
# Cross entropy of matrices beyond 32-bit offsets
# ---------------------------------------------------------------------------

def test_xent_with_a_weight_beyond_32_bit_offsets():
    """A weight of more than 2^31 elements, zero but for its last rows: the gradients there are as the formula's."""
    g = torch.Generator(device=DEV).manual_seed(30)
    rows, hidden, vocab, last = 6, 4096, 600003, 300
    assert vocab * hidden > 1 << 31
    w = torch.zeros(vocab, hidden, dtype=BF16, device=DEV)
    w[-last:].normal_(generator=g).mul_(0.08)
    h = torch.randn(rows, hidden, device=DEV, generator=g).to(BF16)
    t = torch.arange(vocab - rows, vocab, device=DEV)
    loss, dh = torch.empty(rows, device=DEV), torch.empty_like(h)
    dw = torch.full((vocab, hidden), 7.0, device=DEV)
    A.adam_xent(h, w, t, loss, dh=dh, dw=dw)
    tail = w[-last:].double().cpu()
    z = h.double().cpu() @ tail.t()
    lse = torch.logaddexp(torch.logsumexp(z, 1), torch.tensor(math.log(vocab - last), dtype=torch.float64))
    hot = torch.zeros(rows, last, dtype=torch.float64)
    hot[torch.arange(rows), last - rows + torch.arange(rows)] = 1
    p = torch.exp(z - lse[:, None])
    gr = p - hot
    dz = (hidden + 8) * 2.0 ** -23 * (h.double().cpu().abs() @ tail.abs().t()).amax(1)
    sums = 2.0 ** -16 + (vocab + 16) * 2.0 ** -24
    close(loss.cpu(), lse - (z * hot).sum(1), 2 * dz + sums + 2.0 ** -18, "loss")
    dg = p * ((2 * dz + sums + 2.0 ** -16 + 2.0 ** -11)[:, None]) + 2.0 ** -39 + gr.abs() * 1.01 * R.u(BF16) ** 2
    a = h.double().cpu().abs()
    close(dw[-last:].cpu(), gr.t() @ h.double().cpu(), dg.t() @ a + 2.0 ** -20 * (gr.abs().t() @ a), "dw")
    close(dh.cpu(), gr @ tail, dg @ tail.abs() + 2.0 ** -13 * (gr.abs() @ tail.abs()) + (gr @ tail).abs() * 1.01 * R.u(BF16), "dh")
    rest = torch.exp(-lse)[None, :] @ h.double().cpu()  # every other row of dw is the same
    bound = torch.exp(-lse)[None, :] * (2 * dz + sums + 2.0 ** -10) @ a + 2.0 ** -38 * a.sum(0)
    for at in (0, 524288, vocab - last - 1):  # 524288: byte offset 2^33 in dw, element 2^31
        close(dw[at: at + 1].cpu(), rest, bound, f"dw row {at}")


def test_xent_with_a_gradient_beyond_32_bit_offsets():
    """G of more than 2^31 elements held at once, against pieces of it.  The logits, lse and G do not depend on the pieces,
    so only the order of float sums and the outputs' rounding do."""
    g = torch.Generator(device=DEV).manual_seed(31)
    rows, hidden, vocab = 18432, 64, 131072
    assert rows * vocab > 1 << 31
    h = torch.randn(rows, hidden, device=DEV, generator=g).to(BF16)
    w = (torch.randn(vocab, hidden, device=DEV, generator=g) / 4).to(BF16)
    t = torch.randint(0, vocab, (rows,), device=DEV, generator=g)
    outs = []
    for piece in (rows, 4096):
        loss, dh, dw = torch.empty(rows, device=DEV), torch.empty_like(h), torch.empty(vocab, hidden, device=DEV)
        A.adam_xent(h, w, t, loss, dh=dh, dw=dw, piece_rows=piece)
        outs.append((loss, dh.float(), dw))
    (loss, dh, dw), (loss2, dh2, dw2) = outs
    assert torch.equal(loss, loss2)
    # a row's |G| add up to 2 at most, so dh's sum of vocab products is off by (vocab + 300) 2^-23 of 2 max |w| each time
    sums = 2 * (vocab + 300) * 2.0 ** -23 * 2 * float(w.abs().max())
    close(dh, dh2, sums + 2 * R.u(BF16) * 1.01 * dh2.abs(), "dh")
    # a column's |G|: 1 for each row of that target, and its probability in every row
    mass = torch.zeros(vocab, dtype=torch.float64, device=DEV)
    for r in range(0, rows, 1024):
        mass += torch.softmax(h[r: r + 1024].float() @ w.float().t(), 1).double().sum(0)
    mass += torch.bincount(t, minlength=vocab)
    close(dw, dw2, (2 * (rows + 300) * 2.0 ** -23 * 1.01 * float(h.abs().max()) * mass)[:, None].expand(-1, hidden), "dw")


# ---------------------------------------------------------------------------
# Graphs: what a replay reads anew
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [60, 700, 1500])  # both gathering paths, two values of G and one
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_xent_replayed_with_other_inputs(dtype, rows):
    """Captured without a workspace of the caller's, with weights; then replayed with other targets (another number of
    rows to compute), weights of other magnitudes and other loss scales, and eager calls between."""
    g = gen(40)
    hidden, vocab = 72, 900
    h, w = torch.randn(rows, hidden, generator=g).to(dtype).to(DEV), (torch.randn(vocab, hidden, generator=g) / 4).to(dtype).to(DEV)
    t, weight, scale = torch.zeros(rows, dtype=torch.int64, device=DEV), torch.ones(rows, device=DEV), torch.ones(1, device=DEV)

    def outputs():
        return torch.empty(rows, device=DEV), torch.empty_like(h), torch.empty(vocab, hidden, device=DEV)

    def call(out):
        A.adam_xent(h, w, t, out[0], weight=weight, dh=out[1], dw=out[2], d_loss_scale=scale)

    eager, graphed = outputs(), outputs()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(graphed)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(graphed)
    for replay, (ignored, magnitude) in enumerate([(0.0, 1.0), (0.5, 2.0 ** -20), (1.0, 1.0), (0.9, 2.0 ** 20), (0.0, 2.0 ** -7)]):
        new = torch.randint(0, vocab, (rows,), generator=g)
        new[torch.rand(rows, generator=g) < ignored] = -100
        t.copy_(new)
        weight.copy_((1 + torch.rand(rows, generator=g)) * magnitude)
        scale.fill_(0.5 / magnitude)
        call(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(bool(torch.isfinite(a).all()) and torch.equal(a, b) for a, b in zip(eager, graphed)), replay
        _ = torch.randn(4096, device=DEV).sum().item()


def test_backward_over_its_own_input():
    """dgate in dh's place: the same bits as in a buffer of its own."""
    g = gen(41)
    rows, cols = 37, 1003
    buf = [torch.empty(A.adam_act8_bytes(rows, cols), dtype=torch.uint8, device=DEV) for _ in range(2)]
    for b in buf:
        A.adam_act8_store(torch.randn(rows, cols, generator=g).to(DEV), b)
    for dtype in (BF16, F16, F32):
        dh = torch.randn(rows, cols, generator=g).to(dtype).to(DEV)
        dg, du, du2 = torch.empty_like(dh), torch.empty_like(dh), torch.empty_like(dh)
        A.adam_glu_backward(dh, *buf, dg, du, "gelu")
        A.adam_glu_backward(dh, *buf, dh, du2, "gelu")
        assert torch.equal(dh, dg) and torch.equal(du, du2)


# ---------------------------------------------------------------------------
# Weight gradient in fp16: activations at the ends of fp16's range
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_wgrad_of_the_largest_and_smallest_fp16_activations(fmt):
    """Every fp16 magnitude from 2^-20 to 65504 has a finite 8-bit value of at most 4 significant bits, which the product
    takes exactly: dy of a unit matrix gives the decoded checkpoint."""
    x = torch.arange(0x0010, 0x7C00, dtype=torch.int32).to(torch.int16).view(F16)  # 16 subnormal steps (2^-20) to 65504
    x = torch.cat([x, -x])
    x = torch.nn.functional.pad(x, (0, -len(x) % 1024)).view(-1, 1024)
    rows = x.shape[0]
    buf = torch.empty(A.adam_act8_bytes(rows, 1024), dtype=torch.uint8, device=DEV)
    A.adam_act8_store(x.to(DEV), buf, fmt)
    want = R.decode(buf, rows, 1024, fmt)
    assert float(want.abs().max()) == 65536 and bool(torch.isfinite(want).all())
    dy, dw = torch.eye(rows, dtype=F16, device=DEV), torch.empty(rows, 1024, device=DEV)
    A.adam_act8_wgrad(dy, buf, dw, fmt)
    assert torch.equal(dw.cpu().double(), want)
    # an infinite activation stays one in e5m2 and is NaN in e4m3, in its column alone
    x[5, 7] = -math.inf
    A.adam_act8_store(x.to(DEV), buf, fmt)
    A.adam_act8_wgrad(dy, buf, dw, fmt)
    bad = ~torch.isfinite(dw.cpu())
    assert bool(bad[5, 7]) and bool(bad[:, 7].all()) and int(bad.sum()) == rows  # 0 times it is NaN too
    assert fmt == "e4m3" or float(dw[5, 7]) == -math.inf
