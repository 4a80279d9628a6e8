"""The embedding and attention over packed documents on the GPU against plain
64-bit implementations (tests/sequence_reference.py), within bounds derived from
the roundings they make: types, odd sizes, strides, masks, documents of every
length, the gradients against differences too, streams, graphs, and a run of the
operators from tokens to the update."""
import math

import pytest
import torch

import adamw_optimizer_step_tensor_amd as A
import sequence_reference as S
import train_reference as R
from test_gpu_train import DEV, BF16, F16, F32, Guarded, close, gen, on_gpu, randn

pytestmark = pytest.mark.gpu

TYPES = [BF16, F16, F32]
HALF = [BF16, F16]


# ---------------------------------------------------------------------------
# Embedding
# ---------------------------------------------------------------------------

def tokens(g, rows, vocab, kind):
    if kind == "same":
        return torch.full((rows,), vocab - 1)
    t = torch.randint(0, vocab, (rows,), generator=g)
    if kind == "skewed":
        t = torch.where(torch.rand(rows, generator=g) < 0.6, t % min(vocab, 3), t)
    t[torch.rand(rows, generator=g) < 0.1] = -100
    return t


@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (3, 1)])
@pytest.mark.parametrize("y_type", TYPES)
@pytest.mark.parametrize("w_type", TYPES)
def test_embed_forward(w_type, y_type, pad, offset):
    for k, (rows, vocab, hidden) in enumerate([(1, 1, 1), (3, 7, 5), (17, 100, 8), (130, 999, 257), (7, 30, 1000)]):
        g = gen(k)
        t = tokens(g, rows, vocab, "any")
        w = randn(g, vocab, hidden).to(w_type)
        if rows > 5:
            t[2], t[4] = -1, vocab
        for scale in (1.0, 32.0, -0.3):
            y = Guarded(rows, hidden, y_type, pad, offset)
            A.adam_embed_forward(t.to(DEV), on_gpu(w, pad, offset), y.view, scale=scale)
            got, want = y.check().double(), S.embed(t, w, torch.tensor(scale).double(), -100)
            assert torch.equal(got.isnan(), want.isnan())
            ok = ~want.isnan()
            # one rounding to float, one to the type
            err = want.abs() * (R.u(y_type) + 2.0 ** -24) * 1.01 + R.tiny(y_type)
            assert bool(((got - want).abs() <= err)[ok].all()), (rows, vocab, hidden, scale)
            assert bool((got[t == -100] == 0).all())


BACKWARD = [(1, 1, 1, "any"), (5, 3, 7, "any"), (16, 40, 8, "any"), (17, 1, 513, "same"), (64, 500, 1001, "skewed"),
            (333, 50, 520, "skewed"), (1000, 70000, 24, "any"), (2049, 20, 40, "skewed"), (16385, 300, 16, "skewed"),
            (20000, 70000, 8, "any"), (40000, 5, 8, "same"), (16384, 131072, 4, "any")]


@pytest.mark.parametrize("rows,vocab,hidden,kind", BACKWARD)
@pytest.mark.parametrize("dy_type,dw_type", [(BF16, F32), (BF16, BF16), (F16, F16), (F32, F32), (F32, BF16), (F16, F32)])
def test_embed_backward(dy_type, dw_type, rows, vocab, hidden, kind):
    g = gen(rows + hidden)
    t = tokens(g, rows, vocab, kind)
    if rows > 5:
        t[1], t[3] = -7, vocab
    dy = randn(g, rows, hidden).to(dy_type)
    dy[(t < 0) | (t >= vocab)] = math.nan  # adds nothing
    old = randn(g, vocab, hidden).to(dw_type)
    for accumulate, pad, offset, scale in ((False, 0, 0, 1.0), (True, 5, 3, 32.0)):
        want, size, count = S.embed_gradient(t, dy, vocab, scale, -100)
        dw = Guarded(vocab, hidden, dw_type, pad, offset)
        dw.view.copy_(old)
        A.adam_embed_backward(t.to(DEV), on_gpu(dy, pad, offset), dw.view, scale=scale, accumulate=accumulate)
        got = dw.check()
        if accumulate:
            assert torch.equal(got[count[:, 0] == 0], old[count[:, 0] == 0])
            want = want + old.double()
            size = size + old.double().abs()
        else:
            assert bool((got[count[:, 0] == 0] == 0).all())
        # float additions of count values and the scaling, then one rounding
        bound = size * (count + 2) * 2.0 ** -24 * 1.01 + want.abs() * 1.01 * R.u(dw_type) + R.tiny(dw_type)
        close(got, want, bound, f"dw accumulate={accumulate}")


def test_embed_backward_is_reproducible_and_ordered():
    """The same bits each time, and from one path of sorting to the other."""
    g = gen(3)
    t = tokens(g, 16384, 1000, "skewed").to(DEV)
    dy = randn(g, 16384, 64).to(DEV)
    first = torch.empty(1000, 64, device=DEV)
    A.adam_embed_backward(t, dy, first)
    for _ in range(3):
        again = torch.full_like(first, 9.0)
        A.adam_embed_backward(t, dy, again)
        assert torch.equal(first, again)
    # one more row, which adds nothing: the list is sorted in passes, its blocks are the same
    more = torch.empty_like(first)
    A.adam_embed_backward(torch.cat([t, t.new_tensor([-100])]), torch.cat([dy, dy[:1]]), more)
    assert torch.equal(first, more)


def test_embed_empty():
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    w = torch.ones(5, 8, device=DEV)
    A.adam_embed_forward(none, w, torch.empty(0, 8, device=DEV))
    dw = torch.ones(5, 8, device=DEV)
    A.adam_embed_backward(none, torch.empty(0, 8, device=DEV), dw, accumulate=True)
    assert bool((dw == 1).all())
    A.adam_embed_backward(none, torch.empty(0, 8, device=DEV), dw)
    assert bool((dw == 0).all())
    A.adam_embed_forward(torch.zeros(3, dtype=torch.int64, device=DEV), w[:, :0], torch.empty(3, 0, device=DEV))


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

class Case:
    """Inputs of a call as views of one fused buffer, and its results."""

    def __init__(self, rows, heads, kv, dim, dtype, offsets=None, prefix=None, causal=True, window=0, scale=None, cap=0.0,
                 slopes=None, seed=0, spread=1.3, layout="fused", d_scale=1.0):
        g = gen(seed)
        self.rows, self.heads, self.kv, self.dim, self.dtype, self.layout = rows, heads, kv, dim, dtype, layout
        self.q, self.k = ((spread * randn(g, rows, n, dim)).to(dtype) for n in (heads, kv))
        self.v = randn(g, rows, kv, dim).to(dtype)
        self.dout = (d_scale * randn(g, rows, heads, dim)).to(dtype)
        self.slopes = slopes
        self.offsets, self.prefix = offsets, prefix
        self.scale = dim ** -0.5 if scale is None else scale
        self.how = dict(causal=causal, window=window, scale=scale, softcap=cap)
        for name, x in (("doc_offsets", offsets), ("prefix", prefix)):
            self.how[name] = None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)
        self.how["slopes"] = None if slopes is None else slopes.to(DEV)
        self.see = S.visible(rows, offsets or [0, rows], prefix, causal, window)
        self.cap = cap

    def place(self, x):
        """x on the GPU: a part of wider rows, rows one element longer, or each head's rows in a block."""
        if self.layout == "fused":
            buf = torch.full((self.rows, x.shape[1] + 2, self.dim), math.nan, dtype=self.dtype, device=DEV)
            view = buf[:, 1:-1]
        elif self.layout == "odd":
            buf = torch.full((self.rows, x.shape[1], self.dim + 1), math.nan, dtype=self.dtype, device=DEV)
            view = buf[:, :, 1:]
        else:
            buf = torch.full((x.shape[1], self.rows, self.dim), math.nan, dtype=self.dtype, device=DEV)
            view = buf.transpose(0, 1)
        view.copy_(x)
        return buf, view

    def run(self, gradient=True):
        q, k, v, dout = (self.place(x)[1] for x in (self.q, self.k, self.v, self.dout))
        outs = {}
        for name, like in (("o", self.q), ("dq", self.q), ("dk", self.k), ("dv", self.v)):
            outs[name] = self.place(torch.full_like(like, 7.0))
        lse = torch.full((self.heads, self.rows), 7.0, device=DEV)
        A.adam_attn_forward(q, k, v, outs["o"][1], lse, **self.how)
        if gradient:
            A.adam_attn_backward(dout, q, k, v, outs["o"][1], lse, outs["dq"][1], outs["dk"][1], outs["dv"][1], **self.how)
        got = dict(lse=lse.cpu())
        for name, (buf, view) in outs.items():
            got[name] = view.cpu()
            view.fill_(math.nan)
            assert bool(buf.isnan().all()), f"{name}: wrote outside"
        return got

    def check(self, gradient=True):
        got = self.run(gradient)
        want, bound = S.attention(self.q, self.k, self.v, self.see, self.scale, self.cap, self.slopes,
                                  self.dout if gradient else None)
        inside, seen = self.see.any(1), self.see.any(0)
        reached = self.reached()
        for name in want:
            x, w, b = got[name], want[name], bound[name]
            at = inside if name in ("o", "dq", "lse") else seen
            if name == "lse":
                x, w, b = x.t(), w.t(), b.t()
            fine = ~reached[name][at]
            if name != "lse":
                # a value near the type's largest (fp16: from 65520 on) may round to infinity
                most = torch.finfo(self.dtype).max
                top = fine & (w[at].abs() + b[at] >= most)
                assert bool((x[at][top].double().abs() >= (w[at][top].abs() - b[at][top]).clamp(max=most)).all()), name
                assert torch.equal(x[at][top].signbit(), w[at][top].signbit()), name
                fine &= ~top
            close(x[at][fine], w[at][fine], b[at][fine], name)
            assert bool((x[~at] == 7.0).all()), f"{name}: wrote rows of no document"
        return got, reached

    def reached(self):
        """The elements of each result that an infinity or a NaN of the inputs reaches by the formulas."""
        group = self.heads // self.kv
        see = self.see.double()

        def by_key(x):  # any seen key
            return (torch.einsum("ij,j...->i...", see, x.double()) > 0).repeat_interleave(group, 1)

        def by_query(x):  # any query that sees the key, of any head of the group
            x = torch.einsum("ij,i...->j...", see, x.double()) > 0
            return x.view(self.rows, self.kv, group, *x.shape[2:]).any(2)

        q, k, v, d = (~torch.isfinite(x) for x in (self.q, self.k, self.v, self.dout))
        weight = q.any(2) | by_key(k.any(2))  # rows x heads: the row's weights
        row = weight | d.any(2) | by_key(v.any(2))
        return dict(lse=weight, o=weight[..., None] | by_key(v), dq=row[..., None].expand(q.shape),
                    dk=by_query(row)[..., None].expand(k.shape), dv=by_query(weight[..., None] | d))


SIZES = [(1, 1, 1, 64), (2, 2, 1, 8), (5, 3, 3, 17), (31, 4, 2, 64), (33, 2, 2, 72), (64, 8, 8, 128), (65, 8, 2, 80),
         (127, 2, 1, 1), (129, 16, 4, 128), (200, 1, 1, 256), (257, 2, 1, 136), (300, 3, 1, 33), (270, 2, 2, 199)]


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("rows,heads,kv,dim", SIZES)
def test_attention_sizes(dtype, rows, heads, kv, dim):
    for causal in (True, False):
        Case(rows, heads, kv, dim, dtype, causal=causal, seed=rows).check()


@pytest.mark.parametrize("layout", ["fused", "odd", "heads"])
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("dim", [64, 128, 96])
def test_attention_layouts(dtype, dim, layout):
    Case(150, 4, 2, dim, dtype, offsets=[0, 40, 150], layout=layout, seed=dim).check()


DOCUMENTS = [[0, 300], [0, 0, 300, 300], [0, 1, 2, 3, 300], [0, 128, 256, 300], [0, 127, 129, 290], [10, 20, 20, 200],
             list(range(0, 301, 3)), [5, 6], [299, 300], [0, 64, 64, 65, 192]]


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("offsets", DOCUMENTS)
def test_attention_documents(dtype, offsets):
    docs = len(offsets) - 1
    lengths = [b - a for a, b in zip(offsets, offsets[1:])]
    Case(300, 2, 1, 64, dtype, offsets=offsets, seed=1).check()
    Case(300, 2, 1, 64, dtype, offsets=offsets, causal=False, seed=2).check()
    Case(300, 2, 1, 64, dtype, offsets=offsets, prefix=[(7 * d) % 50 for d in range(docs)], seed=3).check()
    Case(300, 2, 1, 64, dtype, offsets=offsets, prefix=[n + 5 for n in lengths], seed=4).check()
    for window in (1, 2, 31, 64, 100, 299, 300, 1000):
        Case(300, 2, 1, 64, dtype, offsets=offsets, window=window, seed=5).check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", HALF)
def test_attention_cap_and_bias(dtype, dim):
    offsets = [0, 100, 131, 260]
    slopes = torch.tensor([0.5, 0.0, 0.03, -0.02])
    Case(260, 4, 2, dim, dtype, offsets=offsets, cap=5.0, seed=1).check()
    Case(260, 4, 2, dim, dtype, offsets=offsets, cap=50.0, spread=4.0, seed=2).check()
    Case(260, 4, 2, dim, dtype, offsets=offsets, slopes=slopes, seed=3).check()
    Case(260, 4, 2, dim, dtype, offsets=offsets, slopes=slopes, causal=False, seed=4).check()
    Case(260, 4, 2, dim, dtype, offsets=offsets, slopes=slopes, cap=30.0, prefix=[20, 3, 60], seed=5).check()
    Case(260, 4, 2, dim, dtype, offsets=offsets, slopes=slopes, cap=30.0, window=40, scale=0.3, seed=6).check()


@pytest.mark.parametrize("dtype", HALF)
def test_attention_longer(dtype):
    """Rows that see more keys than a first walk takes, and several tiles of them."""
    Case(1100, 2, 1, 64, dtype, offsets=[0, 900, 1100], seed=7).check()
    Case(700, 2, 2, 128, dtype, causal=False, seed=8).check()


def test_attention_forward_alone():
    c = Case(200, 2, 1, 64, BF16, seed=9)
    q, k, v = (x.to(DEV) for x in (c.q, c.k, c.v))
    o, same = torch.empty_like(q), torch.empty_like(q)
    A.adam_attn_forward(q, k, v, o)
    A.adam_attn_forward(q, k, v, same, torch.empty(2, 200, device=DEV))
    assert torch.equal(o, same)
    c.check(gradient=False)


@pytest.mark.parametrize("spread", [30.0, 1e-3])
@pytest.mark.parametrize("dtype", HALF)
def test_attention_large_and_small_scores(dtype, spread):
    """Scores of thousands: the bounds grow with them, the results stay finite."""
    Case(150, 2, 1, 64, dtype, spread=spread, seed=10).check()


@pytest.mark.parametrize("d_scale", [1e-7, 1e-4, 1e3, 2e4])
def test_attention_fp16_gradients_of_any_size(d_scale):
    """Upstream gradients near the ends of fp16: each gradient is what its own value rounds to."""
    Case(150, 2, 1, 64, F16, d_scale=d_scale, spread=0.5, seed=11).check()


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["q", "k", "v", "dout"])
@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (F16, 64), (BF16, 128), (BF16, 256), (F16, 200)])
def test_attention_hidden_infinities_and_nan(dtype, dim, which, value):
    """One reaches the rows that see it, by the formula, and no others: neither of its own document's earlier rows nor
    of the neighbours' in the same tile."""
    offsets = [0, 60, 61, 150, 200]
    for rows, causal, prefix in (([70], True, None), ([3, 59, 60, 149], True, None), ([62, 140], True, [5, 1, 20, 0]),
                                 ([100], False, None)):
        c = Case(200, 4, 2, dim, dtype, offsets=offsets, causal=causal, prefix=prefix, seed=12)
        for n, i in enumerate(rows):
            getattr(c, which)[i, n % 2, (7 * i) % dim] = value
        got, reached = c.check()
        if math.isnan(value):
            for name, at in reached.items():
                x = got[name].t() if name == "lse" else got[name]
                assert not bool(torch.isfinite(x[at]).any()), name
        assert 0 < int(reached["dq"].sum()) < reached["dq"].numel()


def test_attention_rows_of_no_document_may_hold_anything():
    c = Case(200, 2, 2, 64, BF16, offsets=[20, 90, 150], seed=13)
    for x in (c.q, c.k, c.v, c.dout):
        x[:20], x[150:] = math.nan, math.inf
    c.check()
