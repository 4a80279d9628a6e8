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


# ---------------------------------------------------------------------------
# Gradients against differences, streams, graphs, sizes, a run of them together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["plain", "cap", "bias"])
def test_attention_gradient_against_differences(kind):
    """The derivative of the sum of dout o along a direction, by central differences of the 64-bit forward pass."""
    slopes = torch.tensor([0.1, 0.02]) if kind == "bias" else None
    c = Case(90, 2, 1, 32, BF16, offsets=[0, 33, 90], cap=4.0 if kind == "cap" else 0.0, slopes=slopes, seed=20)
    got = c.run()
    g = gen(21)
    h = 2.0 ** -10
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        x = getattr(c, name)
        step = randn(g, *x.shape).double()

        def value(sign):
            args = dict(q=c.q.double(), k=c.k.double(), v=c.v.double())
            args[name] = args[name] + sign * h * step
            total = 0.0
            for head in range(2):
                z = c.scale * args["q"][:, head] @ args["k"][:, 0].t()
                if c.cap:
                    z = c.cap * torch.tanh(z / c.cap)
                if slopes is not None:
                    z = z - slopes[head].double() * (torch.arange(90)[:, None] - torch.arange(90)[None, :]).abs()
                p = torch.softmax(torch.where(c.see, z, -math.inf), 1)
                total = total + (c.dout[:, head].double() * (p @ args["v"][:, 0])).sum()
            return float(total)

        want = (value(1) - value(-1)) / (2 * h)
        have = float((got[grad].double() * step).sum())
        # each entry off by at most 2^-6 of itself and of the root mean square (three roundings of 2^-8, a few of the
        # terms of its sums as large as it), signs at random: 6 standard deviations; the difference's h^2 term is below it
        size = got[grad].double()
        bound = 6 * 2.0 ** -6 * float(((size ** 2 + (size ** 2).mean()) * step ** 2).sum().sqrt())
        assert abs(have - want) <= bound, (name, have, want, bound)


def test_same_bits_each_time_and_on_another_stream():
    c = Case(300, 4, 2, 64, BF16, offsets=[0, 120, 300], seed=22)
    first = c.run()
    stream = torch.cuda.Stream()
    for _ in range(2):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            again = c.run()
        torch.cuda.current_stream().wait_stream(stream)
        assert all(torch.equal(first[n], again[n]) for n in first)


def test_stream_argument_and_workspaces():
    """Two calls at once, each with its stream and workspace."""
    g = gen(23)
    q, k, v, d = (randn(g, 400, 2, 64).to(BF16).to(DEV) for _ in range(4))
    how = dict(q=q, k=k, v=v)
    o, lse = torch.empty_like(q), torch.empty(2, 400, device=DEV)
    plan = A.adam_attn_plan(q, k, v, o, lse)
    assert set(plan) == {"forward_bytes", "backward_bytes"}
    A.adam_attn_forward(q, k, v, o, lse)
    want = [torch.empty_like(q) for _ in range(3)]
    A.adam_attn_backward(d, q, k, v, o, lse, *want)
    torch.cuda.synchronize()
    runs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        ws = torch.empty(plan["backward_bytes"], dtype=torch.uint8, device=DEV)
        outs = [torch.zeros_like(q) for _ in range(4)] + [torch.zeros_like(lse)]
        torch.cuda.synchronize()
        A.adam_attn_forward(q, k, v, outs[3], outs[4], workspace=ws, stream=s)
        A.adam_attn_backward(d, q, k, v, outs[3], outs[4], *outs[:3], workspace=ws, stream=s)
        runs.append(outs)
    torch.cuda.synchronize()
    for outs in runs:
        assert torch.equal(outs[3], o) and all(torch.equal(a, b) for a, b in zip(outs, want))
    with pytest.raises(ValueError, match="needed"):
        A.adam_attn_forward(**how, o=o, workspace=torch.empty(1, dtype=torch.uint8, device=DEV))


def test_step_from_tokens_to_update_in_a_graph():
    """A tied model of one attention layer: lookup, attention, cross entropy, their gradients into one weight, the norm
    and the step; recorded once and replayed with other tokens, documents and gradients, against eager calls."""
    rows, vocab, heads, dim = 200, 500, 4, 32
    hidden = heads * dim
    g = gen(24)
    w0 = randn(g, vocab, hidden) * 0.3

    def build():
        s = dict(p=w0.clone().to(DEV), m=torch.zeros(vocab, hidden, device=DEV), v=torch.zeros(vocab, hidden, device=DEV),
                 g=torch.zeros(vocab, hidden, device=DEV), w=w0.to(BF16).to(DEV))
        s["tl"] = A.adam_tl_build([dict(p=s["p"].view(-1), m=s["m"].view(-1), v=s["v"].view(-1), g=s["g"].view(-1),
                                        p_out=s["w"].view(-1))], A.make_desc(g="f32", p_out="bf16"))
        s["token"] = torch.zeros(rows, dtype=torch.int64, device=DEV)
        s["target"] = torch.zeros(rows, dtype=torch.int64, device=DEV)
        s["offsets"] = torch.zeros(4, dtype=torch.int32, device=DEV)
        for n in ("x", "dx"):
            s[n] = torch.zeros(rows, 3 * hidden, dtype=BF16, device=DEV)
        for n in ("o", "do", "y", "dy"):
            s[n] = torch.zeros(rows, hidden, dtype=BF16, device=DEV)
        s["lse"], s["loss"] = torch.zeros(heads, rows, device=DEV), torch.zeros(rows, device=DEV)
        s["sumsq"] = torch.zeros(1, dtype=torch.float64, device=DEV)
        s["lr"], s["step"] = torch.tensor([1e-2], device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        s["scale"], s["noop"] = torch.ones(1, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        s["ws"] = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
        return s

    def step(s):
        hp = A.AdamHParams(0.9, 0.95, 1e-8, 0.1, 1, 1)
        A.adam_embed_forward(s["token"], s["w"], s["y"], scale=4.0)
        for i in range(3):
            s["x"][:, i * hidden: (i + 1) * hidden].copy_(s["y"])
        x, dx = s["x"].view(rows, 3 * heads, dim), s["dx"].view(rows, 3 * heads, dim)
        q, k, v = (x[:, i * heads: (i + 1) * heads] for i in range(3))
        o = s["o"].view(rows, heads, dim)
        A.adam_attn_forward(q, k, v, o, s["lse"], doc_offsets=s["offsets"], workspace=s["ws"])
        A.adam_xent(s["o"], s["w"], s["target"], s["loss"], dh=s["do"], dw=s["g"], workspace=s["ws"])
        A.adam_attn_backward(s["do"].view(rows, heads, dim), q, k, v, o, s["lse"], *(dx[:, i * heads: (i + 1) * heads]
                             for i in range(3)), doc_offsets=s["offsets"], workspace=s["ws"])
        torch.add(s["dx"][:, :hidden], s["dx"][:, hidden: 2 * hidden], out=s["dy"])
        s["dy"].add_(s["dx"][:, 2 * hidden:])
        A.adam_embed_backward(s["token"], s["dy"], s["g"], scale=4.0, accumulate=True, workspace=s["ws"])
        A.adam_grad_sumsq(s["tl"], s["sumsq"])
        s["scale"].fill_(1.0)
        A.adam_clip_grad_scale(s["sumsq"], s["scale"], 1.0, d_noop=s["noop"])
        A.adam_step_capturable(s["tl"], hp, s["lr"], s["step"], s["scale"], s["noop"])

    def feed(s, k):
        r = gen(100 + k)
        s["token"].copy_(torch.randint(0, vocab, (rows,), generator=r))
        s["target"].copy_(torch.randint(0, vocab, (rows,), generator=r))
        s["offsets"].copy_(torch.tensor([0, 30 + 17 * k, 120 + k, rows], dtype=torch.int32))

    eager, recorded = build(), build()
    feed(recorded, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = build()
        feed(warm, 0)
        step(warm)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(recorded)
    losses = []
    for k in range(4):
        feed(eager, k)
        feed(recorded, k)
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for n in ("o", "lse", "loss", "do", "dx", "g", "p", "m", "v", "w", "step", "sumsq"):
            assert torch.equal(eager[n], recorded[n]), (k, n)
        losses.append(float(eager["loss"].mean()))
    assert int(eager["step"]) == 4 and all(math.isfinite(x) for x in losses)
    for s in (eager, recorded, warm):
        s["tl"].destroy()


def test_replay_of_the_careful_kernels():
    """A NaN that comes in a later replay is kept to the rows that see it, and is gone in the next one."""
    g = gen(25)
    q, k, v, d = (randn(g, 200, 2, 64).to(BF16).to(DEV) for _ in range(4))
    o, lse = torch.empty_like(q), torch.empty(2, 200, device=DEV)
    grads = [torch.empty_like(q) for _ in range(3)]
    plan = A.adam_attn_plan(q, k, v, o, lse)
    ws = torch.empty(plan["backward_bytes"], dtype=torch.uint8, device=DEV)

    def run():
        A.adam_attn_forward(q, k, v, o, lse, workspace=ws)
        A.adam_attn_backward(d, q, k, v, o, lse, *grads, workspace=ws)

    run()
    torch.cuda.synchronize()
    want = [x.clone() for x in (o, *grads)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    keep = v[150].clone()
    for k_ in range(3):
        v[150] = math.nan
        graph.replay()
        torch.cuda.synchronize()
        assert bool(torch.isfinite(o[:150]).all()) and not bool(torch.isfinite(o[150:]).any())
        assert bool(torch.isfinite(grads[0][:150]).all()) and not bool(torch.isfinite(grads[0][150:]).any())
        v[150] = keep
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (o, *grads)))


def test_attention_many_documents_equals_each_alone():
    """4000 rows of documents of 1 to 700 tokens, 8 heads on 2 of 128: every document as it is by itself."""
    g = gen(26)
    rows = 4000
    offsets = [0, 1, 3, 10, 74, 202, 203, 333, 845, 1545, 1546, 1610, 2310, 2310, 2900, 3599, 3998]
    q, d = (randn(g, rows, 8, 128).to(BF16).to(DEV) for _ in range(2))
    k, v = (randn(g, rows, 2, 128).to(BF16).to(DEV) for _ in range(2))
    o, lse, dq, dk, dv = (torch.zeros_like(q), torch.zeros(8, rows, device=DEV), torch.zeros_like(q), torch.zeros_like(k),
                          torch.zeros_like(v))
    how = dict(doc_offsets=torch.tensor(offsets, dtype=torch.int32, device=DEV))
    A.adam_attn_forward(q, k, v, o, lse, **how)
    A.adam_attn_backward(d, q, k, v, o, lse, dq, dk, dv, **how)
    for a, b in zip(offsets, offsets[1:]):
        if a == b:
            continue
        s = slice(a, b)
        o1, lse1 = torch.zeros_like(q[s]), torch.zeros(8, b - a, device=DEV)
        g1 = [torch.zeros_like(x[s]) for x in (q, k, v)]
        A.adam_attn_forward(q[s], k[s], v[s], o1, lse1)
        A.adam_attn_backward(d[s], q[s], k[s], v[s], o1, lse1, *g1)
        # the tiles lie elsewhere: other orders of the sums, other roundings of weights (2^-8 each, 8 and 4 of their
        # standard deviations for results whose terms have signs at random)
        for x, y in ((o[s], o1), (dq[s], g1[0]), (dk[s], g1[1]), (dv[s], g1[2])):
            x, y = x.double(), y.double()
            assert float((x - y).norm()) <= 4 * 2.0 ** -8 * float(y.norm()) + 1e-2 * 2.0 ** -8 * float(d.double().norm()) / rows
        assert float((lse[:, s] - lse1).abs().max()) <= 1e-4
    assert bool((o[3998:] == 0).all()) and bool((dq[3998:] == 0).all()) and bool((dk[3998:] == 0).all())


def test_attention_beyond_32_bit_offsets():
    """Rows that begin more than 2^31 elements into their tensors: the last ones are what they are alone."""
    rows, stride = 1100, 1 << 21
    big = torch.empty(rows, stride, dtype=BF16, device=DEV)
    assert big.numel() > 1 << 31
    g = gen(27)
    view = big.as_strided((rows, 4, 64), (stride, 64, 1))
    view.copy_(randn(g, rows, 4, 64).to(BF16))
    q, k, v = view[:, :2], view[:, 2:3], view[:, 3:4]
    o, lse = big.as_strided((rows, 2, 64), (stride, 64, 1), 1024), torch.empty(2, rows, device=DEV)
    dense = [x.contiguous() for x in (q, k, v)]
    want, want_lse = torch.empty_like(dense[0]), torch.empty_like(lse)
    A.adam_attn_forward(q, k, v, o, lse, window=100)
    A.adam_attn_forward(*dense, want, want_lse, window=100)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_embedding_beyond_32_bit_offsets():
    """A weight of more than 2^31 elements: its last rows are read, and their gradients written, as in a small one."""
    vocab, hidden = 300000, 8192
    g = gen(28)
    w = torch.zeros(vocab, hidden, dtype=BF16, device=DEV)
    tail = randn(g, 7, hidden).to(BF16).to(DEV)
    w[-7:] = tail
    t = torch.tensor([6, 0, 3, 3, 6, 5]).to(DEV)
    y, small = torch.empty(6, hidden, dtype=BF16, device=DEV), torch.empty(6, hidden, dtype=BF16, device=DEV)
    A.adam_embed_forward(t + vocab - 7, w, y)
    A.adam_embed_forward(t, tail, small)
    assert torch.equal(y, small)
    w.fill_(3.0)
    dw = torch.empty(7, hidden, dtype=BF16, device=DEV)
    A.adam_embed_backward(t + vocab - 7, y, w)
    A.adam_embed_backward(t, y, dw)
    assert torch.equal(w[-7:], dw) and int((w[:-7] != 0).sum()) == 0
