"""The embedding's and attention's C ABI on the CPU: workspaces follow the header,
and every refusal it names returns its status before anything touches a device."""
import ctypes
import math

import pytest

import adamw_optimizer_step_tensor_amd as A
from adamw_optimizer_step_tensor_amd import train as TR

BASE = 1 << 40  # fake, well-separated device addresses: refusals never touch them
GAP = 1 << 42
F32, BF16, F16 = A.DT_F32, A.DT_BF16, A.DT_F16
OK, EINVAL, EDTYPE = A.ADAM_OK, A.ADAM_EINVAL, A.ADAM_EDTYPE


def at(k, offset=0):
    return BASE + k * GAP + offset


FWD = dict(token=at(0), rows=10, w=at(1), wt=BF16, vocab=100, hidden=64, ws=64, scale=1.0, ignore=-100, y=at(2), yt=BF16,
           ys=64)


def forward(**kw):
    a = {**FWD, **kw}
    return TR.lib().adam_embed_forward(a["token"], a["rows"], a["w"], a["wt"], a["vocab"], a["hidden"], a["ws"], a["scale"],
                                       a["ignore"], a["y"], a["yt"], a["ys"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(wt=9), EINVAL), (dict(yt=-1), EINVAL), (dict(wt=A.DT_NONE), EDTYPE), (dict(yt=A.DT_NONE), EDTYPE),
    (dict(rows=-1), EINVAL), (dict(rows=(1 << 30) + 1), EINVAL), (dict(vocab=-1), EINVAL), (dict(vocab=1 << 31), EINVAL),
    (dict(hidden=-1), EINVAL), (dict(hidden=(1 << 30) + 1, ws=1 << 30, ys=1 << 30), EINVAL), (dict(ws=63), EINVAL),
    (dict(ys=63), EINVAL), (dict(scale=math.nan), EINVAL), (dict(scale=math.inf), EINVAL), (dict(token=None), EINVAL),
    (dict(w=None), EINVAL), (dict(y=None), EINVAL), (dict(vocab=0), EINVAL), (dict(token=at(0, 4)), EINVAL),
    (dict(w=at(1, 1)), EINVAL), (dict(y=at(2, 1)), EINVAL), (dict(wt=F32, w=at(1, 2)), EINVAL), (dict(y=at(1)), EINVAL),
    (dict(y=at(0)), EINVAL), (dict(y=at(1, 99 * 128)), EINVAL),
])
def test_embed_forward_refusals(kw, want):
    assert forward(**kw) == want


BWD = dict(token=at(0), rows=10, dy=at(1), gt=BF16, gs=64, scale=1.0, ignore=-100, dw=at(2), ot=F32, vocab=100, hidden=64,
           os=64, acc=0, wsp=at(3), size=1 << 30)


def backward(**kw):
    a = {**BWD, **kw}
    return TR.lib().adam_embed_backward(a["token"], a["rows"], a["dy"], a["gt"], a["gs"], a["scale"], a["ignore"], a["dw"],
                                        a["ot"], a["vocab"], a["hidden"], a["os"], a["acc"], a["wsp"], a["size"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(gt=9), EINVAL), (dict(ot=-1), EINVAL), (dict(gt=A.DT_NONE), EDTYPE), (dict(ot=A.DT_NONE), EDTYPE),
    (dict(acc=2), EINVAL), (dict(rows=-1), EINVAL), (dict(rows=(1 << 30) + 1), EINVAL), (dict(vocab=1 << 31), EINVAL),
    (dict(hidden=(1 << 30) + 1, gs=1 << 30, os=1 << 30), EINVAL), (dict(gs=63), EINVAL), (dict(os=63), EINVAL),
    (dict(scale=math.nan), EINVAL), (dict(token=None), EINVAL), (dict(dy=None), EINVAL), (dict(dw=None), EINVAL),
    (dict(vocab=0), EINVAL), (dict(token=at(0, 4)), EINVAL), (dict(dy=at(1, 1)), EINVAL), (dict(dw=at(2, 2)), EINVAL),
    (dict(wsp=None), EINVAL), (dict(wsp=at(3, 16)), EINVAL), (dict(size=100), EINVAL), (dict(dw=at(1)), EINVAL),
    (dict(dw=at(0)), EINVAL), (dict(wsp=at(1)), EINVAL), (dict(wsp=at(0)), EINVAL), (dict(wsp=at(2)), EINVAL),
])
def test_embed_backward_refusals(kw, want):
    assert backward(**kw) == want


def test_embed_without_rows_or_columns():
    assert forward(rows=0, token=None, y=None) == OK
    assert forward(hidden=0, ws=0, ys=0, w=None, y=None) == OK
    assert backward(rows=0, token=None, dy=None, acc=1, wsp=None, size=0) == OK
    assert backward(hidden=0, gs=0, os=0, dw=None) == OK
    assert backward(rows=0, vocab=0, dw=None, wsp=None, size=0) == OK


def test_embed_workspace():
    assert A.adam_embed_backward_workspace(0, 100, 64) == 0
    assert A.adam_embed_backward_workspace(10, 0, 64) == 0
    assert A.adam_embed_backward_workspace(10, 100, 64) == 512  # the sorted tokens and their order, one block: no parts
    # more rows than are ranked at once are sorted in passes, between two lists
    small, large = A.adam_embed_backward_workspace(16384, 100, 8), A.adam_embed_backward_workspace(16385, 100, 8)
    assert large > small + 2 * 16384 * 4
    n = ctypes.c_int64()
    L = TR.lib()
    assert L.adam_embed_backward_workspace(-1, 1, 1, ctypes.byref(n)) == EINVAL
    assert L.adam_embed_backward_workspace(1, 1, 1, None) == EINVAL
    assert L.adam_embed_backward_workspace(1 << 30, 1 << 20, 4096, ctypes.byref(n)) == OK


# q, k, v side by side in one projection's output, and their gradients alike
ATT = dict(rows=100, heads=8, kv_heads=2, head_dim=64, type=BF16, q=at(0), q_stride=768, q_head_stride=64,
           k=at(0, 1024), k_stride=768, k_head_stride=64, v=at(0, 1280), v_stride=768, v_head_stride=64,
           o=at(1), o_stride=512, o_head_stride=64, lse=at(2), doc_offsets=at(3), docs=3, prefix=None, causal=1, window=0,
           scale=0.125, softcap=0.0, slopes=None, dout=at(4), dout_stride=512, dout_head_stride=64,
           dq=at(5), dq_stride=768, dq_head_stride=64, dk=at(5, 1024), dk_stride=768, dk_head_stride=64,
           dv=at(5, 1280), dv_stride=768, dv_head_stride=64)


def attn(call, ws=at(6), size=1 << 30, **kw):
    return getattr(TR.lib(), call)(ctypes.byref(TR.AdamAttnDesc(**{**ATT, **kw})), ws, size, None)


BOTH = [
    (dict(type=9), EINVAL), (dict(type=F32), EDTYPE), (dict(type=A.DT_NONE), EDTYPE), (dict(rows=-1), EINVAL),
    (dict(rows=(1 << 30) + 1), EINVAL), (dict(heads=0), EINVAL), (dict(heads=65536), EINVAL), (dict(kv_heads=0), EINVAL),
    (dict(kv_heads=3), EINVAL), (dict(head_dim=0), EINVAL), (dict(head_dim=257), EINVAL), (dict(causal=2), EINVAL),
    (dict(window=-1), EINVAL), (dict(window=5, causal=0), EINVAL), (dict(prefix=at(7), causal=0), EINVAL),
    (dict(prefix=at(7), window=5), EINVAL), (dict(docs=-1), EINVAL), (dict(docs=2, doc_offsets=None), EINVAL),
    (dict(docs=0, doc_offsets=None), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL),
    (dict(scale=math.nan), EINVAL), (dict(scale=math.inf), EINVAL), (dict(softcap=-1.0), EINVAL),
    (dict(softcap=math.nan), EINVAL), (dict(softcap=math.inf), EINVAL), (dict(rows=1 << 30, heads=1 << 10, kv_heads=2), EINVAL),
    (dict(q_stride=-1), EINVAL), (dict(k_stride=(1 << 21) + 1), EINVAL), (dict(v_head_stride=-1), EINVAL),
    (dict(o_stride=-8), EINVAL), (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL),
    (dict(o=None), EINVAL), (dict(q=at(0, 1)), EINVAL), (dict(lse=at(2, 2)), EINVAL), (dict(doc_offsets=at(3, 2)), EINVAL),
    (dict(slopes=at(7, 2)), EINVAL), (dict(ws=None), EINVAL), (dict(size=0), EINVAL), (dict(ws=at(6, 16)), EINVAL),
    (dict(ws=at(0)), EINVAL), (dict(ws=at(3)), EINVAL),
]


@pytest.mark.parametrize("call", ["adam_attn_forward", "adam_attn_backward"])
@pytest.mark.parametrize("kw,want", BOTH)
def test_attention_refusals(call, kw, want):
    assert attn(call, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(o=at(0)), EINVAL), (dict(o=at(0, 256)), EINVAL), (dict(lse=at(1)), EINVAL), (dict(ws=at(1)), EINVAL),
    (dict(ws=at(2)), EINVAL), (dict(lse=at(3)), EINVAL), (dict(o_head_stride=63), EINVAL), (dict(o_stride=511), EINVAL),
])
def test_attention_forward_refusals(kw, want):
    assert attn("adam_attn_forward", **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(lse=None), EINVAL), (dict(dout=None), EINVAL), (dict(dq=None), EINVAL), (dict(dk=None), EINVAL),
    (dict(dv=None), EINVAL), (dict(dq=at(5, 1)), EINVAL), (dict(dq_stride=-1), EINVAL), (dict(dout_stride=1 << 22), EINVAL),
    (dict(dq=at(0)), EINVAL), (dict(dk=at(5)), EINVAL), (dict(dv=at(5, 1024)), EINVAL), (dict(dq=at(4)), EINVAL),
    (dict(dq=at(1)), EINVAL), (dict(dv=at(2)), EINVAL), (dict(dq_head_stride=32), EINVAL), (dict(dk_stride=100), EINVAL),
    (dict(ws=at(5)), EINVAL), (dict(ws=at(4)), EINVAL), (dict(dq_head_stride=96), EINVAL),
])
def test_attention_backward_refusals(kw, want):
    assert attn("adam_attn_backward", **kw) == want


def test_attention_of_nothing():
    for call in ("adam_attn_forward", "adam_attn_backward"):
        assert attn(call, rows=0, q=None, k=None, v=None, o=None, lse=None, dout=None, dq=None, dk=None, dv=None, ws=None,
                    size=0) == OK
        assert attn(call, docs=0, ws=None, size=0) == OK


def plan(**kw):
    st = TR.AdamAttnStats()
    rc = TR.lib().adam_attn_plan(ctypes.byref(TR.AdamAttnDesc(**{**ATT, **kw})), ctypes.byref(st))
    return rc, st.as_dict()


def test_attention_plan():
    rc, st = plan()
    assert rc == OK and 0 < st["forward_bytes"] < st["backward_bytes"]
    assert st["backward_bytes"] >= 2 * 8 * 100 * 4  # two floats for each row and query head
    rc, st = plan(rows=0)
    assert rc == OK and st == dict(forward_bytes=0, backward_bytes=0)
    assert plan(head_dim=300)[0] == EINVAL
    L = TR.lib()
    assert L.adam_attn_plan(None, ctypes.byref(TR.AdamAttnStats())) == EINVAL
    assert L.adam_attn_plan(ctypes.byref(TR.AdamAttnDesc(**ATT)), None) == EINVAL
    assert L.adam_attn_forward(None, None, 0, None) == EINVAL


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, dtype=torch.int64)
    w, y = torch.zeros(10, 8), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        A.adam_embed_forward(t, w, y)
    with pytest.raises(ValueError, match="token"):
        A.adam_embed_forward(t.int(), w, y)
    with pytest.raises(ValueError, match="y has"):
        A.adam_embed_forward(t, w, y[:3])
    with pytest.raises(ValueError, match="dy has"):
        A.adam_embed_backward(t, y[:, :4], w)
    q, k = torch.zeros(6, 4, 16).bfloat16(), torch.zeros(6, 2, 16).bfloat16()
    with pytest.raises(ValueError, match="GPU"):
        A.adam_attn_forward(q, k, k, torch.zeros_like(q))
    with pytest.raises(ValueError, match="v has"):
        A.adam_attn_forward(q, k, q, torch.zeros_like(q))
    with pytest.raises(ValueError, match="lse"):
        A.adam_attn_forward(q, k, k, torch.zeros_like(q), torch.zeros(6, 4))
    with pytest.raises(ValueError, match="contiguous last"):
        A.adam_attn_forward(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, torch.zeros_like(q))
    with pytest.raises(ValueError, match="doc_offsets"):
        A.adam_attn_forward(q, k, k, torch.zeros_like(q), doc_offsets=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="dtype"):
        A.adam_attn_forward(q, k.half(), k, torch.zeros_like(q))
    with pytest.raises(A.AdamError):  # float32 heads
        A.adam_attn_forward(q.float(), k.float(), k.float(), q.float().clone())
