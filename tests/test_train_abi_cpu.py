"""The training operators' C ABI on the CPU: every declared call is exported
and bound, sizes and plans follow the header, and every refusal the header
names returns its status before anything touches a device."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import adamw_optimizer_step_tensor_amd as A
from adamw_optimizer_step_tensor_amd import train as TR

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "adam_train.h")
BASE = 1 << 40  # fake, well-separated device addresses: refusals never touch them
GAP = 1 << 36
F32, BF16, F16 = A.DT_F32, A.DT_BF16, A.DT_F16
E4M3, E5M2 = TR.ACT8_E4M3, TR.ACT8_E5M2
OK, EINVAL, EDTYPE = A.ADAM_OK, A.ADAM_EINVAL, A.ADAM_EDTYPE


def at(k, offset=0):
    return BASE + k * GAP + offset


def test_every_declared_call_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^int (adam_\w+)\s*\(", text, flags=re.M))
    assert names == set(TR.TRAIN_EXPORTED)
    for n in names:
        assert hasattr(TR.lib(), n)
        assert callable(getattr(A, n)), n


@pytest.mark.parametrize("rows,cols,want", [(0, 0, 0), (0, 7, 0), (5, 0, 0), (1, 1, 256 + 1), (1, 33, 256 + 2),
                                            (8, 32, 256 + 8), (9, 32, 512 + 9), (3, 100, 512 + 12)])
def test_checkpoint_bytes(rows, cols, want):
    assert A.adam_act8_bytes(rows, cols) == want


def test_checkpoint_bytes_refusals():
    n = ctypes.c_int64()
    L = TR.lib()
    assert L.adam_act8_bytes(-1, 4, ctypes.byref(n)) == EINVAL
    assert L.adam_act8_bytes(4, 1 << 31, ctypes.byref(n)) == EINVAL
    assert L.adam_act8_bytes(4, 4, None) == EINVAL
    assert L.adam_act8_bytes((1 << 31) - 1, (1 << 31) - 1, ctypes.byref(n)) == OK


STORE = dict(x=at(0), t=BF16, rows=4, cols=64, stride=64, fmt=E4M3, ckpt=at(1))


def store(**kw):
    a = {**STORE, **kw}
    return TR.lib().adam_act8_store(a["x"], a["t"], a["rows"], a["cols"], a["stride"], a["fmt"], a["ckpt"], None)


def load(**kw):
    a = {**STORE, **kw}
    return TR.lib().adam_act8_load(a["ckpt"], a["fmt"], a["rows"], a["cols"], a["x"], a["t"], a["stride"], None)


@pytest.mark.parametrize("call", [store, load])
@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), EINVAL), (dict(cols=-1), EINVAL), (dict(rows=1 << 31), EINVAL), (dict(stride=63), EINVAL),
    (dict(x=None), EINVAL), (dict(ckpt=None), EINVAL), (dict(ckpt=at(1, 8)), EINVAL), (dict(x=at(0, 1)), EINVAL),
    (dict(t=F32, x=at(0, 2)), EINVAL), (dict(fmt=0), EINVAL), (dict(fmt=3), EINVAL), (dict(t=9), EINVAL),
    (dict(t=-1), EINVAL), (dict(t=A.DT_NONE), EDTYPE), (dict(ckpt=at(0, 256)), EINVAL),
    (dict(x=at(1, 128), cols=32), EINVAL),
])
def test_store_and_load_refusals(call, kw, want):
    assert call(**kw) == want


@pytest.mark.parametrize("call", [store, load])
def test_nothing_to_store(call):
    assert call(rows=0, x=None, ckpt=None) == OK
    assert call(cols=0, stride=0, x=None, ckpt=None) == OK


FWD = dict(gate=at(0), up=at(0, 128), t=BF16, rows=4, cols=64, in_stride=128, act=1, h=at(1), h_stride=64, fmt=E4M3,
           cg=at(2), cu=at(3))


def forward(**kw):
    a = {**FWD, **kw}
    return TR.lib().adam_glu_forward(a["gate"], a["up"], a["t"], a["rows"], a["cols"], a["in_stride"], a["act"],
                                     a["h"], a["h_stride"], a["fmt"], a["cg"], a["cu"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(act=0), EINVAL), (dict(act=3), EINVAL), (dict(fmt=7), EINVAL), (dict(t=A.DT_NONE), EDTYPE),
    (dict(gate=None), EINVAL), (dict(up=None), EINVAL), (dict(h=None), EINVAL), (dict(cu=None), EINVAL),
    (dict(cg=None), EINVAL), (dict(cg=at(2, 4)), EINVAL), (dict(in_stride=63), EINVAL), (dict(h_stride=63), EINVAL),
    (dict(h=at(0)), EINVAL), (dict(h=at(0, 130), h_stride=128), EINVAL), (dict(cg=at(0)), EINVAL),
    (dict(cg=at(3)), EINVAL), (dict(h=at(2)), EINVAL), (dict(gate=at(0, 1)), EINVAL),
])
def test_forward_refusals(kw, want):
    assert forward(**kw) == want


BWD = dict(dh=at(0), t=BF16, rows=4, cols=64, dh_stride=64, act=1, fmt=E4M3, cg=at(2), cu=at(3), dg=at(4),
           du=at(4, 128), d_stride=128, h=at(5), h_stride=64, ch=at(6))


def backward(**kw):
    a = {**BWD, **kw}
    return TR.lib().adam_glu_backward(a["dh"], a["t"], a["rows"], a["cols"], a["dh_stride"], a["act"], a["fmt"],
                                      a["cg"], a["cu"], a["dg"], a["du"], a["d_stride"], a["h"], a["h_stride"],
                                      a["ch"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(act=0), EINVAL), (dict(fmt=0), EINVAL), (dict(t=A.DT_NONE), EDTYPE), (dict(dh=None), EINVAL),
    (dict(cg=None), EINVAL), (dict(cu=None), EINVAL), (dict(dg=None), EINVAL), (dict(du=None), EINVAL),
    (dict(d_stride=60), EINVAL), (dict(dh_stride=60), EINVAL), (dict(h_stride=60), EINVAL),
    (dict(ch=at(6, 8)), EINVAL), (dict(du=at(4, 126)), EINVAL), (dict(du=at(4)), EINVAL), (dict(h=at(4)), EINVAL),
    (dict(ch=at(2)), EINVAL), (dict(ch=at(4)), EINVAL), (dict(dg=at(0)), EINVAL),
    (dict(dg=at(0, 2), d_stride=64, du=at(7)), EINVAL), (dict(h=at(0)), EINVAL),
])
def test_backward_refusals(kw, want):
    assert backward(**kw) == want


WG = dict(dy=at(0), t=BF16, dys=64, ckpt=at(1), fmt=E4M3, rows=100, n=64, k=96, dw=at(2), wt=F32, dws=96, acc=0,
          ws=at(3), size=1 << 34)


def wgrad(**kw):
    a = {**WG, **kw}
    return TR.lib().adam_act8_wgrad(a["dy"], a["t"], a["dys"], a["ckpt"], a["fmt"], a["rows"], a["n"], a["k"],
                                    a["dw"], a["wt"], a["dws"], a["acc"], a["ws"], a["size"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(t=F32), EDTYPE), (dict(t=A.DT_NONE), EDTYPE), (dict(wt=F16), EDTYPE), (dict(wt=A.DT_NONE), EDTYPE),
    (dict(t=11), EINVAL), (dict(fmt=0), EINVAL), (dict(acc=2), EINVAL), (dict(rows=-1), EINVAL), (dict(n=-1), EINVAL),
    (dict(k=(1 << 21) + 1, dws=1 << 22), EINVAL), (dict(rows=(1 << 30) + 1), EINVAL),
    (dict(n=1 << 21, k=1 << 21, dys=1 << 21, dws=1 << 21), EINVAL), (dict(dys=63), EINVAL), (dict(dws=95), EINVAL),
    (dict(dw=None), EINVAL), (dict(dy=None), EINVAL), (dict(ckpt=None), EINVAL), (dict(ckpt=at(1, 8)), EINVAL),
    (dict(dw=at(2, 2)), EINVAL), (dict(dw=at(0)), EINVAL), (dict(dw=at(1)), EINVAL),
    (dict(dys=65, ws=None), EINVAL), (dict(dys=65, size=16), EINVAL), (dict(dys=65, ws=at(3, 16)), EINVAL),
    (dict(dys=65, ws=at(2)), EINVAL),
])
def test_wgrad_refusals(kw, want):
    assert wgrad(**kw) == want


def test_wgrad_workspace():
    n = ctypes.c_int64()
    L = TR.lib()
    # few steps and nothing to pack: no workspace
    assert L.adam_act8_wgrad_workspace(100, 64, 96, at(0), 64, ctypes.byref(n)) == OK and n.value == 0
    # an odd stride packs dy: 100 rows of 64 16-bit values
    assert L.adam_act8_wgrad_workspace(100, 64, 96, at(0), 65, ctypes.byref(n)) == OK and n.value == 100 * 128
    assert L.adam_act8_wgrad_workspace(100, 64, 96, at(0, 2), 64, ctypes.byref(n)) == OK and n.value == 100 * 128
    # one tile over many rows is split: every part holds a tile of 256 x 256 floats
    assert L.adam_act8_wgrad_workspace(65536, 64, 96, at(0), 64, ctypes.byref(n)) == OK
    assert n.value > 0 and n.value % (256 * 256 * 4) == 0
    assert L.adam_act8_wgrad_workspace(100, 64, 0, at(0), 64, ctypes.byref(n)) == OK and n.value == 0
    assert L.adam_act8_wgrad_workspace(100, 64, 96, at(0), 60, ctypes.byref(n)) == EINVAL
    assert L.adam_act8_wgrad_workspace(100, 64, 96, at(0), 64, None) == EINVAL


XE = dict(rows=100, hidden=64, vocab=1000, type=BF16, dw_type=F32, h=at(0), h_stride=64, w=at(1), w_stride=64,
          target=at(2), weight=at(3), ignore_index=-100, loss=at(4), lse=at(5), dh=at(6), dh_stride=64, dw=at(7),
          dw_stride=64, accumulate=0, d_loss_scale=at(8), piece_rows=0)


def xent(ws=at(9), size=1 << 34, **kw):
    d = TR.AdamXentDesc(**{**XE, **kw})
    return TR.lib().adam_xent(ctypes.byref(d), ws, size, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), EINVAL), (dict(hidden=0, h_stride=64), EINVAL), (dict(vocab=0), EINVAL),
    (dict(vocab=1 << 21), EINVAL), (dict(rows=(1 << 30) + 1), EINVAL),
    (dict(rows=1 << 20, vocab=1 << 20, piece_rows=1 << 20), EINVAL),
    (dict(hidden=1 << 21, vocab=1 << 20, h_stride=1 << 21, w_stride=1 << 21, dh_stride=1 << 21, dw_stride=1 << 21), EINVAL),
    (dict(type=F32), EDTYPE), (dict(type=A.DT_NONE), EDTYPE),
    (dict(dw_type=F16), EDTYPE), (dict(dw_type=A.DT_NONE), EDTYPE), (dict(type=5), EINVAL), (dict(dw_type=-1), EINVAL),
    (dict(h_stride=63), EINVAL), (dict(w_stride=63), EINVAL), (dict(dh_stride=63), EINVAL),
    (dict(dw_stride=63), EINVAL), (dict(h=None), EINVAL), (dict(w=None), EINVAL), (dict(target=None), EINVAL),
    (dict(loss=None), EINVAL), (dict(accumulate=2), EINVAL), (dict(piece_rows=-1), EINVAL),
    (dict(ws=None), EINVAL), (dict(size=100), EINVAL), (dict(ws=at(9, 16)), EINVAL), (dict(h=at(0, 1)), EINVAL),
    (dict(target=at(2, 4)), EINVAL), (dict(loss=at(4, 2)), EINVAL), (dict(dw=at(7, 2)), EINVAL),
    (dict(dh=at(0)), EINVAL), (dict(dw=at(1)), EINVAL), (dict(dw=at(6)), EINVAL), (dict(lse=at(4)), EINVAL),
    (dict(loss=at(2)), EINVAL), (dict(ws=at(7)), EINVAL), (dict(lse=at(3)), EINVAL),
])
def test_xent_refusals(kw, want):
    assert xent(**kw) == want


def plan(**kw):
    d = TR.AdamXentDesc(**{**XE, **kw})
    st = TR.AdamXentStats()
    rc = TR.lib().adam_xent_plan(ctypes.byref(d), ctypes.byref(st))
    return rc, st.as_dict()


def test_xent_plan():
    rc, st = plan()
    assert rc == OK and st["piece_rows"] == 256 and st["pieces"] == 1
    # with gradient: as many rows as keep 16-bit G within 1 GiB
    rc, st = plan(rows=20000, vocab=131072, hidden=4096, h_stride=4096, w_stride=4096, dh_stride=4096, dw_stride=4096)
    assert rc == OK and st["piece_rows"] == 4096 and st["pieces"] == 5
    assert (1 << 30) < st["workspace_bytes"] < (1 << 30) + (1 << 29)
    # a 16-bit dw would need its sums in float: one piece where that is no larger
    kw = dict(vocab=131072, hidden=4096, h_stride=4096, w_stride=4096, dh_stride=4096, dw_stride=4096, dw_type=BF16)
    rc, st = plan(rows=8192, **kw)
    assert rc == OK and st["pieces"] == 1
    rc, st = plan(rows=50000, **kw)
    assert rc == OK and st["piece_rows"] == 4096 and st["pieces"] == 13
    assert st["workspace_bytes"] > (1 << 30) + 131072 * 4096 * 4
    # loss alone
    rc, st = plan(rows=50000, vocab=131072, dh=None, dw=None, dw_type=A.DT_NONE)
    assert rc == OK and st["piece_rows"] == 16384 and st["pieces"] == 4
    # asked for
    rc, st = plan(rows=1000, piece_rows=300)
    assert rc == OK and st["piece_rows"] == 512 and st["pieces"] == 2
    rc, st = plan(rows=0)
    assert rc == OK and st["pieces"] == 1
    assert TR.lib().adam_xent_plan(None, ctypes.byref(TR.AdamXentStats())) == EINVAL
    assert TR.lib().adam_xent_plan(ctypes.byref(TR.AdamXentDesc(**XE)), None) == EINVAL


def test_xent_without_rows_or_gradient_does_nothing():
    assert xent(rows=0, h=None, target=None, loss=None, dw=None, dw_type=A.DT_NONE, ws=None, size=0) == OK


C_CLIENT = r"""
#include <stddef.h>
#include "adam_train.h"
int main(void)
{
    int64_t n = -1;
    adam_xent_desc d = {0};
    adam_xent_stats st;
    if (adam_act8_bytes(9, 32, &n) != ADAM_OK || n != 512 + 9) return 1;
    if (adam_act8_store(NULL, ADAM_DT_F32, 1, 1, 1, ADAM_ACT8_E4M3, NULL, NULL) != ADAM_EINVAL) return 2;
    d.rows = 10;
    d.hidden = d.h_stride = d.w_stride = 8;
    d.vocab = 100;
    d.type = ADAM_DT_BF16;
    if (adam_xent_plan(&d, &st) != ADAM_OK || st.pieces != 1 || st.workspace_bytes <= 0) return 3;
    if (adam_xent(&d, NULL, 0, NULL) != ADAM_EINVAL) return 4;
    return 0;
}
"""


def test_header_is_c99_and_links(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    rocm, pkg = os.environ.get("ROCM_PATH", "/opt/rocm"), os.path.dirname(A.LIBRARY_PATH)
    source, exe = tmp_path / "client.c", tmp_path / "client"
    source.write_text(C_CLIENT)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-D__HIP_PLATFORM_AMD__",
                    f"-I{os.path.join(ROOT, 'include')}", "-isystem", os.path.join(rocm, "include"), str(source), "-o",
                    str(exe), f"-L{pkg}", "-l:libadamw_mi355x.so", f"-Wl,-rpath,{pkg}"], check=True)
    assert subprocess.run([str(exe)], timeout=120).returncode == 0


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    ck = torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        A.adam_act8_store(x, ck)
    with pytest.raises(ValueError, match="fmt"):
        A.adam_act8_store(x, ck, "int8")
    with pytest.raises(ValueError, match="contiguous rows"):
        A.adam_act8_store(x.t(), ck)
    with pytest.raises(ValueError, match="needed"):
        A.adam_act8_store(x, ck[:100])
    with pytest.raises(ValueError, match="2-D"):
        A.adam_act8_store(x[0], ck)
    with pytest.raises(ValueError, match="uint8"):
        A.adam_act8_store(x, ck.to(torch.int8))
    with pytest.raises(ValueError, match="shape"):
        A.adam_glu_forward(x, x[:, :32], x)
    with pytest.raises(ValueError, match="act"):
        A.adam_glu_forward(x, x, x, "relu")
    with pytest.raises(ValueError, match="stride"):
        A.adam_glu_forward(x, torch.zeros(4, 128)[:, :64], x)
    t = torch.zeros(4, dtype=torch.int64)
    loss = torch.zeros(4)
    w = torch.zeros(10, 64)
    with pytest.raises(ValueError, match="target"):
        A.adam_xent(x, w, t.int(), loss)
    with pytest.raises(ValueError, match="loss"):
        A.adam_xent(x, w, t, loss[:3])
    with pytest.raises(ValueError, match="w has"):
        A.adam_xent(x, w[:, :32], t, loss)
    with pytest.raises(A.AdamError):  # float32 hidden states
        A.adam_xent(x, w, t, loss)
