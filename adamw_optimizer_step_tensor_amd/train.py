"""Binding of the training operators (``include/adam_train.h``): the embedding
of tokens with its gradient, attention over packed documents with its gradient,
8-bit activation checkpoints with the backward steps that read them, and softmax
cross entropy over a large vocabulary with its gradient.

Argument marshalling only, like the rest of the package: the caller passes
every output, and each function has the name of the C call it makes.  Tensors
are 2-D with contiguous rows (any row stride), on one device; the call runs on
that device's current stream unless ``stream`` is given.  A workspace may be
passed (uint8, as many bytes as the plan says; one per call that may run at the
same time); otherwise one is allocated for the call.  Attention takes tensors of
rows x heads x head_dim, whose last dimension is contiguous.

    A.adam_embed_forward(tokens, w_embed, x)
    A.adam_attn_forward(q, k, v, o, lse, doc_offsets=offsets)               # q, k, v: views of qkv
    ...
    A.adam_attn_backward(d_o, q, k, v, o, lse, dq, dk, dv, doc_offsets=offsets)
    A.adam_embed_backward(tokens, dx, grad_w_embed)                         # accumulate=True: a tied weight
    ...
    ckpt_g, ckpt_u = (torch.empty(A.adam_act8_bytes(T, F), dtype=torch.uint8, device="cuda") for _ in range(2))
    A.adam_glu_forward(x[:, :F], x[:, F:], h, "silu", ckpt_g, ckpt_u)      # x: gate and up side by side
    ...
    A.adam_xent(hidden, w, target, loss, dh=dh, dw=dw, d_loss_scale=scale)
    ...
    A.adam_glu_backward(d_h, ckpt_g, ckpt_u, dx[:, :F], dx[:, F:], "silu", ckpt_h=ckpt_h)
    A.adam_act8_wgrad(dy, ckpt_h, grad_w_down)                            # grad_w_down: the handle's g
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import DT_BF16, DT_F16, DT_F32, DT_NONE, _check, c_f32, c_i32, c_i64, c_vp
from . import lib as _base_lib

ACT8_E4M3, ACT8_E5M2 = 1, 2
ACT_SILU, ACT_GELU = 1, 2
FORMATS = {"e4m3": ACT8_E4M3, "e5m2": ACT8_E5M2}
ACTS = {"silu": ACT_SILU, "gelu": ACT_GELU}

TRAIN_EXPORTED = ("adam_act8_bytes", "adam_act8_store", "adam_act8_load", "adam_glu_forward", "adam_glu_backward",
                  "adam_act8_wgrad_workspace", "adam_act8_wgrad", "adam_xent_plan", "adam_xent", "adam_embed_forward",
                  "adam_embed_backward_workspace", "adam_embed_backward", "adam_attn_plan", "adam_attn_forward",
                  "adam_attn_backward")


class AdamXentDesc(ctypes.Structure):
    """adam_xent_desc"""
    _fields_ = [("rows", c_i64), ("hidden", c_i64), ("vocab", c_i64), ("type", c_i32), ("dw_type", c_i32),
                ("h", c_vp), ("h_stride", c_i64), ("w", c_vp), ("w_stride", c_i64), ("target", c_vp),
                ("weight", c_vp), ("ignore_index", c_i64), ("loss", c_vp), ("lse", c_vp), ("dh", c_vp),
                ("dh_stride", c_i64), ("dw", c_vp), ("dw_stride", c_i64), ("accumulate", c_i32),
                ("d_loss_scale", c_vp), ("piece_rows", c_i64)]


class AdamXentStats(ctypes.Structure):
    """adam_xent_stats"""
    _fields_ = [("workspace_bytes", c_i64), ("piece_rows", c_i64), ("pieces", c_i64)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class AdamAttnDesc(ctypes.Structure):
    """adam_attn_desc"""
    _fields_ = [("rows", c_i64), ("heads", c_i64), ("kv_heads", c_i64), ("head_dim", c_i64), ("type", c_i32),
                ("q", c_vp), ("q_stride", c_i64), ("q_head_stride", c_i64),
                ("k", c_vp), ("k_stride", c_i64), ("k_head_stride", c_i64),
                ("v", c_vp), ("v_stride", c_i64), ("v_head_stride", c_i64),
                ("o", c_vp), ("o_stride", c_i64), ("o_head_stride", c_i64), ("lse", c_vp),
                ("doc_offsets", c_vp), ("docs", c_i64), ("prefix", c_vp), ("causal", c_i32), ("window", c_i64),
                ("scale", c_f32), ("softcap", c_f32), ("slopes", c_vp),
                ("dout", c_vp), ("dout_stride", c_i64), ("dout_head_stride", c_i64),
                ("dq", c_vp), ("dq_stride", c_i64), ("dq_head_stride", c_i64),
                ("dk", c_vp), ("dk_stride", c_i64), ("dk_head_stride", c_i64),
                ("dv", c_vp), ("dv_stride", c_i64), ("dv_head_stride", c_i64)]


class AdamAttnStats(ctypes.Structure):
    """adam_attn_stats"""
    _fields_ = [("forward_bytes", c_i64), ("backward_bytes", c_i64)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


_declared = None


def lib():
    """The loaded library with the training calls' signatures."""
    global _declared
    L = _base_lib()
    if _declared is L:
        return L
    i64p = ctypes.POINTER(c_i64)
    L.adam_act8_bytes.argtypes = [c_i64, c_i64, i64p]
    L.adam_act8_store.argtypes = [c_vp, c_i32, c_i64, c_i64, c_i64, c_i32, c_vp, c_vp]
    L.adam_act8_load.argtypes = [c_vp, c_i32, c_i64, c_i64, c_vp, c_i32, c_i64, c_vp]
    L.adam_glu_forward.argtypes = [c_vp, c_vp, c_i32, c_i64, c_i64, c_i64, c_i32, c_vp, c_i64, c_i32, c_vp, c_vp, c_vp]
    L.adam_glu_backward.argtypes = [c_vp, c_i32, c_i64, c_i64, c_i64, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_i64,
                                    c_vp, c_i64, c_vp, c_vp]
    L.adam_act8_wgrad_workspace.argtypes = [c_i64, c_i64, c_i64, c_vp, c_i64, i64p]
    L.adam_act8_wgrad.argtypes = [c_vp, c_i32, c_i64, c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i32, c_i64, c_i32,
                                  c_vp, c_i64, c_vp]
    L.adam_xent_plan.argtypes = [ctypes.POINTER(AdamXentDesc), ctypes.POINTER(AdamXentStats)]
    L.adam_xent.argtypes = [ctypes.POINTER(AdamXentDesc), c_vp, c_i64, c_vp]
    L.adam_embed_forward.argtypes = [c_vp, c_i64, c_vp, c_i32, c_i64, c_i64, c_i64, c_f32, c_i64, c_vp, c_i32, c_i64,
                                     c_vp]
    L.adam_embed_backward_workspace.argtypes = [c_i64, c_i64, c_i64, i64p]
    L.adam_embed_backward.argtypes = [c_vp, c_i64, c_vp, c_i32, c_i64, c_f32, c_i64, c_vp, c_i32, c_i64, c_i64, c_i64,
                                      c_i32, c_vp, c_i64, c_vp]
    L.adam_attn_plan.argtypes = [ctypes.POINTER(AdamAttnDesc), ctypes.POINTER(AdamAttnStats)]
    L.adam_attn_forward.argtypes = L.adam_attn_backward.argtypes = [ctypes.POINTER(AdamAttnDesc), c_vp, c_i64, c_vp]
    for name in TRAIN_EXPORTED:
        getattr(L, name).restype = c_i32
    _declared = L
    return L


# ---------------------------------------------------------------------------
# Marshalling helpers
# ---------------------------------------------------------------------------

_CODES = {}


def _dtype(x) -> int:
    if not _CODES:
        import torch

        _CODES.update({torch.float32: DT_F32, torch.bfloat16: DT_BF16, torch.float16: DT_F16})
    code = _CODES.get(x.dtype)
    if code is None:
        raise ValueError(f"dtype {x.dtype} is not float32, bfloat16 or float16")
    return code


def _matrix(x, name, shape=None, dtype=None):
    """Row stride of a 2-D tensor with contiguous rows."""
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = x.shape
    if shape is not None and x.shape != shape and (rows, cols) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected {tuple(shape)}")
    if dtype is not None and x.dtype != dtype:
        raise ValueError(f"{name} has dtype {x.dtype}, expected {dtype}")
    if cols > 1 and x.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    # a single row or column has no stride of its own
    return max(cols, 1) if rows <= 1 else x.stride(0)


def _vector(x, name, n, dtype):
    if x is None:
        return None
    if x.dim() != 1 or x.numel() != n or x.dtype != dtype or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} elements")
    return x.data_ptr()


def _bytes(x, name, need):
    if x is None:
        return None
    import torch

    if x.dtype != torch.uint8 or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous uint8 tensor")
    if x.numel() < need:
        raise ValueError(f"{name} holds {x.numel()} bytes, {need} needed")
    return x.data_ptr()


def _one_device(*tensors) -> int:
    """The index of the GPU that all the given tensors lie on."""
    index = None
    for t in tensors:
        if t is None:
            continue
        i = t.get_device()  # -1: not on a GPU
        if i < 0:
            raise ValueError("tensors must be on the GPU")
        if index is None:
            index = i
        elif i != index:
            raise ValueError(f"tensors on cuda:{index} and cuda:{i}")
    return index


def _option(table, key, name):
    if key not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}")
    return table[key]


class _On:
    """Makes a device current for a call and gives the stream's address: the
    device's current stream, or the caller's (a torch stream or an address)."""

    def __init__(self, index: int, stream):
        import torch

        self.index, self.stream, self.guard = index, stream, None
        if stream is None:
            self.address = torch._C._cuda_getCurrentRawStream(index)
        elif isinstance(stream, int):
            self.address = stream
        else:
            if stream.device.index != index:
                raise ValueError(f"stream on {stream.device}, tensors on cuda:{index}")
            self.address = stream.cuda_stream
        if torch.cuda.current_device() != index:
            self.guard = torch.cuda.device(index)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.address

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def empty(self, need: int):
        """A workspace whose reuse the allocator orders after this call."""
        import torch

        if self.stream is None:
            return torch.empty(need, dtype=torch.uint8, device=f"cuda:{self.index}")
        s = self.stream
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s, device=self.index) if s else torch.cuda.default_stream(self.index)
        with torch.cuda.stream(s):
            return torch.empty(need, dtype=torch.uint8, device=f"cuda:{self.index}")


def _workspace(workspace, need, on):
    """(address, bytes, owner) of the caller's workspace or of one for this
    call; the owner has to live until the call is enqueued."""
    if need == 0:
        return None, 0, None
    if workspace is None:
        workspace = on.empty(need)
    return _bytes(workspace, "workspace", need), workspace.numel(), workspace


# ---------------------------------------------------------------------------
# The C ABI, one function each
# ---------------------------------------------------------------------------

def adam_act8_bytes(rows: int, cols: int) -> int:
    """Bytes of a checkpoint of a rows x cols matrix."""
    n = c_i64()
    _check(lib().adam_act8_bytes(rows, cols, ctypes.byref(n)), "adam_act8_bytes")
    return n.value


def adam_act8_store(x, ckpt, fmt: str = "e4m3", stream=None) -> None:
    """Stores the matrix x (float32, bfloat16 or float16) as an 8-bit
    checkpoint into the uint8 buffer ``ckpt``."""
    stride, f = _matrix(x, "x"), _option(FORMATS, fmt, "fmt")
    rows, cols = x.shape
    at = _bytes(ckpt, "ckpt", adam_act8_bytes(rows, cols))
    with _On(_one_device(x, ckpt), stream) as s:
        _check(lib().adam_act8_store(x.data_ptr(), _dtype(x), rows, cols, stride, f, at, s), "adam_act8_store")


def adam_act8_load(ckpt, x, fmt: str = "e4m3", stream=None) -> None:
    """Decodes a checkpoint into the matrix x."""
    stride, f = _matrix(x, "x"), _option(FORMATS, fmt, "fmt")
    rows, cols = x.shape
    at = _bytes(ckpt, "ckpt", adam_act8_bytes(rows, cols))
    with _On(_one_device(x, ckpt), stream) as s:
        _check(lib().adam_act8_load(at, f, rows, cols, x.data_ptr(), _dtype(x), stride, s), "adam_act8_load")


def adam_glu_forward(gate, up, h, act: str = "silu", ckpt_gate=None, ckpt_up=None, fmt: str = "e4m3",
                     stream=None) -> None:
    """h = a(gate) * up, and the checkpoints of gate and up in the same pass."""
    rows, cols = gate.shape
    in_stride = _matrix(gate, "gate")
    if _matrix(up, "up", gate.shape, gate.dtype) != in_stride:
        raise ValueError("gate and up must have the same row stride")
    h_stride = _matrix(h, "h", gate.shape, gate.dtype)
    f, a = _option(FORMATS, fmt, "fmt"), _option(ACTS, act, "act")
    n8 = adam_act8_bytes(rows, cols)
    cg, cu = _bytes(ckpt_gate, "ckpt_gate", n8), _bytes(ckpt_up, "ckpt_up", n8)
    with _On(_one_device(gate, up, h, ckpt_gate, ckpt_up), stream) as s:
        _check(lib().adam_glu_forward(gate.data_ptr(), up.data_ptr(), _dtype(gate), rows, cols, in_stride, a,
                                      h.data_ptr(), h_stride, f, cg, cu, s), "adam_glu_forward")


def adam_glu_backward(dh, ckpt_gate, ckpt_up, dgate, dup, act: str = "silu", fmt: str = "e4m3", h=None, ckpt_h=None,
                      stream=None) -> None:
    """dgate and dup of h = a(gate) * up from the checkpoints; h and its
    checkpoint again where wanted."""
    rows, cols = dh.shape
    dh_stride = _matrix(dh, "dh")
    d_stride = _matrix(dgate, "dgate", dh.shape, dh.dtype)
    if _matrix(dup, "dup", dh.shape, dh.dtype) != d_stride:
        raise ValueError("dgate and dup must have the same row stride")
    h_stride = 0 if h is None else _matrix(h, "h", dh.shape, dh.dtype)
    f, a = _option(FORMATS, fmt, "fmt"), _option(ACTS, act, "act")
    n8 = adam_act8_bytes(rows, cols)
    cg, cu, ch = (_bytes(c, n, n8) for c, n in ((ckpt_gate, "ckpt_gate"), (ckpt_up, "ckpt_up"), (ckpt_h, "ckpt_h")))
    with _On(_one_device(dh, ckpt_gate, ckpt_up, dgate, dup, h, ckpt_h), stream) as s:
        _check(lib().adam_glu_backward(dh.data_ptr(), _dtype(dh), rows, cols, dh_stride, a, f, cg, cu,
                                       dgate.data_ptr(), dup.data_ptr(), d_stride,
                                       None if h is None else h.data_ptr(), h_stride, ch, s), "adam_glu_backward")


def adam_act8_wgrad_workspace(dy, k: int) -> int:
    """Workspace bytes of adam_act8_wgrad for dy (rows x n) and k inputs."""
    n = c_i64()
    _check(lib().adam_act8_wgrad_workspace(dy.shape[0], dy.shape[1], k, dy.data_ptr(), _matrix(dy, "dy"),
                                           ctypes.byref(n)), "adam_act8_wgrad_workspace")
    return n.value


def adam_act8_wgrad(dy, ckpt, dw, fmt: str = "e4m3", accumulate: bool = False, workspace=None, stream=None) -> None:
    """dw (n x k) = (accumulate ? dw : 0) + dy^T x, with x the decoded
    checkpoint of rows x k."""
    dy_stride = _matrix(dy, "dy")
    rows, n = dy.shape
    dw_stride = _matrix(dw, "dw", (n, dw.shape[1]) if dw.dim() == 2 else None)
    k, f = dw.shape[1], _option(FORMATS, fmt, "fmt")
    at = _bytes(ckpt, "ckpt", adam_act8_bytes(rows, k))
    on = _On(_one_device(dy, ckpt, dw, workspace), stream)
    need = adam_act8_wgrad_workspace(dy, k)
    with on as s:
        ws, size, owner = _workspace(workspace, need, on)
        _check(lib().adam_act8_wgrad(dy.data_ptr(), _dtype(dy), dy_stride, at, f, rows, n, k, dw.data_ptr(),
                                     _dtype(dw), dw_stride, 1 if accumulate else 0, ws, size, s), "adam_act8_wgrad")
        del owner


def _xent_desc(h, w, target, loss, lse, weight, dh, dw, d_loss_scale, ignore_index, accumulate, piece_rows):
    import torch

    h_stride, w_stride = _matrix(h, "h"), _matrix(w, "w", dtype=h.dtype)
    rows, hidden = h.shape
    vocab = w.shape[0]
    _matrix(w, "w", (vocab, hidden))
    f32 = torch.float32
    d = AdamXentDesc(rows=rows, hidden=hidden, vocab=vocab, type=_dtype(h), dw_type=DT_NONE, h=h.data_ptr(),
                     h_stride=h_stride, w=w.data_ptr(), w_stride=w_stride,
                     target=_vector(target, "target", rows, torch.int64), weight=_vector(weight, "weight", rows, f32),
                     ignore_index=ignore_index, loss=_vector(loss, "loss", rows, f32),
                     lse=_vector(lse, "lse", rows, f32), accumulate=1 if accumulate else 0, piece_rows=piece_rows)
    if dh is not None:
        d.dh_stride, d.dh = _matrix(dh, "dh", (rows, hidden), h.dtype), dh.data_ptr()
    if dw is not None:
        d.dw_stride, d.dw, d.dw_type = _matrix(dw, "dw", (vocab, hidden)), dw.data_ptr(), _dtype(dw)
    if d_loss_scale is not None:
        if d_loss_scale.dtype != f32 or d_loss_scale.numel() != 1:
            raise ValueError("d_loss_scale must be one float32")
        d.d_loss_scale = d_loss_scale.data_ptr()
    return d


def adam_xent_plan(h, w, target=None, loss=None, *, lse=None, weight=None, dh=None, dw=None, d_loss_scale=None,
                   ignore_index: int = -100, accumulate: bool = False, piece_rows: int = 0) -> dict:
    """workspace_bytes, piece_rows and pieces of an adam_xent call with the
    same h, w, dh, dw and piece_rows."""
    d = _xent_desc(h, w, target, loss, lse, weight, dh, dw, d_loss_scale, ignore_index, accumulate, piece_rows)
    st = AdamXentStats()
    _check(lib().adam_xent_plan(ctypes.byref(d), ctypes.byref(st)), "adam_xent_plan")
    return st.as_dict()


def adam_xent(h, w, target, loss, *, lse=None, weight=None, dh=None, dw=None, d_loss_scale=None,
              ignore_index: int = -100, accumulate: bool = False, piece_rows: int = 0, workspace: Optional[object] = None,
              stream=None) -> None:
    """Cross entropy of the logits w h against int64 targets: loss (and lse)
    per row, and dh and dw of d_loss_scale * sum(loss) where they are given."""
    d = _xent_desc(h, w, target, loss, lse, weight, dh, dw, d_loss_scale, ignore_index, accumulate, piece_rows)
    st = AdamXentStats()
    _check(lib().adam_xent_plan(ctypes.byref(d), ctypes.byref(st)), "adam_xent_plan")
    on = _On(_one_device(h, w, target, loss, lse, weight, dh, dw, d_loss_scale, workspace), stream)
    with on as s:
        ws, size, owner = _workspace(workspace, st.workspace_bytes, on)
        _check(lib().adam_xent(ctypes.byref(d), ws, size, s), "adam_xent")
        del owner


def adam_embed_forward(token, w, y, scale: float = 1.0, ignore_index: int = -100, stream=None) -> None:
    """y[t] = scale * w[token[t]] for int64 tokens; rows of ignore_index are 0."""
    import torch

    w_stride = _matrix(w, "w")
    vocab, hidden = w.shape
    rows = token.numel()
    at, y_stride = _vector(token, "token", rows, torch.int64), _matrix(y, "y", (rows, hidden))
    with _On(_one_device(token, w, y), stream) as s:
        _check(lib().adam_embed_forward(at, rows, w.data_ptr(), _dtype(w), vocab, hidden, w_stride, scale, ignore_index,
                                        y.data_ptr(), _dtype(y), y_stride, s), "adam_embed_forward")


def adam_embed_backward_workspace(rows: int, vocab: int, hidden: int) -> int:
    """Workspace bytes of adam_embed_backward."""
    n = c_i64()
    _check(lib().adam_embed_backward_workspace(rows, vocab, hidden, ctypes.byref(n)), "adam_embed_backward_workspace")
    return n.value


def adam_embed_backward(token, dy, dw, scale: float = 1.0, ignore_index: int = -100, accumulate: bool = False,
                        workspace=None, stream=None) -> None:
    """dw[v] = (accumulate ? dw[v] : 0) + scale * the sum of the rows of dy whose token is v."""
    import torch

    dw_stride = _matrix(dw, "dw")
    vocab, hidden = dw.shape
    rows = token.numel()
    at, dy_stride = _vector(token, "token", rows, torch.int64), _matrix(dy, "dy", (rows, hidden))
    on = _On(_one_device(token, dy, dw, workspace), stream)
    need = adam_embed_backward_workspace(rows, vocab, hidden)
    with on as s:
        ws, size, owner = _workspace(workspace, need, on)
        _check(lib().adam_embed_backward(at, rows, dy.data_ptr(), _dtype(dy), dy_stride, scale, ignore_index,
                                         dw.data_ptr(), _dtype(dw), vocab, hidden, dw_stride, 1 if accumulate else 0,
                                         ws, size, s), "adam_embed_backward")
        del owner


def _heads(x, name, shape, dtype):
    """(address, row stride, head stride) of a tensor of rows x heads x head_dim."""
    if x.dim() != 3 or x.shape != shape:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected {tuple(shape)}")
    if x.dtype != dtype:
        raise ValueError(f"{name} has dtype {x.dtype}, expected {dtype}")
    rows, heads, dim = shape
    row, head, last = x.stride()
    if dim > 1 and last != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    # a dimension of one entry has no stride of its own
    if heads == 1:
        head = dim
    if rows <= 1:
        row = head * heads
    return x.data_ptr(), row, head


def _attn_desc(q, k, v, o, lse, doc_offsets, prefix, causal, window, scale, softcap, slopes):
    import torch

    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must have shape (rows, heads, head_dim)")
    rows, heads, dim = q.shape
    shape, kv_shape = q.shape, (rows, k.shape[1], dim)
    d = AdamAttnDesc(rows=rows, heads=heads, kv_heads=kv_shape[1], head_dim=dim, type=_dtype(q), docs=1,
                     causal=1 if causal else 0, window=window, scale=dim ** -0.5 if scale is None else scale,
                     softcap=softcap)
    d.q, d.q_stride, d.q_head_stride = _heads(q, "q", shape, q.dtype)
    d.k, d.k_stride, d.k_head_stride = _heads(k, "k", kv_shape, q.dtype)
    d.v, d.v_stride, d.v_head_stride = _heads(v, "v", kv_shape, q.dtype)
    d.o, d.o_stride, d.o_head_stride = _heads(o, "o", shape, q.dtype)
    if lse is not None:
        if lse.shape != (heads, rows) or lse.dtype != torch.float32 or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 tensor of shape {(heads, rows)}")
        d.lse = lse.data_ptr()
    if doc_offsets is not None:
        d.docs = doc_offsets.numel() - 1
        if d.docs < 0:
            raise ValueError("doc_offsets must hold one entry more than there are documents")
        d.doc_offsets = _vector(doc_offsets, "doc_offsets", d.docs + 1, torch.int32)
    d.prefix = _vector(prefix, "prefix", d.docs, torch.int32)
    d.slopes = _vector(slopes, "slopes", heads, torch.float32)
    return d, shape, kv_shape


def adam_attn_plan(q, k, v, o, lse=None, *, doc_offsets=None, prefix=None, causal: bool = True, window: int = 0,
                   scale: Optional[float] = None, softcap: float = 0.0, slopes=None) -> dict:
    """forward_bytes and backward_bytes: the workspaces of the two passes."""
    d, _, _ = _attn_desc(q, k, v, o, lse, doc_offsets, prefix, causal, window, scale, softcap, slopes)
    st = AdamAttnStats()
    _check(lib().adam_attn_plan(ctypes.byref(d), ctypes.byref(st)), "adam_attn_plan")
    return st.as_dict()


def adam_attn_forward(q, k, v, o, lse=None, *, doc_offsets=None, prefix=None, causal: bool = True, window: int = 0,
                      scale: Optional[float] = None, softcap: float = 0.0, slopes=None, workspace=None,
                      stream=None) -> None:
    """Attention over packed documents (int32 doc_offsets, one more than the
    documents; None: one document).  scale is 1 / sqrt(head_dim) by default; lse
    (float32, heads x rows) is what the backward pass needs."""
    d, _, _ = _attn_desc(q, k, v, o, lse, doc_offsets, prefix, causal, window, scale, softcap, slopes)
    st = AdamAttnStats()
    _check(lib().adam_attn_plan(ctypes.byref(d), ctypes.byref(st)), "adam_attn_plan")
    on = _On(_one_device(q, k, v, o, lse, doc_offsets, prefix, slopes, workspace), stream)
    with on as s:
        ws, size, owner = _workspace(workspace, st.forward_bytes, on)
        _check(lib().adam_attn_forward(ctypes.byref(d), ws, size, s), "adam_attn_forward")
        del owner


def adam_attn_backward(dout, q, k, v, o, lse, dq, dk, dv, *, doc_offsets=None, prefix=None, causal: bool = True,
                       window: int = 0, scale: Optional[float] = None, softcap: float = 0.0, slopes=None,
                       workspace=None, stream=None) -> None:
    """dq, dk and dv from o and lse as adam_attn_forward left them with the same
    arguments."""
    d, shape, kv_shape = _attn_desc(q, k, v, o, lse, doc_offsets, prefix, causal, window, scale, softcap, slopes)
    d.dout, d.dout_stride, d.dout_head_stride = _heads(dout, "dout", shape, q.dtype)
    d.dq, d.dq_stride, d.dq_head_stride = _heads(dq, "dq", shape, q.dtype)
    d.dk, d.dk_stride, d.dk_head_stride = _heads(dk, "dk", kv_shape, q.dtype)
    d.dv, d.dv_stride, d.dv_head_stride = _heads(dv, "dv", kv_shape, q.dtype)
    st = AdamAttnStats()
    _check(lib().adam_attn_plan(ctypes.byref(d), ctypes.byref(st)), "adam_attn_plan")
    on = _On(_one_device(dout, q, k, v, o, lse, dq, dk, dv, doc_offsets, prefix, slopes, workspace), stream)
    with on as s:
        ws, size, owner = _workspace(workspace, st.backward_bytes, on)
        _check(lib().adam_attn_backward(ctypes.byref(d), ws, size, s), "adam_attn_backward")
        del owner
