"""Binding of include/lin_step.h: the rest of a hybrid model's decode step
beside the linear-attention state path. A paged key-value cache with its append
and decode attention, and the norms around a block. Same manner as the state
path's binding: caller's tensors, the C entry points' names, LinStateError."""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _check, _stream, dtype_code, lib

LIN_ST_BAD_PAGE = 512
LIN_ACT_NONE, LIN_ACT_SILU, LIN_ACT_SIGMOID = 0, 1, 2
_ACTS = {None: LIN_ACT_NONE, "silu": LIN_ACT_SILU, "sigmoid": LIN_ACT_SIGMOID}

STEP_EXPORTED = ("lin_state_kv_append", "lin_state_attn_workspace", "lin_state_attn_decode",
                 "lin_state_block_norm")

_i32, _i64, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class KVCacheT(ctypes.Structure):
    _fields_ = [("num_layers", _i32), ("num_pages", _i32), ("page_size", _i32),
                ("num_kv_heads", _i32), ("head_dim", _i32), ("dtype", _i32),
                ("k", _vp), ("v", _vp),
                ("layer_stride", _i64), ("page_stride", _i64), ("token_stride", _i64),
                ("head_stride", _i64)]


class KVAppendArgsT(ctypes.Structure):
    _fields_ = [("layer", _i32), ("batch", _i32), ("n", _i32), ("max_pages", _i32),
                ("k", _vp), ("v", _vp), ("req_stride", _i64), ("token_stride", _i64),
                ("page_table", _vp), ("page_table_stride", _i64), ("pos", _vp), ("n_tok", _vp),
                ("parent", _vp), ("accept_node", _vp), ("status", _vp)]


class AttnArgsT(ctypes.Structure):
    _fields_ = [("layer", _i32), ("batch", _i32), ("n_q", _i32), ("num_q_heads", _i32),
                ("out_dtype", _i32), ("max_pages", _i32), ("scale", _f32),
                ("q", _vp), ("req_stride", _i64), ("token_stride", _i64), ("out", _vp),
                ("page_table", _vp), ("page_table_stride", _i64), ("kv_len", _vp),
                ("parent", _vp), ("status", _vp)]


class NormArgsT(ctypes.Structure):
    _fields_ = [("rows", _i64), ("channels", _i32), ("group", _i32), ("x_dtype", _i32),
                ("io_dtype", _i32), ("h_dtype", _i32), ("gate_act", _i32), ("eps", _f32),
                ("scale", _f32), ("x", _vp), ("gate", _vp), ("w_post", _vp), ("residual", _vp),
                ("scale_w", _vp), ("w_pre", _vp), ("h_out", _vp), ("y", _vp), ("x_stride", _i64),
                ("gate_stride", _i64), ("residual_stride", _i64), ("h_stride", _i64),
                ("y_stride", _i64)]


_P = ctypes.POINTER
lib.lin_state_kv_append.argtypes = [_P(KVCacheT), _P(KVAppendArgsT), _vp]
lib.lin_state_kv_append.restype = ctypes.c_int
lib.lin_state_attn_workspace.argtypes = [_P(KVCacheT), _P(AttnArgsT)]
lib.lin_state_attn_workspace.restype = ctypes.c_size_t
lib.lin_state_attn_decode.argtypes = [_P(KVCacheT), _P(AttnArgsT), _vp, ctypes.c_size_t, _vp]
lib.lin_state_attn_decode.restype = ctypes.c_int
lib.lin_state_block_norm.argtypes = [_P(NormArgsT), _vp]
lib.lin_state_block_norm.restype = ctypes.c_int


class KVCache:
    """The paged key-value cache: k, v torch tensors [layers][pages][page_size]
    [kv_heads][head_dim], allocated here (zeros) or given as views of any
    16-byte-multiple strides with head_dim contiguous (heads-first pages:
    permute). A request's token t lies in page page_table[r][t // page_size]."""

    def __init__(self, num_layers: int, num_pages: int, page_size: int, num_kv_heads: int,
                 head_dim: int, dtype=torch.bfloat16, device="cuda",
                 k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None):
        shape = (num_layers, num_pages, page_size, num_kv_heads, head_dim)
        if k is None:
            k = torch.zeros(shape, dtype=dtype, device=device)
        if v is None:
            v = torch.zeros(shape, dtype=dtype, device=device)
        for name, t in (("k", k), ("v", v)):
            if tuple(t.shape) != shape or t.dtype != dtype or t.stride(4) != 1:
                raise ValueError(f"cache {name}: want {shape} of {dtype} with head_dim contiguous, "
                                 f"got {tuple(t.shape)} of {t.dtype}, strides {t.stride()}")
        if k.stride() != v.stride():
            raise ValueError(f"cache: k and v must have the same strides, got {k.stride()} and {v.stride()}")
        self.k, self.v, self.dtype = k, v, dtype
        self.num_layers, self.num_pages, self.page_size = num_layers, num_pages, page_size
        self.num_kv_heads, self.head_dim = num_kv_heads, head_dim

    def desc(self) -> KVCacheT:
        k, v = self.k, self.v
        es = k.element_size()
        s = k.stride()
        return KVCacheT(self.num_layers, self.num_pages, self.page_size, self.num_kv_heads,
                        self.head_dim, dtype_code(k.dtype), k.data_ptr(), v.data_ptr(),
                        s[0] * es, s[1] * es, s[2] * es, s[3] * es)


def _ptr32(t: Optional[torch.Tensor], name: str, shape):
    """Address of a contiguous int32 tensor of this shape, or None."""
    if t is None:
        return None
    if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name}: want a contiguous int32 tensor {shape}, got {tuple(t.shape)} of {t.dtype}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, heads: int, dim: int, dtype):
    """[B][n][heads][dim] with the heads of a token contiguous."""
    if t.dim() != 4 or t.shape[2] != heads or t.shape[3] != dim or t.dtype != dtype:
        raise ValueError(f"{name}: want [batch][n][{heads}][{dim}] of {dtype}, got {tuple(t.shape)} of {t.dtype}")
    s = t.stride()
    if s[3] != 1 or (heads > 1 and s[2] != dim):
        raise ValueError(f"{name}: the heads of a token must be contiguous, got strides {s}")
    return s


def _table(t: torch.Tensor, batch: int):
    if t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != batch or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"page_table: want int32 [{batch}][max_pages] with contiguous rows, got "
                         f"{tuple(t.shape)} of {t.dtype}")
    return t.shape[1], t.stride(0)


def lin_state_kv_append(cache: KVCache, *, layer: int, k, v, page_table, pos, n_tok=None,
                        parent=None, accept_node=None, status=None, stream=None) -> None:
    """Calls lin_state_kv_append: the new rows k, v [B][n][kv_heads][head_dim]
    (views of a projection's output do) go to token positions from pos[r] on:
    all n, the first n_tok[r], or the accepted path of a draft tree (parent
    [B][n], accept_node [B])."""
    H, D = cache.num_kv_heads, cache.head_dim
    s = _rows(k, "k", H, D, cache.dtype)
    if _rows(v, "v", H, D, cache.dtype) != s or v.shape != k.shape:
        raise ValueError("k and v must have the same shape and strides")
    B, n = k.shape[0], k.shape[1]
    es = k.element_size()
    pages, pstride = _table(page_table, B)
    a = KVAppendArgsT(layer, B, n, pages, k.data_ptr(), v.data_ptr(), s[0] * es, s[1] * es,
                      page_table.data_ptr(), pstride, _ptr32(pos, "pos", (B,)),
                      _ptr32(n_tok, "n_tok", (B,)), _ptr32(parent, "parent", (B, n)),
                      _ptr32(accept_node, "accept_node", (B,)),
                      None if status is None else status.data_ptr())
    _check(lib.lin_state_kv_append(ctypes.byref(cache.desc()), ctypes.byref(a), _stream(stream)),
           "lin_state_kv_append")


def lin_state_attn_workspace(cache: KVCache, *, batch: int, n_q: int, num_q_heads: int,
                             max_pages: int, out_dtype=None) -> int:
    """Bytes of workspace lin_state_attn_decode needs for these sizes."""
    a = AttnArgsT()
    a.batch, a.n_q, a.num_q_heads, a.max_pages = batch, n_q, num_q_heads, max_pages
    a.out_dtype = dtype_code(out_dtype or cache.dtype)
    return int(lib.lin_state_attn_workspace(ctypes.byref(cache.desc()), ctypes.byref(a)))


def lin_state_attn_decode(cache: KVCache, *, layer: int, q, out, page_table, kv_len,
                          scale: Optional[float] = None, parent=None, status=None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Calls lin_state_attn_decode: q [B][n_q][q_heads][head_dim] (a view of a
    projection's output does), the n_q newest tokens of each request, over its
    kv_len[r] cached tokens, those n_q included; out [B][n_q][q_heads][head_dim]
    contiguous. scale: 1/sqrt(head_dim) unless given. parent [B][n_q]: a draft
    tree. `workspace` is a uint8 device tensor of at least
    lin_state_attn_workspace() bytes (allocated here when omitted)."""
    D = cache.head_dim
    if q.dim() != 4:
        raise ValueError(f"q: want [batch][n_q][q_heads][{D}], got {tuple(q.shape)}")
    B, n, Hq, _ = q.shape
    s = _rows(q, "q", Hq, D, cache.dtype)
    if out.shape != q.shape or not out.is_contiguous():
        raise ValueError(f"out: want a contiguous tensor {tuple(q.shape)}, got {tuple(out.shape)}")
    es = q.element_size()
    pages, pstride = _table(page_table, B)
    a = AttnArgsT(layer, B, n, Hq, dtype_code(out.dtype), pages,
                  D ** -0.5 if scale is None else scale, q.data_ptr(), s[0] * es, s[1] * es,
                  out.data_ptr(), page_table.data_ptr(), pstride, _ptr32(kv_len, "kv_len", (B,)),
                  _ptr32(parent, "parent", (B, n)), None if status is None else status.data_ptr())
    d = cache.desc()
    if workspace is None:
        need = int(lib.lin_state_attn_workspace(ctypes.byref(d), ctypes.byref(a)))
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            if stream is not None:  # freed here while the launch on `stream` may still run
                workspace.record_stream(stream if isinstance(stream, torch.cuda.Stream)
                                        else torch.cuda.ExternalStream(int(stream)))
    ptr, size = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                     workspace.numel() * workspace.element_size())
    _check(lib.lin_state_attn_decode(ctypes.byref(d), ctypes.byref(a), ptr, size, _stream(stream)),
           "lin_state_attn_decode")


def lin_state_block_norm(*, x, gate=None, gate_act: Optional[str] = None, w_post=None,
                         residual=None, scale: float = 1.0, scale_w=None, w_pre=None,
                         h_out=None, y=None, eps: float = 1e-6, stream=None) -> None:
    """Calls lin_state_block_norm on rows [T][C] (any row strides):
    t = x, normed over groups of w_post.numel() channels, times act(gate)
    ("silu" / "sigmoid"); h_out = residual + scale * scale_w * t;
    y = the norm of h over the row, times w_pre. Every part but x is optional."""
    if x.dim() != 2:
        raise ValueError(f"x: want [rows][channels], got {tuple(x.shape)}")
    T, C = x.shape
    if gate_act not in _ACTS:
        raise ValueError(f"gate_act: want None, 'silu' or 'sigmoid', got {gate_act!r}")
    io = hd = None
    ptr, stride = [], []
    for name, t in (("x", x), ("gate", gate), ("residual", residual), ("h_out", h_out), ("y", y)):
        if t is None:
            ptr.append(None)
            stride.append(0)
            continue
        if t.shape != x.shape or (C > 1 and t.stride(1) != 1):
            raise ValueError(f"{name}: want [{T}][{C}] with contiguous rows, got {tuple(t.shape)}, "
                             f"strides {t.stride()}")
        if name in ("gate", "y"):
            if io is not None and t.dtype != io:
                raise ValueError(f"gate, the weights and y must have one dtype, got {io} and {t.dtype}")
            io = t.dtype
        elif name != "x":
            if hd is not None and t.dtype != hd:
                raise ValueError(f"residual and h_out must have one dtype, got {hd} and {t.dtype}")
            hd = t.dtype
        ptr.append(t.data_ptr())
        stride.append(t.stride(0))
    weights = []
    for name, w in (("w_post", w_post), ("scale_w", scale_w), ("w_pre", w_pre)):
        if w is None:
            weights.append(None)
            continue
        if w.dim() != 1 or not w.is_contiguous() or (name != "w_post" and w.numel() != C):
            raise ValueError(f"{name}: want a contiguous vector"
                             f"{'' if name == 'w_post' else f' of {C}'}, got {tuple(w.shape)}")
        if io is not None and w.dtype != io:
            raise ValueError(f"gate, the weights and y must have one dtype, got {io} and {w.dtype}")
        io = w.dtype
        weights.append(w.data_ptr())
    a = NormArgsT(T, C, w_post.numel() if w_post is not None else 0, dtype_code(x.dtype),
                  dtype_code(io or x.dtype), dtype_code(hd or x.dtype), _ACTS[gate_act], eps, scale,
                  ptr[0], ptr[1], weights[0], ptr[2], weights[1], weights[2], ptr[3], ptr[4], *stride)
    _check(lib.lin_state_block_norm(ctypes.byref(a), _stream(stream)), "lin_state_block_norm")
