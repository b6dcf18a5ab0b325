"""Binding of include/lin_step.h: the rest of a hybrid model's decode step
beside the linear-attention state path. A paged key-value cache with its append
and decode attention, and the norms around a block. Same manner as the state
path's binding: caller's tensors, the C entry points' names, LinStateError."""

from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch

from . import LIN_BF16, LIN_F32, LinStateError, dtype_code, lib

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


# A decode step makes these calls once per layer, so what a call costs on the
# host counts: the argument structures are packed in one go (a ctypes Structure
# of 20 fields takes several times as long) and handed over as bytes.
_CODE = {"c_int": "i", "c_long": "q", "c_longlong": "q", "c_void_p": "P", "c_float": "f"}


def _packer(cls) -> struct.Struct:
    p = struct.Struct("@" + "".join(_CODE[t.__name__] for _, t in cls._fields_))
    assert p.size <= ctypes.sizeof(cls) < p.size + 8  # tail padding alone may differ
    return struct.Struct(p.format + f"{ctypes.sizeof(cls) - p.size}x")


_pack_append, _pack_attn, _pack_norm = (_packer(c).pack for c in (KVAppendArgsT, AttnArgsT, NormArgsT))


def _entry(name, *argtypes):
    f = lib[name]  # a handle of its own, with these argument types
    f.argtypes, f.restype = argtypes, ctypes.c_int
    return f


_call_append = _entry("lin_state_kv_append", _vp, ctypes.c_char_p, _vp)
_call_attn = _entry("lin_state_attn_decode", _vp, ctypes.c_char_p, _vp, ctypes.c_size_t, _vp)
_call_norm = _entry("lin_state_block_norm", ctypes.c_char_p, _vp)
# the current stream's handle without the object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = torch.cuda.current_device


def _stream_of(stream, device: int):
    """The given stream's handle, or that of the device's current stream."""
    if stream is None:
        return _raw_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


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
        if k.device != v.device:
            raise ValueError(f"cache: k and v must lie on one device, got {k.device} and {v.device}")
        self._k, self._v, self.dtype = k, v, dtype
        self.num_layers, self.num_pages, self.page_size = num_layers, num_pages, page_size
        self.num_kv_heads, self.head_dim = num_kv_heads, head_dim

        es, st = k.element_size(), k.stride()
        self._desc = KVCacheT(num_layers, num_pages, page_size, num_kv_heads, head_dim,
                              dtype_code(dtype), k.data_ptr(), v.data_ptr(),
                              st[0] * es, st[1] * es, st[2] * es, st[3] * es)
        self._addr = ctypes.addressof(self._desc)

    @property
    def k(self) -> torch.Tensor:
        return self._k

    @property
    def v(self) -> torch.Tensor:
        return self._v

    def desc(self) -> KVCacheT:
        return self._desc


_DT = {torch.float32: LIN_F32, torch.bfloat16: LIN_BF16}


def _dt(dtype) -> int:
    code = _DT.get(dtype)
    return dtype_code(dtype) if code is None else code  # raises


def _raise(rc: int, where: str):
    raise LinStateError(rc, where)


def _launch_device(t: torch.Tensor, name: str) -> int:
    """The GPU of t, on which the call's other tensors have to lie too. Kernels
    are launched on the current device, which it therefore has to be."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name}: want a CUDA tensor, got one on {t.device}")
    if device != _current_device():
        raise ValueError(f"{name}: lies on cuda:{device}, which is not the current device (cuda:{_current_device()})")
    return device


def _addr(t: torch.Tensor, name: str, device: int) -> int:
    if t.get_device() != device:
        raise ValueError(f"{name}: want a CUDA tensor on cuda:{device}, got one on {t.device}")
    return t.data_ptr()


def _ptr32(t: Optional[torch.Tensor], name: str, shape, device: int) -> int:
    """Address of a contiguous int32 tensor of this shape, or 0 for None."""
    if t is None:
        return 0
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: want a contiguous int32 tensor {shape}, got {tuple(t.shape)} of {t.dtype}")
    return _addr(t, name, device)


def _status(t: Optional[torch.Tensor], device: int) -> int:
    """Address of the status word, or 0 for None."""
    if t is None:
        return 0
    if t.dtype is not torch.int32 or t.numel() < 1:
        raise ValueError(f"status: want an int32 tensor of one word, got {tuple(t.shape)} of {t.dtype}")
    return _addr(t, "status", device)


def _rows(t: torch.Tensor, name: str, heads: int, dim: int, dtype):
    """Shape and strides of [B][n][heads][dim] with a token's heads contiguous."""
    shape = t.shape
    if len(shape) != 4 or shape[2] != heads or shape[3] != dim or t.dtype is not dtype:
        raise ValueError(f"{name}: want [batch][n][{heads}][{dim}] of {dtype}, got {tuple(shape)} of {t.dtype}")
    s = t.stride()
    if s[3] != 1 or (heads > 1 and s[2] != dim):
        raise ValueError(f"{name}: the heads of a token must be contiguous, got strides {s}")
    return shape, s


def _table(t: torch.Tensor, batch: int):
    shape, s = t.shape, t.stride()
    if t.dtype is not torch.int32 or len(shape) != 2 or shape[0] != batch or (shape[1] > 1 and s[1] != 1):
        raise ValueError(f"page_table: want int32 [{batch}][max_pages] with contiguous rows, got "
                         f"{tuple(shape)} of {t.dtype}")
    return shape[1], s[0]


def lin_state_kv_append(cache: KVCache, *, layer: int, k, v, page_table, pos, n_tok=None,
                        parent=None, accept_node=None, status=None, stream=None) -> None:
    """Calls lin_state_kv_append: the new rows k, v [B][n][kv_heads][head_dim]
    (views of a projection's output do) go to token positions from pos[r] on:
    all n, the first n_tok[r], or the accepted path of a draft tree (parent
    [B][n], accept_node [B])."""
    H, D = cache.num_kv_heads, cache.head_dim
    shape, s = _rows(k, "k", H, D, cache.dtype)
    vshape, vs = _rows(v, "v", H, D, cache.dtype)
    if vs != s or vshape != shape:
        raise ValueError("k and v must have the same shape and strides")
    B, n = shape[0], shape[1]
    es = 2 if cache.dtype is torch.bfloat16 else 4
    pages, pstride = _table(page_table, B)
    dev = _launch_device(cache._k, "cache")
    a = _pack_append(layer, B, n, pages, _addr(k, "k", dev), _addr(v, "v", dev), s[0] * es, s[1] * es,
                     _addr(page_table, "page_table", dev), pstride,
                     _ptr32(pos, "pos", (B,), dev), _ptr32(n_tok, "n_tok", (B,), dev),
                     _ptr32(parent, "parent", (B, n), dev), _ptr32(accept_node, "accept_node", (B,), dev),
                     _status(status, dev))
    rc = _call_append(cache._addr, a, _stream_of(stream, dev))
    if rc:
        _raise(rc, "lin_state_kv_append")


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
    shape, s = _rows(q, "q", q.shape[2], D, cache.dtype)
    B, n, Hq, _ = shape
    if out.shape != shape or not out.is_contiguous():
        raise ValueError(f"out: want a contiguous tensor {tuple(shape)}, got {tuple(out.shape)}")
    es = 2 if cache.dtype is torch.bfloat16 else 4
    pages, pstride = _table(page_table, B)
    dev = _launch_device(cache._k, "cache")
    a = _pack_attn(layer, B, n, Hq, _dt(out.dtype), pages, D ** -0.5 if scale is None else scale,
                   _addr(q, "q", dev), s[0] * es, s[1] * es, _addr(out, "out", dev),
                   _addr(page_table, "page_table", dev), pstride,
                   _ptr32(kv_len, "kv_len", (B,), dev), _ptr32(parent, "parent", (B, n), dev), _status(status, dev))
    if workspace is None:
        need = lin_state_attn_workspace(cache, batch=B, n_q=n, num_q_heads=Hq, max_pages=pages,
                                        out_dtype=out.dtype)
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:  # from that stream's own memory: it is used there, and freed before it ends
            with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                                   else torch.cuda.ExternalStream(int(stream))):
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if not workspace.is_contiguous():
        raise ValueError(f"workspace: want a contiguous tensor, got strides {workspace.stride()}")
    rc = _call_attn(cache._addr, a, _addr(workspace, "workspace", dev), workspace.numel() * workspace.element_size(),
                    _stream_of(stream, dev))
    if rc:
        _raise(rc, "lin_state_attn_decode")


def _norm_row(t, name: str, shape, dtype, device: int):
    """(address, row stride, dtype) of a [T][C] tensor, or of None."""
    if t is None:
        return 0, 0, dtype
    s = t.stride()
    if t.shape != shape or (s[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name}: want {list(shape)} with contiguous rows, got {tuple(t.shape)}, strides {s}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name}: gate, the weights and y must have one dtype, and residual and h_out "
                         f"one: got {t.dtype} beside {dtype}")
    return _addr(t, name, device), s[0], t.dtype


def _norm_weight(w, name: str, channels: Optional[int], dtype, device: int):
    if w is None:
        return 0, dtype
    if w.dim() != 1 or not w.is_contiguous() or (channels is not None and w.shape[0] != channels):
        raise ValueError(f"{name}: want a contiguous vector{'' if channels is None else f' of {channels}'}, "
                         f"got {tuple(w.shape)}")
    if dtype is not None and w.dtype is not dtype:
        raise ValueError(f"{name}: gate, the weights and y must have one dtype, got {w.dtype} beside {dtype}")
    return _addr(w, name, device), w.dtype


def lin_state_block_norm(*, x, gate=None, gate_act: Optional[str] = None, w_post=None,
                         residual=None, scale: float = 1.0, scale_w=None, w_pre=None,
                         h_out=None, y=None, eps: float = 1e-6, stream=None) -> None:
    """Calls lin_state_block_norm on rows [T][C] (any row strides):
    t = x, normed over groups of w_post.numel() channels, times act(gate)
    ("silu" / "sigmoid"); h_out = residual + scale * scale_w * t;
    y = the norm of h over the row, times w_pre. Every part but x is optional."""
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x: want [rows][channels], got {tuple(shape)}")
    T, C = shape
    act = _ACTS.get(gate_act)
    if act is None:
        raise ValueError(f"gate_act: want None, 'silu' or 'sigmoid', got {gate_act!r}")
    dev = _launch_device(x, "x")
    px, sx, xd = _norm_row(x, "x", shape, None, dev)
    pg, sg, io = _norm_row(gate, "gate", shape, None, dev)
    py, sy, io = _norm_row(y, "y", shape, io, dev)
    pr, sr, hd = _norm_row(residual, "residual", shape, None, dev)
    ph, sh, hd = _norm_row(h_out, "h_out", shape, hd, dev)
    pw, io = _norm_weight(w_post, "w_post", None, io, dev)
    ps, io = _norm_weight(scale_w, "scale_w", C, io, dev)
    pp, io = _norm_weight(w_pre, "w_pre", C, io, dev)
    a = _pack_norm(T, C, w_post.shape[0] if w_post is not None else 0, _dt(xd), _dt(io or xd), _dt(hd or xd),
                   act, eps, scale, px, pg, pw, pr, ps, pp, ph, py, sx, sg, sr, sh, sy)
    rc = _call_norm(a, _stream_of(stream, dev))
    if rc:
        _raise(rc, "lin_state_block_norm")
