"""Binding of include/lin_prompt.h: what a prompt, whole or in chunks, needs of a
hybrid model's full-attention layers. Block tables and slot maps from the requests'
lengths, rotary positions with the append to the paged cache, and attention of a
batch's newest tokens over it. Same manner as the decode step's binding: caller's
tensors, the C entry points' names, LinStateError."""

from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import dtype_code, lib
from .step import (KVCache, KVCacheT, _addr, _dt, _entry, _f32, _i32, _i64, _launch_device, _P, _packer, _ptr32, _raise,
                   _status, _stream_of, _table, _vp)

LIN_ST_NO_PAGES = 1024

PROMPT_EXPORTED = ("lin_state_kv_plan", "lin_state_rope", "lin_state_attn_chunk_workspace", "lin_state_attn_chunk")


class KVPlanArgsT(ctypes.Structure):
    _fields_ = [("batch", _i32), ("n", _i32), ("tokens", _i32), ("page_size", _i32), ("num_pages", _i32),
                ("max_pages", _i32), ("num_free", _i32), ("length", _vp), ("n_new", _vp), ("parent", _vp),
                ("page_table", _vp), ("page_table_stride", _i64), ("free_pages", _vp), ("taken", _vp),
                ("cu_seqlens", _vp), ("kv_len", _vp), ("position", _vp), ("slot", _vp), ("status", _vp)]


class RopeArgsT(ctypes.Structure):
    _fields_ = [("layer", _i32), ("tokens", _i32), ("num_q_heads", _i32), ("num_k_heads", _i32),
                ("head_dim", _i32), ("rot_dim", _i32), ("interleaved", _i32), ("dtype", _i32), ("scale", _f32),
                ("q", _vp), ("k", _vp), ("v", _vp), ("q_out", _vp), ("k_out", _vp), ("q_stride", _i64),
                ("k_stride", _i64), ("v_stride", _i64), ("q_out_stride", _i64), ("k_out_stride", _i64),
                ("position", _vp), ("inv_freq", _vp), ("slot", _vp), ("status", _vp)]


class AttnChunkArgsT(ctypes.Structure):
    _fields_ = [("layer", _i32), ("batch", _i32), ("tokens", _i32), ("num_q_heads", _i32), ("out_dtype", _i32),
                ("max_pages", _i32), ("scale", _f32), ("q", _vp), ("token_stride", _i64), ("out", _vp),
                ("page_table", _vp), ("page_table_stride", _i64), ("cu_seqlens", _vp), ("kv_len", _vp),
                ("status", _vp)]


lib.lin_state_kv_plan.argtypes = [_P(KVPlanArgsT), _vp]
lib.lin_state_kv_plan.restype = ctypes.c_int
lib.lin_state_rope.argtypes = [_P(KVCacheT), _P(RopeArgsT), _vp]
lib.lin_state_rope.restype = ctypes.c_int
lib.lin_state_attn_chunk_workspace.argtypes = [_P(KVCacheT), _P(AttnChunkArgsT)]
lib.lin_state_attn_chunk_workspace.restype = ctypes.c_size_t
lib.lin_state_attn_chunk.argtypes = [_P(KVCacheT), _P(AttnChunkArgsT), _vp, ctypes.c_size_t, _vp]
lib.lin_state_attn_chunk.restype = ctypes.c_int

_pack_plan, _pack_rope, _pack_chunk = (_packer(c).pack for c in (KVPlanArgsT, RopeArgsT, AttnChunkArgsT))
_call_plan = _entry("lin_state_kv_plan", ctypes.c_char_p, _vp)
_call_rope = _entry("lin_state_rope", _vp, ctypes.c_char_p, _vp)
_call_chunk = _entry("lin_state_attn_chunk", _vp, ctypes.c_char_p, _vp, ctypes.c_size_t, _vp)


def _slots(t: Optional[torch.Tensor], tokens: int, device: int) -> int:
    if t is None:
        return 0
    if t.dtype is not torch.int64 or t.shape != (tokens,) or not t.is_contiguous():
        raise ValueError(f"slot: want a contiguous int64 tensor ({tokens},), got {tuple(t.shape)} of {t.dtype}")
    return _addr(t, "slot", device)


def lin_state_kv_plan(*, page_size: int, num_pages: int, length, page_table, n_new=None, n: int = 1, parent=None,
                      free_pages=None, tokens: Optional[int] = None, cu_seqlens=None, kv_len=None, position=None,
                      slot=None, taken=None, status=None, stream=None) -> None:
    """Calls lin_state_kv_plan: request r has length[r] cached tokens and gets n_new[r]
    more (or n each, or a draft tree's, parent [B][n]). New pages come from free_pages,
    in request order, into page_table [B][max_pages]; written are cu_seqlens [B+1],
    kv_len [B], position and slot (int64) of every packed token, and taken [1], each
    unless None. `tokens`: rows of the packed arrays (position's or slot's unless given)."""
    if length.dim() != 1:
        raise ValueError(f"length: want [batch], got {tuple(length.shape)}")
    B = length.shape[0]
    if tokens is None:
        t = position if position is not None else slot
        if t is None:
            raise ValueError("tokens: how many packed rows there are, where neither position nor slot says so")
        tokens = t.numel()
    if parent is not None:
        if parent.dim() != 2:
            raise ValueError(f"parent: want [batch][n], got {tuple(parent.shape)}")
        n = parent.shape[1]
    # (a table without entries may have any strides)
    pages, pstride = _table(page_table if page_table.numel() else page_table.new_empty(page_table.shape), B)
    dev = _launch_device(length, "length")
    free = pfree = 0
    if free_pages is not None:
        if free_pages.dim() != 1:
            raise ValueError(f"free_pages: want a vector, got {tuple(free_pages.shape)}")
        free = free_pages.shape[0]
        # an empty list is not none: any address does
        pfree = _ptr32(free_pages, "free_pages", (free,), dev) or length.data_ptr()
    a = _pack_plan(B, n, tokens, page_size, num_pages, pages, free, _ptr32(length, "length", (B,), dev),
                   _ptr32(n_new, "n_new", (B,), dev), _ptr32(parent, "parent", (B, n), dev),
                   _addr(page_table, "page_table", dev), pstride, pfree,
                   _ptr32(taken, "taken", (1,), dev), _ptr32(cu_seqlens, "cu_seqlens", (B + 1,), dev),
                   _ptr32(kv_len, "kv_len", (B,), dev), _ptr32(position, "position", (tokens,), dev),
                   _slots(slot, tokens, dev), _status(status, dev))
    rc = _call_plan(a, _stream_of(stream, dev))
    if rc:
        _raise(rc, "lin_state_kv_plan")


def rope_frequencies(rot_dim: int, base: float = 10000.0, *, linear: Optional[float] = None,
                     ntk: Optional[float] = None, yarn: Optional[float] = None, trained: int = 4096,
                     beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda") -> Tuple[torch.Tensor, float]:
    """inv_freq (fp32 [rot_dim / 2], base^(-2 i / rot_dim)) and scale for lin_state_rope.
    For a context `linear`, `ntk` or `yarn` times as long as trained on (one at most):
    linear: positions divided by the factor. ntk: the base grown so that the slowest
    pair's wave is that much longer and the fastest stays. yarn (Peng et al. 2023, "YaRN"):
    pairs that turn more than beta_fast times in `trained` tokens stay, those that turn
    less than beta_slow times are divided by the factor, between them the share that stays
    grows linearly with the turns, as the paper has it; and cosines and sines are scaled by
    0.1 ln(factor) + 1. Checkpoints trained with a ramp that is linear in the pair's index
    instead (common, and log-linear in the turns: a pair of 5.7 turns keeps 0.50 of its
    frequency there, 0.15 here), or with another scale, need their own inv_freq and scale,
    which lin_state_rope takes as well."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim: want an even number of channels, got {rot_dim}")
    given = [x for x in (linear, ntk, yarn) if x is not None]
    if len(given) > 1 or any(not x >= 1.0 for x in given):
        raise ValueError("linear, ntk, yarn: one factor at most, 1 or more")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    scale = 1.0
    if ntk is not None and rot_dim > 2:
        base = base * ntk ** (rot_dim / (rot_dim - 2))
    f = float(base) ** (-i / rot_dim)
    if linear is not None:
        f = f / linear
    if yarn is not None:
        turns = trained * f / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / yarn)
        scale = 0.1 * math.log(yarn) + 1.0
    return f.to(torch.float32).to(device), scale


def _heads(t: torch.Tensor, name: str, tokens: int, dim: int, dtype, device: int):
    """(address, heads, token stride in bytes) of [T][heads][dim] with a token's heads
    contiguous."""
    shape, s = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != tokens or shape[2] != dim or t.dtype is not dtype:
        raise ValueError(f"{name}: want [{tokens}][heads][{dim}] of {dtype}, got {tuple(shape)} of {t.dtype}")
    if s[2] != 1 or (shape[1] > 1 and s[1] != dim):
        raise ValueError(f"{name}: the heads of a token must be contiguous, got strides {s}")
    return _addr(t, name, device), shape[1], s[0] * (2 if dtype is torch.bfloat16 else 4)


def lin_state_rope(cache: Optional[KVCache] = None, *, position, inv_freq, q=None, k=None, v=None, q_out=None,
                   k_out=None, layer: int = 0, slot=None, scale: float = 1.0, interleaved: bool = False, status=None,
                   stream=None) -> None:
    """Calls lin_state_rope: turns the first 2 inv_freq.numel() channels of every head of
    q and k ([T][heads][head_dim], views of a projection's output do) by the angles
    position[t] inv_freq[i], times `scale`: into q_out and k_out (q and k themselves do),
    and, with a cache, the turned keys and v into its rows slot[t] (int64) of `layer`."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q, k: one at least")
    if x.dim() != 3:
        raise ValueError(f"q, k: want [tokens][heads][head_dim], got {tuple(x.shape)}")
    T, _, D = x.shape
    dt = x.dtype
    dev = _launch_device(x, "q" if q is not None else "k")
    pq, hq, sq = _heads(q, "q", T, D, dt, dev) if q is not None else (0, 0, 0)
    pk, hk, sk = _heads(k, "k", T, D, dt, dev) if k is not None else (0, 0, 0)
    pv = pqo = pko = sv = sqo = sko = 0
    if q_out is not None:
        pqo, h, sqo = _heads(q_out, "q_out", T, D, dt, dev)
        if h != hq:
            raise ValueError(f"q_out: want {hq} heads, as q, got {h}")
    if k_out is not None:
        pko, h, sko = _heads(k_out, "k_out", T, D, dt, dev)
        if h != hk:
            raise ValueError(f"k_out: want {hk} heads, as k, got {h}")
    at = 0
    if cache is not None:
        if k is None or v is None or slot is None:
            raise ValueError("a cache needs k, v and slot")
        pv, h, sv = _heads(v, "v", T, D, dt, dev)
        if h != hk:
            raise ValueError(f"v: want {hk} heads, as k, got {h}")
        _addr(cache._k, "cache", dev)
        at = cache._addr
    if inv_freq.dtype is not torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq: want a contiguous fp32 vector, got {tuple(inv_freq.shape)} of {inv_freq.dtype}")
    a = _pack_rope(layer, T, hq, hk, D, 2 * inv_freq.shape[0], 1 if interleaved else 0, _dt(dt), scale, pq, pk, pv,
                   pqo, pko, sq, sk, sv, sqo, sko, _ptr32(position, "position", (T,), dev),
                   _addr(inv_freq, "inv_freq", dev), _slots(slot, T, dev) if cache is not None else 0,
                   _status(status, dev))
    rc = _call_rope(at, a, _stream_of(stream, dev))
    if rc:
        _raise(rc, "lin_state_rope")


def lin_state_attn_chunk_workspace(cache: KVCache, *, batch: int, tokens: int, num_q_heads: int, max_pages: int,
                                   out_dtype=None) -> int:
    """Bytes of workspace lin_state_attn_chunk needs for these sizes."""
    a = AttnChunkArgsT()
    a.batch, a.tokens, a.num_q_heads, a.max_pages = batch, tokens, num_q_heads, max_pages
    a.out_dtype = dtype_code(out_dtype or cache.dtype)
    return int(lib.lin_state_attn_chunk_workspace(ctypes.byref(cache.desc()), ctypes.byref(a)))


def lin_state_attn_chunk(cache: KVCache, *, layer: int, q, out, page_table, cu_seqlens, kv_len,
                         scale: Optional[float] = None, status=None, workspace: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """Calls lin_state_attn_chunk: q [T][q_heads][head_dim] (a view of a projection's
    output does), packed: request r's rows cu_seqlens[r] .. cu_seqlens[r+1] are its newest
    tokens, each over the kv_len[r] cached ones up to its own; out [T][q_heads][head_dim]
    contiguous. scale: 1/sqrt(head_dim) unless given. `workspace` is a uint8 device
    tensor of at least lin_state_attn_chunk_workspace() bytes (allocated here when
    omitted)."""
    D = cache.head_dim
    if q.dim() != 3:
        raise ValueError(f"q: want [tokens][q_heads][{D}], got {tuple(q.shape)}")
    dev = _launch_device(cache._k, "cache")
    T = q.shape[0]
    pq, Hq, sq = _heads(q, "q", T, D, cache.dtype, dev)
    if out.shape != q.shape or not out.is_contiguous():
        raise ValueError(f"out: want a contiguous tensor {tuple(q.shape)}, got {tuple(out.shape)}")
    if kv_len.dim() != 1:
        raise ValueError(f"kv_len: want [batch], got {tuple(kv_len.shape)}")
    B = kv_len.shape[0]
    pages, pstride = _table(page_table, B)
    a = _pack_chunk(layer, B, T, Hq, _dt(out.dtype), pages, D ** -0.5 if scale is None else scale, pq, sq,
                    _addr(out, "out", dev), _addr(page_table, "page_table", dev), pstride,
                    _ptr32(cu_seqlens, "cu_seqlens", (B + 1,), dev), _ptr32(kv_len, "kv_len", (B,), dev),
                    _status(status, dev))
    if workspace is None:
        need = lin_state_attn_chunk_workspace(cache, batch=B, tokens=T, num_q_heads=Hq, max_pages=pages,
                                              out_dtype=out.dtype)
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:  # from that stream's own memory: it is used there, and freed before it ends
            with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                                   else torch.cuda.ExternalStream(int(stream))):
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if not workspace.is_contiguous():
        raise ValueError(f"workspace: want a contiguous tensor, got strides {workspace.stride()}")
    rc = _call_chunk(cache._addr, a, _addr(workspace, "workspace", dev), workspace.numel() * workspace.element_size(),
                     _stream_of(stream, dev))
    if rc:
        _raise(rc, "lin_state_attn_chunk")
