"""Decode-step operators, host side: refusals before any launch, and the
oracle's pins. CPU only."""

import ctypes

import numpy as np
import pytest
import torch

import linear_attention_state_chunked_gb300 as L
from oracle import lin_step_oracle as O

FAKE = 0x300000  # never dereferenced by the host-side checks


def cache_desc(layers=2, pages=10, ps=16, H=2, D=128, dt=L.LIN_BF16):
    es = 2 if dt == L.LIN_BF16 else 4
    row = D * es
    return L.KVCacheT(layers, pages, ps, H, D, dt, 0x100000, 0x200000,
                      pages * ps * H * row, ps * H * row, H * row, row)


def append_args(**kw):
    a = L.KVAppendArgsT()
    a.batch, a.n, a.max_pages = 4, 3, 5
    a.k = a.v = a.page_table = a.pos = FAKE
    a.token_stride, a.req_stride, a.page_table_stride = 512, 1536, 5
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attn_args(**kw):
    a = L.AttnArgsT()
    a.batch, a.n_q, a.num_q_heads, a.max_pages, a.out_dtype, a.scale = 4, 3, 8, 5, L.LIN_BF16, 0.1
    a.q = a.out = a.page_table = a.kv_len = FAKE
    a.token_stride, a.req_stride, a.page_table_stride = 2048, 3 * 2048, 5
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def norm_args(**kw):
    a = L.NormArgsT()
    a.rows, a.channels, a.eps, a.scale = 4, 64, 1e-6, 1.0
    a.x_dtype = a.io_dtype = a.h_dtype = L.LIN_BF16
    a.x = a.h_out = FAKE
    a.x_stride = a.gate_stride = a.residual_stride = a.h_stride = a.y_stride = 64
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def refused(rc, code, text):
    assert rc == code, (rc, L.lib.lin_state_last_error())
    assert text in L.lib.lin_state_last_error().decode()


@pytest.mark.parametrize("change,code,text", [
    (dict(num_pages=0), L.LIN_EINVAL, "positive"),
    (dict(page_size=0), L.LIN_EINVAL, "positive"),
    (dict(dtype=7), L.LIN_EINVAL, "dtype"),
    (dict(head_dim=96), L.LIN_EUNSUPPORTED, "head_dim"),
    (dict(k=None), L.LIN_EINVAL, "NULL"),
    (dict(v=0x200008), L.LIN_EINVAL, "aligned"),
    (dict(token_stride=520), L.LIN_EINVAL, "multiples of 16"),
    (dict(head_stride=-256), L.LIN_EINVAL, "non-negative"),
    (dict(head_stride=128), L.LIN_EINVAL, "overlap"),
    (dict(page_stride=4096), L.LIN_EINVAL, "overlap"),
    (dict(layer_stride=8192), L.LIN_EINVAL, "overlap"),
    (dict(page_stride=1 << 62), L.LIN_EINVAL, "range"),
])
def test_cache_descriptor_is_checked_by_both_calls(change, code, text):
    c = cache_desc()
    for k, v in change.items():
        setattr(c, k, v)
    refused(L.lib.lin_state_kv_append(ctypes.byref(c), ctypes.byref(append_args()), None), code, text)
    refused(L.lib.lin_state_attn_decode(ctypes.byref(c), ctypes.byref(attn_args()), None, 0, None), code, text)
    assert L.lib.lin_state_attn_workspace(ctypes.byref(c), ctypes.byref(attn_args())) == 0


def test_heads_first_and_layer_inner_strides_are_accepted():
    """Any nesting of the four axes passes the overlap check (the refusal is
    the next one, a bad layer)."""
    row = 256
    for perm in ((0, 1, 3, 2), (1, 0, 2, 3), (3, 2, 1, 0)):
        c = cache_desc()
        counts = [c.num_layers, c.num_pages, c.page_size, c.num_kv_heads]
        strides, at = [0] * 4, row
        for axis in reversed(perm):
            strides[axis], at = at, at * counts[axis]
        c.layer_stride, c.page_stride, c.token_stride, c.head_stride = strides
        refused(L.lib.lin_state_kv_append(ctypes.byref(c), ctypes.byref(append_args(layer=2)), None),
                L.LIN_EINVAL, "layer 2")


@pytest.mark.parametrize("change,code,text", [
    (dict(layer=2), L.LIN_EINVAL, "layer"),
    (dict(batch=-1), L.LIN_EINVAL, "negative"),
    (dict(n=-1), L.LIN_EINVAL, "negative"),
    (dict(pos=None), L.LIN_EINVAL, "NULL"),
    (dict(k=FAKE + 8), L.LIN_EINVAL, "aligned"),
    (dict(parent=FAKE), L.LIN_EINVAL, "both"),
    (dict(accept_node=FAKE), L.LIN_EINVAL, "both"),
    (dict(parent=FAKE, accept_node=FAKE, n_tok=FAKE), L.LIN_EINVAL, "exclude"),
    (dict(parent=FAKE, accept_node=FAKE, n=33, req_stride=33 * 512), L.LIN_EUNSUPPORTED, "32 drafts"),
    (dict(token_stride=520), L.LIN_EINVAL, "multiples of 16"),
    (dict(token_stride=256), L.LIN_EINVAL, "smaller"),
    (dict(page_table_stride=4), L.LIN_EINVAL, "page_table_stride"),
])
def test_append_refusals(change, code, text):
    c = cache_desc()
    refused(L.lib.lin_state_kv_append(ctypes.byref(c), ctypes.byref(append_args(**change)), None), code, text)


@pytest.mark.parametrize("change,code,text", [
    (dict(layer=-1), L.LIN_EINVAL, "layer"),
    (dict(batch=65536), L.LIN_EINVAL, "batch"),
    (dict(n_q=0), L.LIN_EINVAL, "n_q"),
    (dict(n_q=33), L.LIN_EUNSUPPORTED, "32 query"),
    (dict(num_q_heads=7), L.LIN_EINVAL, "multiple"),
    (dict(out_dtype=3), L.LIN_EINVAL, "out_dtype"),
    (dict(q=None), L.LIN_EINVAL, "NULL"),
    (dict(out=FAKE + 4), L.LIN_EINVAL, "aligned"),
    (dict(token_stride=1024), L.LIN_EINVAL, "smaller"),
    (dict(req_stride=2056), L.LIN_EINVAL, "multiples of 16"),
    (dict(page_table_stride=1), L.LIN_EINVAL, "page_table_stride"),
])
def test_attn_refusals(change, code, text):
    c = cache_desc()
    a = attn_args(**change)
    refused(L.lib.lin_state_attn_decode(ctypes.byref(c), ctypes.byref(a), 0x400000, 1 << 40, None), code, text)


def test_attn_refuses_a_small_workspace():
    c, a = cache_desc(), attn_args()
    need = L.lib.lin_state_attn_workspace(ctypes.byref(c), ctypes.byref(a))
    if need > 0:
        refused(L.lib.lin_state_attn_decode(ctypes.byref(c), ctypes.byref(a), 0x400000, need - 1, None),
                L.LIN_EWORKSPACE, "workspace")
        refused(L.lib.lin_state_attn_decode(ctypes.byref(c), ctypes.byref(a), None, need, None),
                L.LIN_EWORKSPACE, "workspace")
        refused(L.lib.lin_state_attn_decode(ctypes.byref(c), ctypes.byref(a), 0x400008, need, None),
                L.LIN_EINVAL, "aligned")


@pytest.mark.parametrize("change,code,text", [
    (dict(rows=-1), L.LIN_EINVAL, "rows"),
    (dict(channels=0), L.LIN_EINVAL, "channels"),
    (dict(channels=32769), L.LIN_EUNSUPPORTED, "32768"),
    (dict(x_dtype=2), L.LIN_EINVAL, "dtype"),
    (dict(x=None), L.LIN_EINVAL, "NULL"),
    (dict(h_out=None), L.LIN_EINVAL, "NULL"),
    (dict(w_pre=FAKE), L.LIN_EINVAL, "together"),
    (dict(y=FAKE), L.LIN_EINVAL, "together"),
    (dict(w_post=FAKE, group=48), L.LIN_EINVAL, "divide"),
    (dict(w_post=FAKE, group=0), L.LIN_EINVAL, "divide"),
    (dict(gate=FAKE), L.LIN_EINVAL, "gate_act"),
    (dict(gate_act=L.LIN_ACT_SILU), L.LIN_EINVAL, "gate_act"),
    (dict(x_stride=63), L.LIN_EINVAL, "x: row stride"),
    (dict(residual=FAKE, residual_stride=8), L.LIN_EINVAL, "residual: row stride"),
    (dict(h_out=FAKE + 1), L.LIN_EINVAL, "h_out is not aligned"),
    (dict(scale_w=FAKE + 1), L.LIN_EINVAL, "weight"),
])
def test_norm_refusals(change, code, text):
    refused(L.lib.lin_state_block_norm(ctypes.byref(norm_args(**change)), None), code, text)


def test_empty_work_is_a_no_op():
    c = cache_desc()
    assert L.lib.lin_state_kv_append(ctypes.byref(c), ctypes.byref(append_args(batch=0)), None) == 0
    assert L.lib.lin_state_kv_append(ctypes.byref(c), ctypes.byref(append_args(n=0)), None) == 0
    assert L.lib.lin_state_attn_decode(ctypes.byref(c), ctypes.byref(attn_args(batch=0)), None, 0, None) == 0
    assert L.lib.lin_state_block_norm(ctypes.byref(norm_args(rows=0)), None) == 0


def test_binding_refuses_wrong_tensors():
    k = torch.zeros((1, 4, 8, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cache v"):
        L.KVCache(1, 4, 8, 2, 64, k=k, v=torch.zeros((1, 4, 8, 2, 32), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="same strides"):
        L.KVCache(1, 4, 8, 2, 64, k=k, v=torch.zeros((1, 4, 2, 8, 64), dtype=torch.bfloat16).transpose(2, 3))
    c = L.KVCache(1, 4, 8, 2, 64, k=k, v=k.clone())
    i32 = dict(dtype=torch.int32)
    new = torch.zeros((3, 2, 2, 64), dtype=torch.bfloat16)
    table, pos = torch.zeros((3, 4), **i32), torch.zeros(3, **i32)
    with pytest.raises(ValueError, match="k: want"):
        L.lin_state_kv_append(c, layer=0, k=new.float(), v=new, page_table=table, pos=pos)
    with pytest.raises(ValueError, match="same shape"):
        L.lin_state_kv_append(c, layer=0, k=new, v=new[:, :1], page_table=table, pos=pos)
    with pytest.raises(ValueError, match="page_table: want int32"):
        L.lin_state_kv_append(c, layer=0, k=new, v=new, page_table=table[:2], pos=pos)
    with pytest.raises(ValueError, match="want a CUDA tensor"):
        L.lin_state_kv_append(c, layer=0, k=new, v=new, page_table=table, pos=pos)
    q = torch.zeros((3, 2, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="out"):
        L.lin_state_attn_decode(c, layer=0, q=q, out=q[:, :1], page_table=table, kv_len=pos)
    with pytest.raises(ValueError, match="contiguous"):
        L.lin_state_attn_decode(c, layer=0, q=q.transpose(2, 3).contiguous().transpose(2, 3), out=q,
                                page_table=table, kv_len=pos)
    x = torch.zeros((3, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="gate_act"):
        L.lin_state_block_norm(x=x, gate=x, gate_act="relu", h_out=x)
    with pytest.raises(ValueError, match="want a CUDA tensor"):
        L.lin_state_block_norm(x=x, h_out=x)


# ---- the oracle's own pins ---------------------------------------------------

def test_oracle_attention_against_torch_softmax_and_a_planted_mistake():
    g = np.random.default_rng(0)
    B, n, H, G, D, ps = 2, 3, 2, 2, 8, 5
    lens = [11, 7]
    k, v = g.normal(size=(2, 6, ps, H, D))
    table = np.array([[4, 0, 2], [5, 1, 3]])
    q = g.normal(size=(B, n, H * G, D))
    out, reach, _ = O.attn_decode(k, v, q, table, lens, 0.3)
    for r in range(B):
        kk = torch.tensor(k[table[r]].reshape(-1, H, D)[:lens[r]])
        vv = torch.tensor(v[table[r]].reshape(-1, H, D)[:lens[r]])
        mask = torch.ones(n, lens[r], dtype=torch.bool).tril(lens[r] - n)
        for h in range(H * G):
            s = (torch.tensor(q[r, :, h]) @ kk[:, h // G].T * 0.3).masked_fill(~mask, -torch.inf)
            want = torch.softmax(s, -1) @ vv[:, h // G]
            assert np.allclose(out[r, :, h], want.numpy(), rtol=1e-12)
            wrong = torch.softmax(s.nan_to_num(neginf=0.0), -1) @ vv[:, h // G]  # mask forgotten
            assert not np.allclose(out[r, 0, h], wrong[0].numpy(), rtol=1e-3)
    assert (reach >= np.abs(out) - 1e-15).all()


def test_oracle_tree_equals_the_chain_of_its_path():
    g = np.random.default_rng(1)
    k, v = g.normal(size=(2, 4, 4, 1, 8))
    q = g.normal(size=(1, 4, 2, 8))
    parent = [[-1, 0, 0, 2]]
    table, length = np.array([[2, 0, 3]]), 9  # 5 committed tokens, 4 drafts
    tree, _, _ = O.attn_decode(k, v, q, table, [length], 1.0, parent)
    path = O.path_to(parent[0], 3)
    assert path == [0, 2, 3]
    k2, v2 = k.copy(), v.copy()
    rows = [O.locate(table[0], 5 + j, 4, 4) for j in path]
    O.kv_append(k2[:, :], v2, np.stack([k[a] for a in rows])[None], np.stack([v[a] for a in rows])[None],
                table, [5])
    chain, _, _ = O.attn_decode(k2, v2, q[:, path], table, [8], 1.0)
    assert np.allclose(tree[:, path], chain, rtol=1e-12)


def test_oracle_append_path_prefix_and_padding():
    k = np.arange(24.0).reshape(2, 3, 2, 2)
    ck, cv = np.zeros((2, 3, 4, 2, 2))
    table = np.array([[1, 2], [0, -1]])
    O.kv_append(ck, cv, k, -k, table, [3, 4], parent=[[-1, -1, 1]] * 2, accept_node=[2, 2])
    assert (ck[1, 3] == k[0, 1]).all() and (ck[2, 0] == k[0, 2]).all() and (cv == -ck).all()
    assert not ck[0].any()  # request 1: its second page is not allocated
    before = ck.copy()
    O.kv_append(ck, cv, k, -k, table, [-1, 0], n_tok=[3, 0])
    assert (ck == before).all()


def test_oracle_norm_closed_forms():
    x = np.full((1, 8), 3.0)
    _, h, y = O.block_norm(x, w_post=np.full(4, 2.0), residual=np.ones((1, 8)), scale=0.5, w_pre=np.ones(8), eps=0.0)
    assert np.allclose(h, 2.0) and np.allclose(y, 1.0)
    _, h, _ = O.block_norm(x, gate=np.zeros((1, 8)), act="sigmoid")
    assert np.allclose(h, 1.5)
    _, h, _ = O.block_norm(x, gate=np.full((1, 8), 40.0), act="silu")
    assert np.allclose(h, 120.0)
