"""Prompt operators on the GPU against the fp64 oracle: block tables and slot maps,
rotary positions with the append, and attention of packed new tokens.

Tolerances are per element. A stored output is off by at most half a step of its type,
eps / 2 of its value, and inside the sums fp32 rounds by u = 2^-24.
Rotary positions: cosine and sine are off by up to 2^-22 = 4 u and scaled with one more
rounding; two products and a sum: |out - want| <= eps/2 |want| + 8 u scale (|x| + |y|).
Attention: a score of D products is off by at most (D + 16) u S, S = scale sum |q k|,
which moves its weight by that share; so do the maximum and the exponential; the weights'
sum and the sum over L values round at most L + 16 times; bf16 outputs of a bf16 cache
take weights rounded to bf16 (2^-8 of each at most), fp32 outputs in three parts (2^-24),
an fp32 cache's products two tf32 parts (three terms of 2^-22). So
|out - want| <= eps/2 |want| + reach (2 S (D + 16 + c) u + (L + 16) u + d)
with reach = sum p |v|."""

import numpy as np
import pytest
import torch

import linear_attention_state_chunked_gb300 as L
from oracle import lin_prompt_oracle as O
from tests.helpers import np64
from tests.test_gpu_step import half_step, make_cache

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


# ---- block tables and slot maps ----------------------------------------------------------

def check_plan(length, n_new, ps, tokens, table, num_pages, free=None, parent=None, want_status=None):
    B = len(length)
    dev = dict(device="cuda")
    t = i32(table)
    out = dict(cu_seqlens=torch.full((B + 1,), 7, dtype=torch.int32, **dev),
               kv_len=torch.full((B,), 7, dtype=torch.int32, **dev),
               position=torch.full((tokens,), 7, dtype=torch.int32, **dev),
               slot=torch.full((tokens,), 7, dtype=torch.int64, **dev),
               taken=torch.full((1,), 7, dtype=torch.int32, **dev))
    status = torch.zeros(1, dtype=torch.int32, **dev)
    L.lin_state_kv_plan(page_size=ps, num_pages=num_pages, length=i32(length),
                        n_new=None if parent is not None else i32(n_new), page_table=t,
                        free_pages=None if free is None else i32(free),
                        parent=None if parent is None else i32(parent), status=status, **out)
    w_table, w_taken, w_cu, w_len, w_pos, w_slot, w_status = O.kv_plan(length, n_new, table, ps, num_pages, tokens,
                                                                        free, parent)
    assert L.lin_state_read_status(status) == w_status
    if want_status is not None:
        assert w_status == want_status
    assert np.array_equal(t.cpu(), w_table)
    assert int(out["taken"]) == w_taken
    assert np.array_equal(out["cu_seqlens"].cpu(), w_cu)
    assert np.array_equal(out["kv_len"].cpu(), w_len)
    assert np.array_equal(out["position"].cpu(), w_pos)
    assert np.array_equal(out["slot"].cpu(), w_slot)
    return out, t


def plan_batch(rng, B, ps, n_hi, c_hi, spare=2):
    length = rng.integers(0, c_hi + 1, B)
    n_new = rng.integers(0, n_hi + 1, B)
    wide = -(-(c_hi + n_hi) // ps) + 1
    table = np.full((B, wide), -1)
    at = 0
    for r in range(B):
        k = -(-int(length[r]) // ps)
        table[r, :k] = at + np.arange(k)
        at += k
    need = sum(-(-int(c + n) // ps) - -(-int(c) // ps) for c, n in zip(length, n_new))
    pages = at + need + spare
    free = at + rng.permutation(need + spare)
    return length, n_new, table, pages, free


@pytest.mark.parametrize("ps", [1, 7, 16, 64])
@pytest.mark.parametrize("B,n_hi,c_hi", [(1, 1, 5), (1, 5000, 100), (3, 40, 40), (70, 200, 500), (600, 9, 50),
                                         (3000, 1, 64)])
def test_plan_ragged_batches(ps, B, n_hi, c_hi):
    rng = np.random.default_rng(B * ps)
    length, n_new, table, pages, free = plan_batch(rng, B, ps, n_hi, c_hi)
    length[rng.random(B) < 0.1] = -1  # padding
    total = int(n_new[length >= 0].sum())
    check_plan(length, n_new, ps, total + 13, table, pages, free, want_status=0)


def test_plan_no_tokens_and_no_requests():
    check_plan([5, 0, -1], [0, 0, 4], 4, 0, [[1, 2], [-1, -1], [-1, -1]], 8, [3, 4], want_status=0)
    check_plan([5, 0], [0, 0], 4, 3, [[1, 2], [-1, -1]], 8, [], want_status=0)
    check_plan([5, 0], [3, 1], 4, 4, [[1, 2], [-1, -1]], 8, [], want_status=O.NO_PAGES)
    check_plan([], [], 4, 3, np.zeros((0, 2), int), 8, [3], want_status=0)


def test_plan_tables_that_hold_the_pages_already():
    """No list: the table is read, not written, and its missing pages are told."""
    table = np.array([[4, 2, 0], [1, 5, -1], [9, 3, 3]])
    check_plan([3, 6, 0], [5, 2, 1], 4, 9, table, 6, want_status=O.BAD_PAGE)


@pytest.mark.parametrize("n", [1, 2, 8, 32])
def test_plan_draft_trees(n):
    """Positions by depth, cache rows by draft; one request's tree breaks the rules."""
    rng = np.random.default_rng(n)
    B, ps = 9, 16
    length, _, table, pages, free = plan_batch(rng, B, ps, 0, 70, spare=40)
    table = np.concatenate([table, np.full((B, 3), -1)], 1)
    parent = [[int(rng.integers(max(-1, j - 4), j)) for j in range(n)] for _ in range(B)]
    check_plan(length, [n] * B, ps, n * B + 5, table, pages, free, parent=parent, want_status=0)
    parent[4][n - 1] = n - 1
    check_plan(length, [n] * B, ps, n * B, table, pages, free, parent=parent, want_status=O.BAD_TREE)


def test_plan_leaves_requests_out():
    """Counts below zero, too many tokens for the table, rows past the end, pages that
    run short: the others go on, and packed rows keep their places."""
    table = np.full((6, 4), -1)
    free = list(range(10, 19))
    check_plan([0, 0, 0, 0, 0, 0], [5, -3, 17, 8, 4, 4], 4, 60, table, 30, free, want_status=O.BAD_SEQLEN)
    check_plan([0] * 6, [5, 3, 9, 8, 4, 4], 4, 20, table, 30, free, want_status=O.BAD_SEQLEN)
    check_plan([0] * 6, [5, 3, 16, 8, 4, 0], 4, 60, table, 30, free, want_status=O.NO_PAGES)
    check_plan([0] * 3, [5, 3, 9], 4, 60, table[:3], 30, [3, 50, 4, -1, 5, 6], want_status=O.BAD_PAGE)


def test_plan_optional_outputs_and_a_strided_table():
    wide = torch.full((3, 10), 77, dtype=torch.int32, device="cuda")
    table = wide[:, 2:6]
    slot = torch.zeros(9, dtype=torch.int64, device="cuda")
    L.lin_state_kv_plan(page_size=2, num_pages=20, length=i32([0, 0, 0]), n=3, page_table=table,
                        free_pages=i32(range(5, 15)), slot=slot)
    assert table[:, :2].tolist() == [[5, 6], [7, 8], [9, 10]] and (table[:, 2:] == 77).all()
    assert (wide[:, :2] == 77).all() and (wide[:, 6:] == 77).all()
    assert slot.tolist() == [10, 11, 12, 14, 15, 16, 18, 19, 20]
    L.lin_state_kv_plan(page_size=2, num_pages=20, length=i32([0, 0, 0]), n=3, page_table=table, tokens=9,
                        free_pages=i32(range(15, 5, -1)))
    assert table[:, :2].tolist() == [[15, 14], [13, 12], [11, 10]]


# ---- rotary positions -----------------------------------------------------------------------

def check_rope(T, Hq, Hk, D, rot, dtype, interleaved, far, seed, scale=1.0, hnd=False, ps=5, in_place=False,
               to_cache=True, base=1e4):
    gen = torch.Generator().manual_seed(seed)
    rows = torch.randn((T, Hq + 2 * Hk, D), generator=gen).to(dtype).cuda()
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:]
    position = torch.randint(far, (T,), generator=gen, dtype=torch.int32)
    position[torch.rand(T, generator=gen) < 0.1] = -1
    pages = -(-T // ps) + 1
    slot = torch.randperm(pages * ps, generator=gen)[:T]
    slot[torch.rand(T, generator=gen) < 0.1] = -1
    inv = (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float()
    cache = None
    if to_cache:
        shape = (2, pages, Hk, ps, D) if hnd else (2, pages, ps, Hk, D)
        kv = [torch.full(shape, 3.0, dtype=dtype, device="cuda") for _ in range(2)]
        kv = [x.transpose(2, 3) for x in kv] if hnd else kv
        cache = L.KVCache(2, pages, ps, Hk, D, dtype=dtype, k=kv[0], v=kv[1])
    want_q, reach_q = O.rope(np64(q), position.numpy(), inv.numpy(), scale, interleaved)
    want_k, reach_k = O.rope(np64(k), position.numpy(), inv.numpy(), scale, interleaved)
    before = rows.clone()
    q_out = q if in_place else torch.full((T, Hq, D), 9.0, dtype=dtype, device="cuda")
    k_out = k if in_place else torch.full((T, Hk, D), 9.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lin_state_rope(cache, layer=1 if to_cache else 0, q=q, k=k, v=v if to_cache else None, q_out=q_out, k_out=k_out,
                     position=position.cuda(), inv_freq=inv.cuda(), slot=slot.cuda() if to_cache else None,
                     scale=scale, interleaved=interleaved, status=status)
    assert L.lin_state_read_status(status) == 0
    live = (position >= 0).numpy()
    for got, want, reach, at in ((q_out, want_q, reach_q, slice(0, Hq)), (k_out, want_k, reach_k, slice(Hq, Hq + Hk))):
        got = np64(got)
        tol = half_step(dtype) * np.abs(want) + 8 * U * reach
        assert (np.abs(got - want) <= tol)[live].all(), np.abs(got - want)[live].max()
        if rot < D:
            assert np.array_equal(got[live][..., rot:], np64(before[:, at])[live][..., rot:])
        stale = np64(before[:, at]) if in_place else np.full(got.shape, 9.0)
        assert np.array_equal(got[~live], stale[~live])
    assert torch.equal(v, before[:, Hq + Hk:])
    if to_cache:
        written = torch.zeros((pages, ps), dtype=torch.bool)
        for t in range(T):
            if live[t] and slot[t] >= 0:
                pg, row = int(slot[t]) // ps, int(slot[t]) % ps
                written[pg, row] = True
                assert torch.equal(cache.k[1, pg, row], k_out[t]) and torch.equal(cache.v[1, pg, row], v[t])
        for x in (cache.k, cache.v):
            assert (x[0] == 3.0).all() and (x[1].cpu()[~written] == 3.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (256, 256), (128, 64), (64, 24), (64, 2), (256, 62), (128, 80)])
def test_rope_layouts_and_parts_of_the_head(D, rot, dtype, interleaved):
    check_rope(33, 6, 2, D, rot, dtype, interleaved, 5000, seed=D + rot)
    check_rope(7, 3, 1, D, rot, dtype, interleaved, 5000, seed=rot, in_place=True, hnd=True, scale=1.25)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("far", [10, 1 << 20, (1 << 31) - 1])
def test_rope_far_positions(far, dtype):
    check_rope(50, 2, 2, 128, 128, dtype, False, far, seed=1, base=5e5)
    check_rope(50, 2, 1, 64, 48, dtype, True, far, seed=2, base=1.0)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 64, 8), (2, 5, 5), (1300, 16, 2), (12000, 2, 1), (13, 7, 1)])
def test_rope_sizes(T, Hq, Hk):
    check_rope(T, Hq, Hk, 64, 16, BF, False, 9000, seed=T, ps=16, to_cache=T < 2000)


@pytest.mark.parametrize("D,rot", [(8, 8), (24, 8), (40, 6), (96, 96), (200, 200), (72, 16)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rope_without_a_cache_takes_other_head_sizes(D, rot, dtype):
    for interleaved in (False, True):
        check_rope(9, 3, 2, D, rot, dtype, interleaved, 500, seed=D, to_cache=False)
        check_rope(9, 3, 2, D, rot, dtype, interleaved, 500, seed=D, to_cache=False, in_place=True)


def test_rope_bad_slots_are_told_and_the_rest_is_written():
    cache = L.KVCache(1, 3, 4, 1, 64)
    k = torch.randn((4, 1, 64), device="cuda").to(BF)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lin_state_rope(cache, k=k, v=k, position=i32([0, 0, 0, -1]), inv_freq=torch.ones(32, device="cuda"),
                     slot=torch.tensor([11, 12, 1 << 40, 0]).cuda(), status=status)
    assert L.lin_state_read_status(status) == L.LIN_ST_BAD_PAGE
    assert torch.equal(cache.k[0, 2, 3], k[0]) and int((cache.k != 0).any(-1).sum()) == 1


def test_rope_single_outputs():
    q = torch.randn((5, 3, 64), device="cuda")
    inv, pos = L.rope_frequencies(64)[0], i32(range(5))
    a, b = torch.empty_like(q), torch.empty_like(q)
    L.lin_state_rope(q=q, q_out=a, position=pos, inv_freq=inv)
    L.lin_state_rope(k=q, k_out=b, position=pos, inv_freq=inv)
    assert torch.equal(a, b) and torch.equal(a[0], q[0])


# ---- attention of packed new tokens ---------------------------------------------------------

def check_chunk(cache, table, q, cu, lens, out_dtype, scale=None, layer=0, status_want=0, **kw):
    """Looks over the call's outputs, and again with room for so many pages that requests of
    many rows go in items of two row tiles, which calls with little work do not."""
    if status_want != L.LIN_ST_BAD_SEQLEN:
        wide = -(-(1 << 26) // (q.shape[0] * q.shape[1] * cache.page_size)) + table.shape[1]
        more = torch.full((table.shape[0], wide), 1 << 30, dtype=torch.int32)  # (never looked up)
        more[:, :table.shape[1]] = table
        look_chunk(cache, more, q, cu, lens, out_dtype, scale, layer, status_want, table, **kw)
    return look_chunk(cache, table, q, cu, lens, out_dtype, scale, layer, status_want, table, **kw)


def look_chunk(cache, given, q, cu, lens, out_dtype, scale, layer, status_want, table, **kw):
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), 7.0, dtype=out_dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lin_state_attn_chunk(cache, layer=layer, q=q, out=out, page_table=given.cuda(), cu_seqlens=i32(cu),
                           kv_len=i32(lens), scale=scale, status=status, **kw)
    assert L.lin_state_read_status(status) == status_want
    s = D ** -0.5 if scale is None else scale
    want, reach, spread = O.attn_chunk(np64(cache.k[layer]), np64(cache.v[layer]), np64(q), table.numpy(), cu, lens, s)
    got = np64(out)
    skipped = np.isnan(want)
    assert (got[skipped] == 7.0).all()
    c, d = ((0.0, 2.0 ** -8 if out_dtype == BF else 2.0 ** -24) if cache.dtype == BF else (12.0, 12.0 * U))
    inner = 2 * spread * (D + 16 + c) * U + (max(list(lens) + [0]) + 16) * U + d
    tol = half_step(out_dtype) * np.abs(want) + reach * inner
    bad = ~skipped & ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:6], np.argwhere(bad)[-3:],
                           float(np.nanmax(np.abs(got - want) - tol)))
    # on the whole a bf16 output is off by its rounding and the weights', each 2^-9 rms at most
    if cache.dtype == BF and out_dtype == BF and (~skipped).sum() > 1000:
        off = np.linalg.norm((got - want)[~skipped]) / max(np.linalg.norm(want[~skipped]), 1e-30)
        assert off < 2.0 ** -8
    return out


def chunk_inputs(cached, new, ps, Hq, Hkv, D, dtype, seed, hnd=False, layers=1, spare=0):
    """Cache, table, packed queries (a view of a projection's rows), cu_seqlens, kv_len."""
    lens = [c + n if c >= 0 else -1 for c, n in zip(cached, new)]
    cache, table, gen = make_cache(lens, ps, Hkv, D, dtype, seed, hnd=hnd, layers=layers)
    cu = np.concatenate([[0], np.cumsum(new)])
    rows = torch.randn((int(cu[-1]) + spare, Hq + 2 * Hkv, D), generator=gen).to(dtype).cuda()
    return cache, table, rows[:, :Hq], cu, lens


TYPES = [(BF, BF), (BF, F32), (F32, F32), (F32, BF)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,out_dtype", TYPES)
def test_chunk_types_and_heads(D, dtype, out_dtype):
    """From one token to a few hundred after none to a thousand; padding, requests
    without new tokens, rows behind the last; NaN wherever no token lies."""
    cached = [0, 0, 0, 63, 64, 100, -1, 1000, 0, 500, 31, 128]
    new = [1, 2, 130, 1, 64, 37, 0, 1, 0, 0, 300, 129]
    x = chunk_inputs(cached, new, 24, 6, 2, D, dtype, seed=D, spare=5)
    check_chunk(*x, out_dtype)


@pytest.mark.parametrize("ps", [1, 7, 16, 64, 100, 128, 300])
@pytest.mark.parametrize("hnd", [False, True])
def test_chunk_page_sizes_and_layouts(ps, hnd):
    cached, new = [5, 99, 0, 257], [60, 1, 101, 130]
    x = chunk_inputs(cached, new, ps, 3, 3, 64, BF, seed=ps, hnd=hnd, layers=2)
    check_chunk(*x, BF, layer=1)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 1), (16, 2), (17, 1), (40, 2), (64, 1), (65, 1), (130, 1),
                                    (300, 1), (8, 8)])
@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64), (BF, 256)])
def test_chunk_group_sizes(Hq, Hkv, dtype, D):
    cached, new = [70, 0, 200], [33, 40, 5]
    x = chunk_inputs(cached, new, 16, Hq, Hkv, D, dtype, seed=Hq)
    check_chunk(*x, dtype)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_chunk_lengths_around_tiles(D, dtype):
    """Every border of tiles of queries and keys, from one side and the other."""
    new = [15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257]
    cached = [0, 1, 127, 128, 129, 0, 64, 65, 63, 1, 0, 255, 256, 257, 3]
    x = chunk_inputs(cached, new, 32, 2, 1, D, dtype, seed=D)
    check_chunk(*x, dtype)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,out_dtype", TYPES)
def test_chunk_few_rows_over_a_long_cache(D, dtype, out_dtype):
    """Items that many CTAs share and the second launch joins."""
    x = chunk_inputs([6000, 3001], [3, 1], 16, 4, 1, D, dtype, seed=D)
    check_chunk(*x, out_dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_chunk_a_whole_prompt(dtype):
    x = chunk_inputs([0, 700], [1500, 900], 64, 4, 2, 128, dtype, seed=3)
    check_chunk(*x, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_chunk_many_requests_of_single_tokens(dtype):
    rng = np.random.default_rng(0)
    cached = rng.integers(0, 400, 300).tolist()
    x = chunk_inputs(cached, [1] * 300, 16, 8, 2, 64, dtype, seed=4)
    check_chunk(*x, dtype)


@pytest.mark.parametrize("dtype,D", [(BF, 64), (BF, 128), (BF, 256), (F32, 64), (F32, 256)])
def test_chunk_queries_that_see_nothing(dtype, D):
    """Fewer cached tokens than queries: the first ones lie before the request."""
    cache, table, q, cu, _ = chunk_inputs([0, 0, 0, 0], [100, 300, 40, 7], 16, 4, 2, D, dtype, seed=5)
    lens = [30, 299, 0, 1]
    out = check_chunk(cache, table, q, cu, lens, dtype)
    assert not out[:70].any() and not out[400:440].any()


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 30.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_chunk_scales(scale, dtype):
    x = chunk_inputs([100, 0], [90, 200], 16, 4, 2, 64, dtype, seed=6)
    check_chunk(*x, dtype, scale=scale)


@pytest.mark.parametrize("dtype,D", [(BF, 64), (BF, 128), (BF, 256), (F32, 64), (F32, 128)])
def test_chunk_bad_pages_are_not_seen(dtype, D):
    cache, table, q, cu, lens = chunk_inputs([300, 20, 0], [80, 5, 200], 16, 4, 2, D, dtype, seed=7)
    table[0, 3], table[0, 7], table[2, 0] = -1, cache.num_pages, 1 << 30
    for r in (0, 1):
        table[1, r] = -5
    out = check_chunk(cache, table, q, cu, lens, dtype, status_want=L.LIN_ST_BAD_PAGE)
    assert not out[80:85].any()


@pytest.mark.parametrize("dtype,D,ps", [(BF, 64, 16), (BF, 128, 16), (BF, 128, 7), (BF, 256, 16), (BF, 256, 9), (F32, 64, 16),
                                        (F32, 256, 16)])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_chunk_hidden_values_have_no_part(dtype, D, ps, what):
    """Keys and values of a later token of the same prompt may be anything: queries before
    it keep their bits, those that see it do not pass for finite."""
    cached, new = [200, 0], [300, 290]
    cache, table, q, cu, lens = chunk_inputs(cached, new, ps, 4, 2, D, dtype, seed=8)

    def run():
        out = torch.zeros(q.shape, dtype=dtype, device="cuda")
        L.lin_state_attn_chunk(cache, layer=0, q=q, out=out, page_table=table.cuda(), cu_seqlens=i32(cu), kv_len=i32(lens))
        return out

    plain = run()
    for r, t in ((0, 350), (0, 470), (1, 1), (1, 289)):
        cache.v[0, table[r, t // ps], t % ps] = what
    wild = run()
    assert torch.equal(wild[:150], plain[:150]) and torch.equal(wild[300:301], plain[300:301])
    assert not torch.isfinite(wild[150:300]).any() and not torch.isfinite(wild[301:]).any()
    for r, t in ((0, 350), (1, 1)):
        cache.k[0, table[r, t // ps], t % ps] = float("nan")
    wild = run()
    assert torch.equal(wild[:150], plain[:150]) and torch.equal(wild[300:301], plain[300:301])


def test_chunk_batches_that_break_the_rules():
    cache, table, q, _, _ = chunk_inputs([100, 100, 100, 100], [30, 30, 30, 30], 16, 2, 1, 64, BF, seed=9)
    lens = [130, table.shape[1] * 16 + 1, 130, 130]
    check_chunk(cache, table, q, np.array([0, 30, 60, 90, 120]), lens, BF, status_want=L.LIN_ST_BAD_SEQLEN)
    lens = [130] * 4
    check_chunk(cache, table, q, np.array([-1, 30, 60, 20, 121]), lens, BF, status_want=L.LIN_ST_BAD_SEQLEN)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_chunk_same_bits_again_and_on_another_stream(dtype):
    cache, table, q, cu, lens = chunk_inputs([900, 0], [100, 400], 16, 8, 2, 128, dtype, seed=10)
    a = check_chunk(cache, table, q, cu, lens, dtype)
    b = check_chunk(cache, table, q, cu, lens, dtype)
    side = torch.cuda.Stream()
    out = torch.zeros(q.shape, dtype=dtype, device="cuda")
    tables = table.cuda(), i32(cu), i32(lens)
    torch.cuda.synchronize()
    L.lin_state_attn_chunk(cache, layer=0, q=q, out=out, page_table=tables[0], cu_seqlens=tables[1],
                           kv_len=tables[2], stream=side)
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(a, out)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n_hi,Hq", [(16, 8), (40, 4)])
def test_chunk_tails_of_many_requests(D, n_hi, Hq):
    """Items of a few tiles that cross the CTAs' ranges everywhere, several pieces to a
    CTA, with one row tile and with two: the same bits each time."""
    rng = np.random.default_rng(D + n_hi)
    cached = rng.integers(300, 2200, 24).tolist()
    new = rng.integers(1, n_hi + 1, 24).tolist()
    x = chunk_inputs(cached, new, 48, Hq, 1, D, BF, seed=D)
    a = check_chunk(*x, BF)
    for _ in range(4):
        assert torch.equal(a, check_chunk(*x, BF))


@pytest.mark.parametrize("D,Hq,Hkv,ps", [(64, 8, 8, 16), (128, 4, 4, 12), (128, 16, 4, 64), (256, 16, 4, 8), (64, 3, 3, 20)])
def test_chunk_batches_of_many_items(D, Hq, Hkv, ps):
    """More than four items to a CTA, which are handed out one by one: requests without
    tokens, with one, with many; padding; rows behind the last one."""
    rng = np.random.default_rng(D)
    cached = rng.integers(0, 200, 90).tolist()
    new = rng.choice([0, 1, 2, 63, 64, 65, 130, 260], 90).tolist()
    cached[7], new[7] = -1, 0
    G, m = Hq // Hkv, (256 if D < 256 else 128)
    rows = int(4.5 * 152 / Hkv * (m // G))  # a captured call's room
    x = chunk_inputs(cached, new, ps, Hq, Hkv, D, BF, seed=D, spare=max(0, rows - sum(new)))
    a = check_chunk(*x, BF)
    assert torch.equal(a, check_chunk(*x, BF))


def test_a_captured_batch_of_many_items_follows_its_lengths():
    """Items handed out by the counter, which each replay begins anew; the same call eagerly,
    then on another stream with a workspace of its own, gives the same bits."""
    T, B, ps, H, D = 9760, 5, 16, 2, 64
    cache, table, gen = make_cache([4000] * B, ps, H, D, BF, 3)
    q = torch.randn((T, 8 * H, D), generator=gen).to(BF).cuda()
    table = table.cuda()
    cu, lens = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.full((B,), -1, dtype=torch.int32, device="cuda")
    out = torch.zeros(q.shape, dtype=BF, device="cuda")
    size = L.lin_state_attn_chunk_workspace(cache, batch=B, tokens=T, num_q_heads=8 * H, max_pages=table.shape[1])
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    args = dict(layer=0, q=q, page_table=table, cu_seqlens=cu, kv_len=lens)
    L.lin_state_attn_chunk(cache, out=out, workspace=work, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lin_state_attn_chunk(cache, out=out, workspace=work, **args)
    for new, cached in (([3000, 1, 0, 777, 2500], [1000, 0, 5, 3000, 64]), ([1, 2, 3, 4, 5], [9, 9, 9, 9, 9]),
                        ([4000, 4000, 1000, 700, 60], [0, 0, 0, 0, 3940])):
        cu.copy_(i32(np.concatenate([[0], np.cumsum(new)])))
        lens.copy_(i32([a + b for a, b in zip(new, cached)]))
        out.zero_()
        graph.replay()
        again, side = torch.zeros_like(out), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        L.lin_state_attn_chunk(cache, out=again, stream=side, **args)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(out, again) and not out[sum(new):].any() and out[:sum(new)].any()


def test_chunk_requests_over_the_same_rows_end():
    """Requests whose packed rows overlap have more items than a batch of that many rows:
    it is told, and the counter that hands items out stops at what a batch can have. (Both
    requests are alike, so it does not matter whose rows are written last.)"""
    T = 9760  # 305 items of 32 tokens to a head: more than four to a CTA
    cache, table, q, _, _ = chunk_inputs([50], [T], 64, 16, 2, 64, BF, seed=12)
    one, many = (torch.zeros(q.shape, dtype=BF, device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lin_state_attn_chunk(cache, layer=0, q=q, out=one, page_table=table.cuda(), cu_seqlens=i32([0, T]),
                           kv_len=i32([50 + T]), status=status)
    assert L.lin_state_read_status(status) == 0
    L.lin_state_attn_chunk(cache, layer=0, q=q, out=many, page_table=table.cuda().repeat(3, 1),
                           cu_seqlens=i32([0, T, 0, T]), kv_len=i32([50 + T] * 3), status=status)
    assert L.lin_state_read_status(status) == L.LIN_ST_BAD_SEQLEN
    assert torch.equal(one, many)


@pytest.mark.parametrize("rot", [2, 30, 62, 100, 126])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rope_parts_that_end_inside_a_chunk(rot, interleaved, dtype):
    """Partners in other chunks of the row, more rows than a block takes at a time, in place."""
    check_rope(700, 7, 3, 128, rot, dtype, interleaved, 100000, rot)
    check_rope(9, 7, 3, 128, rot, dtype, interleaved, 100000, rot, in_place=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ps", [5, 20, 40])
@pytest.mark.parametrize("hnd", [False, True])
def test_chunk_pages_of_any_size(D, ps, hnd):
    """Pages that TMA takes in boxes of 8 and those that it does not."""
    cached, new = [5, 300, 0], [60, 70, 290]
    x = chunk_inputs(cached, new, ps, 4, 2, D, BF, seed=ps, hnd=hnd, layers=2)
    check_chunk(*x, BF, layer=1)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", [(300, 2), (3, 8)])
def test_chunk_long_sums_keep_their_size(D, n, G):
    """Values of one sign over more tokens than a run of the tensor unit, whose sums lose
    towards 0: the mean output stays within 2^-11, the documented loss, and the weights'
    rounding, which is of no sign (2^-9 rms over sqrt(tokens): nothing)."""
    length, ps, H = 70000, 64, 1
    gen = torch.Generator(device="cuda").manual_seed(D)
    pages = -(-length // ps)
    k = torch.randn((1, pages, ps, H, D), generator=gen, device="cuda").to(BF)
    v = (torch.rand((1, pages, ps, H, D), generator=gen, device="cuda") + 0.5).to(BF)
    cache = L.KVCache(1, pages, ps, H, D, k=k, v=v)
    q = (torch.randn((n, G, D), generator=gen, device="cuda") * 0.2).to(BF)
    out = torch.empty_like(q)
    # (one item of 70,000 keys is cut into ranges; many requests over the same pages are not)
    B = 170 if n == 300 else 1
    rep = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(B, 1)
    qs, outs = q.repeat(B, 1, 1), out.repeat(B, 1, 1)
    L.lin_state_attn_chunk(cache, layer=0, q=qs, out=outs, page_table=rep, cu_seqlens=i32(np.arange(B + 1) * n),
                           kv_len=i32([length] * B))
    got = outs[-n:].double()
    kk, vv = k.reshape(-1, D)[:length].double(), v.reshape(-1, D)[:length].double()
    rows = range(0, n, 37)
    for j in rows:
        s = (q[j].double() @ kk.T) * D ** -0.5
        s[:, length - n + j + 1:] = -float("inf")
        want = torch.softmax(s, -1) @ vv
        assert abs(float((got[j] - want).mean() / want.mean())) < 2.0 ** -11
        assert float(((got[j] - want) / want).abs().max()) < 2.0 ** -8 + 2.0 ** -10


def test_chunk_references_move():
    """Scores that grow along the keys by far more than a weight may: the reference moves
    in many tiles, in the first and the last of a piece, and some rows' alone."""
    for D, n, c in ((64, 200, 900), (128, 200, 900), (256, 100, 900), (128, 3, 5000)):
        cache, table, q, cu, lens = chunk_inputs([c], [n], 16, 4, 2, D, BF, seed=D)
        t = torch.arange(lens[0])
        for h in range(2):
            grow = (1.0 + t / 20.0) * (1.0 if h == 0 else (t % 3 == 0).float())
            key = torch.zeros(lens[0], D)
            key[:, 0] = grow
            pages = table[0, t // 16].long().cuda()
            cache.k[0][pages, (t % 16).cuda(), h] = key.to(BF).cuda()
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(1)).to(BF).cuda())
        q[:, :, 0] = (torch.rand(q.shape[:2], generator=torch.Generator().manual_seed(2)) * 60 - 20).to(BF).cuda()
        check_chunk(cache, table, q, cu, lens, BF)


def test_a_captured_prompt_follows_its_lengths():
    """Plan, rotary positions with the append, and attention captured once and replayed for
    chunk after chunk of two prompts, against the same tokens in one eager call each."""
    torch.manual_seed(0)
    B, ps, Hq, Hkv, D, room = 2, 16, 4, 2, 128, 160
    total = [300, 211]
    data = [torch.randn((n, Hq + 2 * Hkv, D), device="cuda").to(BF) for n in total]
    inv = L.rope_frequencies(D)[0]

    def state():
        wide = 20
        return dict(cache=L.KVCache(1, B * wide, ps, Hkv, D), length=i32([0] * B), n_new=i32([0] * B),
                    table=torch.full((B, wide), -1, dtype=torch.int32, device="cuda"),
                    free=torch.arange(B * wide, dtype=torch.int32, device="cuda"), taken=i32([0]), cu=i32([0] * (B + 1)),
                    kv=i32([0] * B), status=i32([0]), ws=None)

    def step(s, rows, out, pos, slot, q):
        L.lin_state_kv_plan(page_size=ps, num_pages=s["cache"].num_pages, length=s["length"], n_new=s["n_new"],
                            page_table=s["table"], free_pages=s["free"], taken=s["taken"], cu_seqlens=s["cu"],
                            kv_len=s["kv"], position=pos, slot=slot, status=s["status"])
        L.lin_state_rope(s["cache"], q=rows[:, :Hq], k=rows[:, Hq:Hq + Hkv], v=rows[:, Hq + Hkv:], q_out=q, position=pos,
                         slot=slot, inv_freq=inv, status=s["status"])
        L.lin_state_attn_chunk(s["cache"], layer=0, q=q, out=out, page_table=s["table"], cu_seqlens=s["cu"],
                               kv_len=s["kv"], status=s["status"], workspace=s["ws"])

    def buffers(T):
        return (torch.zeros((T, Hq, D), dtype=BF, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda"),
                torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros((T, Hq, D), dtype=BF, device="cuda"))

    whole = state()
    whole["n_new"].copy_(i32(total))
    out, pos, slot, q = buffers(sum(total))
    step(whole, torch.cat(data), out, pos, slot, q)
    want = out.split(total)

    s = state()
    rows = torch.zeros((room, Hq + 2 * Hkv, D), dtype=BF, device="cuda")
    cout, cpos, cslot, cq = buffers(room)
    s["ws"] = torch.empty(L.lin_state_attn_chunk_workspace(s["cache"], batch=B, tokens=room, num_q_heads=Hq, max_pages=20),
                          dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(s, rows, cout, cpos, cslot, cq)  # nothing new yet
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s, rows, cout, cpos, cslot, cq)
    done, used, got = [0, 0], 0, [[], []]
    for sizes in ([100, 60], [1, 1], [0, 150], [159, 0], [40, 0]):
        rows.zero_()
        at = 0
        for r, n in enumerate(sizes):
            rows[at:at + n] = data[r][done[r]:done[r] + n]
            at += n
        s["length"].copy_(i32(done))
        s["n_new"].copy_(i32(sizes))
        s["free"].copy_(torch.roll(torch.arange(40, dtype=torch.int32), -used))
        graph.replay()
        used += int(s["taken"])
        at = 0
        for r, n in enumerate(sizes):
            got[r].append(cout[at:at + n].clone())
            at += n
            done[r] += n
    assert done == total and L.lin_state_read_status(s["status"]) == 0
    for r in range(2):
        x, y = torch.cat(got[r]).double(), want[r].double()
        # the same sums cut and joined elsewhere: two bf16 roundings and the weights'
        assert float((x - y).norm() / y.norm()) < 2.0 ** -7
