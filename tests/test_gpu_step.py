"""Decode-step operators on the GPU against the fp64 oracle: the paged cache's
append, decode attention (steps, chains and trees of drafts) and the norms
around a block.

Tolerances are per element. A stored output is off by at most half a step of
its type, eps / 2 of its value. Inside the sums fp32 rounds by u = 2^-24:
  * a score of D products is off by at most (D + 16) u S, S = scale sum |q k|,
    which moves its weight by that share; so do the maximum and the exponential;
  * the weights' sum and the sum over L values round at most L + 16 times;
  * a bf16 cache's weights go in two bf16 parts (2^-16; three for fp32 outputs:
    2^-24), an fp32 cache's products in two tf32 parts (three terms of 2^-22).
So |out - want| <= eps/2 |want| + reach (2 S (D + 16 + c) u + (L + 16) u + d)
with reach = sum p |v|."""

import numpy as np
import pytest
import torch

import linear_attention_state_chunked_gb300 as L
from oracle import lin_step_oracle as O
from tests.helpers import np64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def pages_for(lens, ps, gen, extra=0, spare=1):
    """A page table (-1 where nothing is allocated) over shuffled pages."""
    need = [-(-(max(x, 0) + extra) // ps) for x in lens]
    wide = max(1, max(need) + spare)
    ids = torch.randperm(sum(need) + 1, generator=gen)
    table = torch.full((len(lens), wide), -1, dtype=torch.int32)
    at = 0
    for r, k in enumerate(need):
        table[r, :k] = ids[at:at + k].to(torch.int32)
        at += k
    return table, sum(need) + 1


def make_cache(lens, ps, H, D, dtype, seed, hnd=False, layers=1, fill=float("nan")):
    """A cache whose rows past each request's length and free pages hold `fill`."""
    gen = torch.Generator().manual_seed(seed)
    table, pages = pages_for(lens, ps, gen)
    shape = (layers, pages, H, ps, D) if hnd else (layers, pages, ps, H, D)
    kv = []
    for _ in range(2):
        x = torch.randn(shape, generator=gen).to(dtype)
        x = x.transpose(2, 3) if hnd else x
        live = torch.zeros((pages, ps), dtype=torch.bool)
        for r, n in enumerate(lens):
            for t in range(max(n, 0)):
                live[table[r, t // ps], t % ps] = True
        x[:, ~live] = fill
        kv.append(x.cuda())
    return L.KVCache(layers, pages, ps, H, D, dtype=dtype, k=kv[0], v=kv[1]), table, gen


def check_attn(cache, table, q, lens, out_dtype, parent=None, scale=None, layer=0, status_want=0, **kw):
    B, n, Hq, D = q.shape
    out = torch.full((B, n, Hq, D), 7.0, dtype=out_dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lin_state_attn_decode(cache, layer=layer, q=q, out=out, page_table=table.cuda(),
                            kv_len=torch.tensor(lens, dtype=torch.int32).cuda(), scale=scale,
                            parent=None if parent is None else torch.tensor(parent, dtype=torch.int32).cuda(),
                            status=status, **kw)
    assert L.lin_state_read_status(status) == status_want
    s = D ** -0.5 if scale is None else scale
    want, reach, spread = O.attn_decode(np64(cache.k[layer]), np64(cache.v[layer]), np64(q), table.numpy(),
                                        lens, s, parent)
    got = np64(out)
    skipped = np.isnan(want)
    assert (got[skipped] == 7.0).all()
    c, d = (0.0, 2.0 ** -16 if out_dtype == BF else 2.0 ** -24) if cache.dtype == BF else (12.0, 12.0 * U)
    inner = 2 * spread * (D + 16 + c) * U + (max(lens) + 16) * U + d
    tol = half_step(out_dtype) * np.abs(want) + reach * inner
    bad = ~skipped & ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], float(np.nanmax(np.abs(got - want) - tol)))
    return out


def queries(B, n, Hq, Hkv, D, dtype, gen):
    rows = torch.randn((B, n, Hq + 2 * Hkv, D), generator=gen).to(dtype).cuda()
    return rows[:, :, :Hq]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_attn_types_and_heads(D, dtype, out_dtype):
    """Lengths 0, 1, around the tiles' ends and long; padding rows; pages that
    end inside a tile; NaN wherever no token lies."""
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 130, -1, 333, 1000]
    cache, table, gen = make_cache(lens, 24, 2, D, dtype, seed=D)
    check_attn(cache, table, queries(len(lens), 1, 6, 2, D, dtype, gen), lens, out_dtype)


@pytest.mark.parametrize("ps", [1, 7, 16, 64, 100])
@pytest.mark.parametrize("hnd", [False, True])
def test_attn_page_sizes_and_layouts(ps, hnd):
    lens = [5, 99, 100, 101, 257]
    cache, table, gen = make_cache(lens, ps, 3, 64, BF, seed=ps, hnd=hnd, layers=2)
    check_attn(cache, table, queries(5, 1, 3, 3, 64, BF, gen), lens, BF, layer=1)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (16, 1), (17, 1), (40, 2), (64, 1), (65, 1), (160, 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_group_sizes(Hq, Hkv, dtype):
    lens = [70, 1, 200]
    cache, table, gen = make_cache(lens, 16, Hkv, 64, dtype, seed=Hq)
    check_attn(cache, table, queries(3, 1, Hq, Hkv, 64, dtype, gen), lens, dtype)


@pytest.mark.parametrize("n", [2, 3, 4, 8, 17, 32])
@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64), (BF, 256), (F32, 256)])
def test_attn_chain_of_drafts(n, dtype, D):
    """Lengths from none over fewer tokens than drafts (rows that see nothing)
    to the drafts spread over a tile's border."""
    lens = [0, 1, n - 1, n, n + 1, 60 + n // 2, 64 + n, 150]
    cache, table, gen = make_cache(lens, 16, 2, D, dtype, seed=n)
    out = check_attn(cache, table, queries(8, n, 6, 2, D, dtype, gen), lens, dtype)
    assert not out[0].any() and not out[1, :n - 1].any()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", [(17, 1), (8, 3), (4, 8), (3, 11), (8, 8), (13, 5), (32, 4), (3, 43)])
@pytest.mark.parametrize("out_dtype,tree", [(BF, False), (F32, True)])
def test_attn_rows_and_tiles(D, n, G, out_dtype, tree):
    """17 to 129 rows per key-value head over lengths around the tiles' ends,
    from none to some that are split, in one batch."""
    lens = [0, 1, n, 62 + n, 64, 127, 128, 129, 900, 1300, -1, 2600]
    rng = np.random.default_rng(n * G)
    parent = [[int(rng.integers(max(-1, j - 4), j)) if j else -1 for j in range(n)] for _ in lens] if tree else None
    cache, table, gen = make_cache(lens, 20, 1, D, BF, seed=n + G)
    check_attn(cache, table, queries(len(lens), n, G, 1, D, BF, gen), lens, out_dtype, parent=parent)


@pytest.mark.parametrize("G", [2, 8, 16, 32])
def test_attn_hidden_drafts_of_many_rows(G):
    """As below, over a longer cache and up to 128 rows, with the bad drafts on
    both sides of a tile's border."""
    lens, n = [258, 700], 4
    parent = [[-1, -1, 0, 1]] * 2
    cache, table, gen = make_cache(lens, 16, 1, 128, BF, seed=G)
    q = queries(2, n, G, 1, 128, BF, gen)
    before = check_attn(cache, table, q, lens, BF, parent=parent).clone()
    for r, t in ((0, 255), (0, 257), (1, 697), (1, 699)):  # drafts 1 and 3
        at = O.locate(table[r], t, 16, cache.num_pages)
        cache.k[0, at[0], at[1]] = float("nan")
        cache.v[0, at[0], at[1], :, ::2] = float("nan")
        cache.v[0, at[0], at[1], :, 1::2] = float("-inf")
    out = torch.zeros_like(before)
    L.lin_state_attn_decode(cache, layer=0, q=q, out=out, page_table=table.cuda(),
                            kv_len=torch.tensor(lens, dtype=torch.int32).cuda(),
                            parent=torch.tensor(parent, dtype=torch.int32).cuda())
    for j in (0, 2):
        assert torch.equal(out[:, j], before[:, j])
    for j in (1, 3):
        assert out[:, j].isnan().all()


def test_attn_repeats_bit_for_bit_with_many_rows():
    lens = [4000, 77, 1500]
    cache, table, gen = make_cache(lens, 16, 2, 128, BF, seed=18)
    q = queries(3, 4, 16, 2, 128, BF, gen)
    first = check_attn(cache, table, q, lens, BF)
    for _ in range(3):
        assert torch.equal(check_attn(cache, table, q, lens, BF), first)


@pytest.mark.parametrize("n", [2, 8, 32])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_draft_trees(n, dtype):
    rng = np.random.default_rng(n)
    lens = [n, n + 3, 100, 61 + n]
    parent = [[int(rng.integers(-1, j)) if j else -1 for j in range(n)] for _ in lens]
    parent[0] = [-1] * n
    parent[1] = list(range(-1, n - 1))
    cache, table, gen = make_cache(lens, 8, 2, 64, dtype, seed=n)
    q = queries(4, n, 4, 2, 64, dtype, gen)
    out = check_attn(cache, table, q, lens, dtype, parent=parent)
    chain = check_attn(cache, table, q, lens, dtype)
    assert torch.equal(out[1], chain[1])  # a tree that is a chain


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_hidden_drafts_may_hold_anything(dtype):
    """A sibling's keys and values have no part in a row that does not see it:
    NaN and infinities there leave every other row as it was."""
    lens, n = [20, 77], 4
    parent = [[-1, -1, 0, 1]] * 2
    cache, table, gen = make_cache(lens, 16, 2, 64, dtype, seed=5)
    q = queries(2, n, 4, 2, 64, dtype, gen)
    before = check_attn(cache, table, q, lens, dtype, parent=parent).clone()
    for r, t in ((0, 17), (1, 74)):  # draft 1 of each request
        at = O.locate(table[r], t, 16, cache.num_pages)
        cache.k[0, at[0], at[1]] = float("nan")
        cache.v[0, at[0], at[1], :, ::2] = float("nan")
        cache.v[0, at[0], at[1], :, 1::2] = float("inf")
    out = torch.zeros_like(before)
    L.lin_state_attn_decode(cache, layer=0, q=q, out=out, page_table=table.cuda(),
                            kv_len=torch.tensor(lens, dtype=torch.int32).cuda(),
                            parent=torch.tensor(parent, dtype=torch.int32).cuda())
    for j in (0, 2):
        assert torch.equal(out[:, j], before[:, j])
    for j in (1, 3):
        assert out[:, j].isnan().all()


def test_attn_scores_of_any_size():
    """Scores of hundreds (one weight is 1, the others 0), negative scales and
    a row of equal scores."""
    lens = [300, 40]
    cache, table, gen = make_cache(lens, 16, 1, 128, F32, seed=9)
    q = queries(2, 2, 4, 1, 128, F32, gen)
    for scale in (30.0, -0.5, 0.0):
        check_attn(cache, table, q, lens, F32, scale=scale)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attn_long_and_ragged(dtype):
    """Requests split over many CTAs beside requests of a few tokens."""
    lens = [9000, 3, 0, 5000, 1, 700, -1, 64]
    cache, table, gen = make_cache(lens, 48, 2, 128, dtype, seed=77)
    check_attn(cache, table, queries(8, 2, 8, 2, 128, dtype, gen), lens, dtype)


def test_attn_many_short_requests():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(-1, 40, 700)]
    cache, table, gen = make_cache(lens, 8, 1, 64, BF, seed=3)
    check_attn(cache, table, queries(700, 1, 4, 1, 64, BF, gen), lens, BF)


@pytest.mark.parametrize("D,n", [(64, 1), (128, 3), (256, 8)])
def test_attn_fp32_error_does_not_grow_with_the_length(D, n):
    """fp32 sums over 64 times the tokens: every rounding is to nearest, so errors
    grow as the outputs' own random sum does. A bias of one cut-off place per
    addition would show: 16,384 tokens are 1,024 additions, 2^-14 of the outputs
    at the most. The bound is 2^-20, four places above the products' 2^-22."""
    gen = torch.Generator().manual_seed(D)
    for length in (256, 16384):
        cache, table, _ = make_cache([length], 64, 1, D, F32, seed=length)
        q = queries(1, n, 4, 1, D, F32, gen)
        out = torch.empty((1, n, 4, D), device="cuda")
        L.lin_state_attn_decode(cache, layer=0, q=q, out=out, page_table=table.cuda(),
                                kv_len=torch.tensor([length], dtype=torch.int32).cuda())
        at = table[0, :length // 64].long().cuda()
        k, v = (t[0, at].reshape(length, D).double() for t in (cache.k, cache.v))
        s = torch.einsum("jhd,td->jht", q[0].double(), k) * D ** -0.5
        hidden = torch.arange(length, device="cuda") > length - n + torch.arange(n, device="cuda")[:, None]
        want = torch.softmax(s.masked_fill(hidden[:, None], -torch.inf), -1) @ v
        assert float((out[0] - want).norm() / want.norm()) < 2.0 ** -20


def test_attn_repeats_bit_for_bit():
    lens = [4000, 77, 1500]
    cache, table, gen = make_cache(lens, 16, 2, 128, BF, seed=8)
    q = queries(3, 4, 8, 2, 128, BF, gen)
    first = check_attn(cache, table, q, lens, BF)
    for _ in range(3):
        assert torch.equal(check_attn(cache, table, q, lens, BF), first)


def test_attn_status_bits():
    """Bad pages count as not seen, a bad tree or length leaves its request out,
    and the rest of the batch completes."""
    lens = [40, 40, 40, 40]
    cache, table, gen = make_cache(lens, 16, 1, 64, BF, seed=4)
    q = queries(4, 2, 2, 1, 64, BF, gen)
    bad = table.clone()
    bad[1, 1] = cache.num_pages
    bad[2, 0] = -5
    check_attn(cache, bad, q, lens, BF, status_want=L.LIN_ST_BAD_PAGE)
    long = [40, 40, 16 * table.shape[1] + 1, 40]
    check_attn(cache, table, q, long, BF, status_want=L.LIN_ST_BAD_SEQLEN)
    trees = [[-1, 0], [-1, 1], [-1, -2], [0, 0]]
    check_attn(cache, table, q, lens, BF, parent=trees, status_want=L.LIN_ST_BAD_TREE)


def test_attn_far_pages():
    """Byte offsets past 2^32 in the pool."""
    pages = 20000
    k, v = (torch.empty((1, pages, 64, 8, 256), dtype=BF, device="cuda") for _ in range(2))
    cache = L.KVCache(1, pages, 64, 8, 256, dtype=BF, k=k, v=v)
    gen = torch.Generator().manual_seed(1)
    ids = [pages - 1, 17000, 3, pages - 2]
    for p in ids:
        for t in (k, v):
            t[0, p] = torch.randn((64, 8, 256), generator=gen).to(BF).cuda()
    table = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32)
    q = queries(1, 1, 8, 8, 256, BF, gen)
    small = L.KVCache(1, 4, 64, 8, 256, dtype=BF, k=k[:, ids].contiguous(), v=v[:, ids].contiguous())
    want = check_attn(small, table, q, [250], BF)
    out = torch.zeros_like(want)
    far = torch.tensor([ids], dtype=torch.int32).cuda()
    length = torch.tensor([250], dtype=torch.int32).cuda()
    L.lin_state_attn_decode(cache, layer=0, q=q, out=out, page_table=far, kv_len=length)
    assert torch.equal(out, want)
    new = torch.randn((1, 3, 8, 256), generator=gen).to(BF).cuda()
    L.lin_state_kv_append(cache, layer=0, k=new, v=-new, page_table=far, pos=length)
    assert torch.equal(k[0, pages - 2, 58:61], new[0]) and torch.equal(v[0, pages - 2, 58:61], -new[0])


def test_attn_on_another_stream_and_in_a_graph():
    lens = [900, 33]
    cache, table, gen = make_cache(lens, 16, 2, 128, BF, seed=12)
    q = queries(2, 2, 8, 2, 128, BF, gen).clone()
    want = check_attn(cache, table, q, lens, BF)
    length = torch.tensor(lens, dtype=torch.int32).cuda()
    table = table.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    L.lin_state_attn_decode(cache, layer=0, q=q, out=out, page_table=table, kv_len=length, stream=side)
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    side.synchronize()
    del junk
    assert torch.equal(out, want)
    size = L.lin_state_attn_workspace(cache, batch=2, n_q=2, num_q_heads=8, max_pages=table.shape[1])
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    out2 = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lin_state_attn_decode(cache, layer=0, q=q, out=out2, page_table=table, kv_len=length, workspace=ws)
    for _ in range(2):
        out2.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out2, want)
    # the lengths are read on the device: a replay follows them
    length.copy_(torch.tensor([17, 33], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2, check_attn(cache, table.cpu(), q, [17, 33], BF))


# ---- append ---------------------------------------------------------------------

def check_append(cache, k, v, table, pos, status_want=0, **idx):
    ck, cv = np64(cache.k[0]), np64(cache.v[0])
    O.kv_append(ck, cv, np64(k), np64(v), table.numpy(), pos, **idx)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = {n: torch.tensor(x, dtype=torch.int32).cuda() for n, x in idx.items()}
    L.lin_state_kv_append(cache, layer=0, k=k, v=v, page_table=table.cuda(),
                          pos=torch.tensor(pos, dtype=torch.int32).cuda(), status=status, **dev)
    assert L.lin_state_read_status(status) == status_want
    assert np.array_equal(np64(cache.k[0]), ck) and np.array_equal(np64(cache.v[0]), cv)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,D", [(1, 64), (3, 128), (8, 256), (33, 64)])
@pytest.mark.parametrize("hnd", [False, True])
def test_append_step_prompt_and_prefix(dtype, H, D, hnd):
    pos = [0, 1, 15, 16, -1, 40, 47]
    cache, table, gen = make_cache([max(p, 0) + 21 for p in pos], 16, H, D, dtype, seed=H, hnd=hnd, fill=0.0)
    for n in (1, 21):
        rows = torch.randn((len(pos), n, 2 * H + 1, D), generator=gen).to(dtype).cuda()
        k, v = rows[:, :, :H], rows[:, :, H + 1:]
        check_append(cache, k, v, table, pos)
        check_append(cache, -k, -v, table, pos, n_tok=[0, 1, n // 2, n, n, n, 0])


def test_append_tree_path():
    pos = [0, 30, 5, -1, 7]
    cache, table, gen = make_cache([60] * 5, 7, 2, 64, BF, seed=2, fill=0.0)
    n = 32
    rng = np.random.default_rng(2)
    parent = [[int(rng.integers(max(-1, j - 3), j)) if j else -1 for j in range(n)] for _ in pos]
    parent[0] = list(range(-1, n - 1))
    k = torch.randn((5, n, 2, 64), generator=gen).to(BF).cuda()
    check_append(cache, k, -k, table, pos, parent=parent, accept_node=[31, 20, -1, 3, 0])


def test_append_status_bits():
    pos = [10, 10, 10, 10]
    cache, table, gen = make_cache([40] * 4, 16, 2, 64, BF, seed=6, fill=0.0)
    k = torch.randn((4, 3, 2, 64), generator=gen).to(BF).cuda()
    bad = table.clone()
    bad[1, 0], bad[2, 0] = cache.num_pages, -2
    check_append(cache, k, k, bad, pos, status_want=L.LIN_ST_BAD_PAGE)
    # the table's last entry is -1, a page that is not allocated
    check_append(cache, k, k, table, [10, 16 * table.shape[1] - 1, 0, 0], n_tok=[3, 1, 3, 3],
                 status_want=L.LIN_ST_BAD_PAGE)
    check_append(cache, -k, k, table, [10, 16 * table.shape[1], 2 ** 31 - 1, 0],
                 status_want=L.LIN_ST_BAD_SEQLEN)
    check_append(cache, k, k, table, pos, n_tok=[4, 3, -1, 0], status_want=L.LIN_ST_BAD_ACCEPT)
    check_append(cache, k, -k, table, pos, parent=[[-1, 0, 1], [-1, 1, 0], [-1, -2, 0], [-1, 0, 0]],
                 accept_node=[2, 1, 1, 3], status_want=L.LIN_ST_BAD_TREE)


def test_step_after_step_equals_one_verify():
    """Appending and attending token by token gives what one verify of the
    chain gives, to the rounding of the two orders of summation."""
    lens, n = [50, 7], 4
    cache, table, gen = make_cache([x + n for x in lens], 16, 2, 128, F32, seed=21, fill=0.0)
    rows = torch.randn((2, n, 8, 128), generator=gen).cuda()
    q, k, v = rows[:, :, :4], rows[:, :, 4:6], rows[:, :, 6:]
    steps = []
    for j in range(n):
        at = [x + j for x in lens]
        check_append(cache, k[:, j:j + 1], v[:, j:j + 1], table, at)
        steps.append(check_attn(cache, table, q[:, j:j + 1], [x + 1 for x in at], F32))
    check_append(cache, k, v, table, lens)
    out = check_attn(cache, table, q, [x + n for x in lens], F32)
    assert torch.allclose(out, torch.cat(steps, 1), rtol=1e-4, atol=1e-5)


# ---- norms ------------------------------------------------------------------------

def check_norm(T, C, xt, io, ht, group=0, gate=None, residual=False, scale=1.0, scale_w=False, pre=False,
               seed=0, wide=0, eps=1e-6, x=None, h_out=True):
    gen = torch.Generator().manual_seed(seed)

    def make(*shape, dtype, pad=0):
        t = torch.randn((*shape[:-1], shape[-1] + pad), generator=gen).to(dtype).cuda()
        return t[..., :shape[-1]]

    a = dict(x=make(T, C, dtype=xt, pad=wide) if x is None else x)
    if gate:
        a.update(gate=make(T, C, dtype=io, pad=wide) * 3, gate_act=gate)
    if group:
        a["w_post"] = make(group, dtype=io)
    if residual:
        a["residual"] = make(T, C, dtype=ht, pad=wide)
    if scale_w:
        a["scale_w"] = make(C, dtype=io)
    if pre:
        a.update(w_pre=make(C, dtype=io), y=make(T, C, dtype=io, pad=wide))
    if h_out:
        a["h_out"] = make(T, C, dtype=ht, pad=wide)
    n = {k: np64(t) for k, t in a.items() if torch.is_tensor(t)}
    t, h, y = O.block_norm(n["x"], n.get("gate"), gate, n.get("w_post"), n.get("residual"), scale,
                           n.get("scale_w"), n.get("w_pre"), eps)
    L.lin_state_block_norm(scale=scale, eps=eps, **a)
    # a sum of S squares rounds at most S + 8 times, halved by the root; the
    # gate's exponential and the products another 32
    e_t = np.abs(t) * ((group / 2 + 32) * U)
    e_h = e_t + 2 * np.abs(h) * U
    if h_out:
        got = np64(a["h_out"])
        tol = half_step(ht) * (np.abs(h) + e_h) + e_h
        assert (np.abs(got - h) <= tol + 1e-300).all(), float((np.abs(got - h) - tol).max())
    if pre:
        # h's own errors move the row's mean square by at most 2 max(e_h/|h|) of
        # the part they belong to: bounded by the error vector's norm
        inv = 1.0 / np.sqrt((h ** 2).mean(1, keepdims=True) + eps)
        move = np.sqrt((e_h ** 2).mean(1, keepdims=True)) * inv
        e_y = np.abs(n["w_pre"]) * inv * e_h + np.abs(y) * (move + (C / 2 + 32) * U)
        tol = half_step(io) * (np.abs(y) + e_y) + e_y
        got = np64(a["y"])
        assert (np.abs(got - y) <= tol + 1e-300).all(), float((np.abs(got - y) - tol).max())


@pytest.mark.parametrize("xt,io,ht", [(a, b, c) for a in (BF, F32) for b in (BF, F32) for c in (BF, F32)])
@pytest.mark.parametrize("C,group", [(256, 64), (96, 96), (515, 103)])
def test_norm_types(xt, io, ht, C, group):
    check_norm(5, C, xt, io, ht, group=group, gate="silu", residual=True, scale=0.3, scale_w=True, pre=True)


@pytest.mark.parametrize("C", [1, 7, 8, 31, 32, 40, 64, 100, 128, 1000, 1024, 1533, 2048, 4096, 4104, 5000, 8192,
                               8191, 12288, 20480, 32768, 32767])
def test_norm_widths(C):
    check_norm(3, C, BF, BF, F32, group=C, gate="sigmoid", residual=True, scale=-1.5, pre=True, seed=C)
    check_norm(9, C, F32, BF, BF, pre=True, seed=C)


@pytest.mark.parametrize("C,group", [(128, 8), (128, 16), (512, 128), (4096, 128), (4096, 256), (768, 96), (640, 80),
                                     (1536, 512), (96, 1), (90, 3), (64, 2), (99, 33), (16384, 2048), (24576, 24),
                                     (32760, 8190)])
def test_norm_groups(C, group):
    check_norm(4, C, BF, BF, BF, group=group, gate="silu", seed=group)


@pytest.mark.parametrize("T", [1, 2, 33, 1000])
@pytest.mark.parametrize("C", [64, 1536])
@pytest.mark.parametrize("wide", [0, 8, 3])
def test_norm_rows_and_strides(T, C, wide):
    check_norm(T, C, BF, BF, F32, group=C // 2, gate="silu", residual=True, scale=0.5, pre=True, wide=wide)


def test_norm_parts_alone():
    for kw in (dict(), dict(residual=True), dict(scale=2.0, scale_w=True), dict(pre=True, h_out=False),
               dict(gate="sigmoid"), dict(group=64), dict(group=64, pre=True, h_out=False)):
        check_norm(6, 256, BF, BF, BF, **kw)


def test_norm_in_place_and_on_another_stream():
    gen = torch.Generator().manual_seed(4)
    x, r, z = (torch.randn((70, 384), generator=gen).to(BF).cuda() for _ in range(3))
    w = torch.randn(384, generator=gen).to(BF).cuda()
    h, y = torch.empty_like(x), torch.empty_like(x)
    L.lin_state_block_norm(x=x, gate=z, gate_act="silu", w_post=w, residual=r, w_pre=w, h_out=h, y=y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x2, r2 = x.clone(), r.clone()
    torch.cuda.synchronize()
    L.lin_state_block_norm(x=x2, gate=z, gate_act="silu", w_post=w, residual=r2, w_pre=w, h_out=r2, y=x2, stream=side)
    side.synchronize()
    assert torch.equal(r2, h) and torch.equal(x2, y)


def test_norm_extreme_rows():
    """Zero rows (eps alone), tiny rows, gates far out (SiLU and sigmoid go to 0
    or pass the value), and an infinity that stays in its row."""
    x = torch.zeros((4, 128), device="cuda")
    x[1] = 1e-20
    x[2] = 1e15
    check_norm(4, 128, F32, F32, F32, group=128, pre=True, x=x)
    z = torch.tensor([[-200.0, -100.0, 0.0, 100.0, 200.0, 3e38, -3e38, 1.0]], device="cuda")
    one = torch.ones((1, 8), device="cuda")
    h = torch.empty((1, 8), device="cuda")
    L.lin_state_block_norm(x=one, gate=z, gate_act="sigmoid", h_out=h)
    assert torch.allclose(h.double(), torch.sigmoid(z.double()), rtol=1e-5, atol=1e-37)
    x = torch.randn((3, 128), device="cuda")
    h, ref = torch.empty_like(x), torch.empty_like(x)
    w = torch.ones(128, device="cuda")
    L.lin_state_block_norm(x=x, w_post=w, h_out=ref)
    x[1, 5] = float("inf")
    L.lin_state_block_norm(x=x, w_post=w, h_out=h)
    assert torch.equal(h[0], ref[0]) and torch.equal(h[2], ref[2]) and h[1].isnan().any()


def test_binding_refuses_wrong_device_tensors():
    c = L.KVCache(1, 4, 8, 2, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    new = torch.zeros((3, 2, 2, 64), dtype=BF, device="cuda")
    table, pos = torch.zeros((3, 4), **i32), torch.zeros(3, **i32)
    with pytest.raises(ValueError, match="pos: want a contiguous int32"):
        L.lin_state_kv_append(c, layer=0, k=new, v=new, page_table=table, pos=pos.long())
    with pytest.raises(ValueError, match="n_tok: want a contiguous int32"):
        L.lin_state_kv_append(c, layer=0, k=new, v=new, page_table=table, pos=pos, n_tok=pos[:2])
    with pytest.raises(ValueError, match="pos: want a CUDA tensor"):
        L.lin_state_kv_append(c, layer=0, k=new, v=new, page_table=table, pos=pos.cpu())
    q = torch.zeros((3, 2, 8, 64), dtype=BF, device="cuda")
    with pytest.raises(L.LinStateError, match="workspace"):
        L.lin_state_attn_decode(c, layer=0, q=q, out=q.clone(), page_table=table, kv_len=pos,
                                workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(L.LinStateError, match="multiple"):
        L.lin_state_attn_decode(c, layer=0, q=q[:, :, :3], out=q[:, :, :3].contiguous(), page_table=table, kv_len=pos)
    x = torch.zeros((3, 64), dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="one dtype"):
        L.lin_state_block_norm(x=x, gate=x, gate_act="silu", w_post=torch.ones(64, device="cuda"), h_out=x)
    with pytest.raises(ValueError, match="h_out: want"):
        L.lin_state_block_norm(x=x, h_out=x[:, :32])
