"""Decode-step operators on the GPU at the edges of their contract: calls in
which nothing is attended, NaN and infinities that are visible, long sums,
workspaces kept for a largest call."""

import numpy as np
import pytest
import torch

import linear_attention_state_chunked_gb300 as L
from tests.test_gpu_step import check_attn, make_cache, queries

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype,n,G", [(BF, 1, 8), (BF, 4, 8), (F32, 1, 4)])
@pytest.mark.parametrize("lens,status_want", [((-1,), 0), ((1 << 20,), L.LIN_ST_BAD_SEQLEN),
                                              ((-1, 1 << 20, -7), L.LIN_ST_BAD_SEQLEN)])
def test_a_call_without_work_ends_before_the_next_launch(dtype, n, G, lens, status_want):
    """A slot that is all padding, or one request that is too long: what runs
    next in the stream has the workspace and the lengths for itself."""
    B = len(lens)
    cache = L.KVCache(1, 40, 64, 1, 128, dtype=dtype)
    q = torch.randn((B, n, G, 128), device="cuda").to(dtype)
    out = torch.full_like(q, 7.0)
    table = torch.arange(40, dtype=torch.int32, device="cuda").expand(B, 40).contiguous()
    size = L.lin_state_attn_workspace(cache, batch=B, n_q=n, num_q_heads=G, max_pages=40)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    length = i32(*lens)
    for _ in range(200):
        L.lin_state_attn_decode(cache, layer=0, q=q, out=out, page_table=table, kv_len=length, workspace=ws,
                                status=status)
        ws.fill_(255)
        assert bool((ws == 255).all())
    assert L.lin_state_read_status(status) == status_want
    assert bool((out == 7.0).all())


def pattern(bits, dtype):
    """One value of this bit pattern."""
    if dtype == F32:
        return torch.tensor(bits - (1 << 32) if bits >> 31 else bits, dtype=torch.int32).view(F32)
    return torch.tensor(bits - (1 << 16) if bits >> 15 else bits, dtype=torch.int16).view(BF)


NANS = [(F32, 0x7fffffff), (F32, 0xffffffff), (F32, 0x7fc00000), (F32, 0x7f800001), (F32, 0xffbfffff),
        (BF, 0x7fff), (BF, 0xffff), (BF, 0x7f81)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", [(1, 4), (2, 12), (4, 12), (2, 40)])
@pytest.mark.parametrize("dtype,bits", NANS)
def test_a_visible_nan_reaches_every_output_that_uses_it(dtype, bits, D, n, G):
    """A NaN of any payload in a query, a key or a value that is seen: NaN in the
    outputs it has a part in, the others as they were, bit for bit."""
    lens, ps = [200, 75, 40], 16
    gen = torch.Generator(device="cuda").manual_seed(D + n + G)
    pages = [-(-x // ps) for x in lens]
    table = torch.zeros((3, max(pages)), dtype=torch.int32)
    for r in range(3):
        table[r, :pages[r]] = torch.arange(sum(pages[:r]), sum(pages[:r + 1]))
    k, v = (torch.randn((1, sum(pages), ps, 2, D), generator=gen, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn((3, n, 2 * G, D), generator=gen, device="cuda").to(dtype)
    bad = pattern(bits, dtype).cuda()

    def attend(q, k, v):
        out = torch.empty((3, n, 2 * G, D), dtype=dtype, device="cuda")
        L.lin_state_attn_decode(L.KVCache(1, sum(pages), ps, 2, D, dtype=dtype, k=k, v=v), layer=0, q=q, out=out,
                                page_table=table.cuda(), kv_len=i32(*lens))
        return out

    plain = attend(q, k, v)
    assert not plain.isnan().any()
    q2 = q.clone()
    q2[1, n - 1, G + 1, 7] = bad
    hit = torch.zeros(plain.shape, dtype=torch.bool, device="cuda")
    hit[1, n - 1, G + 1] = True
    out = attend(q2, k, v)
    assert bool(out[hit].isnan().all()) and torch.equal(out[~hit], plain[~hit])
    page, row = int(table[0, 33 // ps]), 33 % ps  # token 33 of request 0, kv head 1
    for in_value in (False, True):
        k2, v2 = k.clone(), v.clone()
        (v2 if in_value else k2)[0, page, row, 1, 9] = bad
        hit = torch.zeros(plain.shape, dtype=torch.bool, device="cuda")
        hit[0, :, G:, 9 if in_value else slice(None)] = True
        out = attend(q, k2, v2)
        assert bool(out[hit].isnan().all()) and torch.equal(out[~hit], plain[~hit])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", [(1, 4), (2, 12), (2, 40)])
@pytest.mark.parametrize("bits", [0x7f7fffff, 0xff7fffff, 0x7f7ff000, 0x7f7fefff])
def test_fp32_values_next_to_the_largest(n, G, D, bits):
    """Keys, queries and values at the end of the range stay finite: products of
    the largest with 2^-125 are 2^3, and one token's weight is 1. Tolerances as
    for other values (2 S (D + 16 + c) u + (L + 16) u + 12 u of sum p |v|, u =
    2^-24), with c = 24: three terms of 2^-22, and 2^-21 where the largest value's
    first part is cut off. A value leaves 2^-12 to the end of the range, as the
    weight itself may round to more than 1."""
    big = float(pattern(bits, F32))
    gen = torch.Generator(device="cuda").manual_seed(D)
    k, v = (torch.randn((1, 2, 16, 1, D), generator=gen, device="cuda") for _ in range(2))
    q = torch.randn((1, n, G, D), generator=gen, device="cuda")

    def check(q, k, v, length):
        out = torch.empty((1, n, G, D), device="cuda")
        L.lin_state_attn_decode(L.KVCache(1, 2, 16, 1, D, dtype=F32, k=k, v=v), layer=0, q=q, out=out,
                                page_table=i32(1, 0)[None].contiguous(), kv_len=i32(length))
        kk, vv = (t[0, [1, 0]].reshape(32, D)[:length].double() for t in (k, v))
        s = torch.einsum("jhd,td->jht", q[0].double(), kk) * D ** -0.5
        hidden = torch.arange(length, device="cuda") > length - n + torch.arange(n, device="cuda")[:, None]
        p = torch.softmax(s.masked_fill(hidden[:, None], -torch.inf), -1)
        spread = float((q[0].double().abs()[:, :, None] * kk.abs()).sum(-1).max()) * D ** -0.5
        tol = (p @ vv.abs()) * (2 * spread * (D + 16 + 24) + length + 16 + 12) * 2.0 ** -24
        assert bool(torch.isfinite(out).all())
        assert bool(((out[0].double() - p @ vv).abs() <= tol).all())

    q2, k2 = q.clone(), k.clone()
    q2[..., 5], k2[0, 1, 3, 0, 5] = 2.0 ** -125, big
    check(q2, k2, v, 30)
    q2, k2 = q.clone(), k.clone()
    q2[..., 5], k2[..., 5] = big, 2.0 ** -125
    check(q2, k2, v, 30)
    v2 = v.clone()
    top = float(pattern(0x7f7ff801, F32))
    v2[0, 1, 0, 0, 5] = max(-top, min(top, big))
    check(q, k, v2, n)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", [(1, 8), (17, 1), (4, 8), (8, 8), (3, 43)])
@pytest.mark.parametrize("positive", [False, True])
def test_fp32_outputs_of_a_bf16_cache_do_not_lose_with_the_length(D, n, G, positive):
    """304 requests that share one sequence's pages, so that the longer one stays
    in one piece: 256 and 16,384 tokens to one bound, 2^-20 of the outputs, as for
    fp32 caches (rounded sums grow as the outputs' own random sum does). Values of
    one sign would show any bias of the additions."""
    B = 304
    for length in (256, 16384):
        gen = torch.Generator(device="cuda").manual_seed(D + n)
        k, v = (torch.randn((1, length // 64, 64, 1, D), generator=gen, device="cuda") for _ in range(2))
        k, v = k.to(BF), (v.abs() + 1 if positive else v).to(BF)
        q = torch.randn((B, n, G, D), generator=gen, device="cuda").to(BF)
        out = torch.empty((B, n, G, D), dtype=F32, device="cuda")
        table = torch.arange(length // 64, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
        L.lin_state_attn_decode(L.KVCache(1, length // 64, 64, 1, D, dtype=BF, k=k, v=v), layer=0, q=q, out=out,
                                page_table=table, kv_len=torch.full((B,), length, dtype=torch.int32, device="cuda"))
        hidden = torch.arange(length, device="cuda") > length - n + torch.arange(n, device="cuda")[:, None]
        for r in (0, 151, 303):
            s = torch.einsum("jhd,td->jht", q[r].double(), k.reshape(length, D).double()) * D ** -0.5
            want = torch.softmax(s.masked_fill(hidden[:, None], -torch.inf), -1) @ v.reshape(length, D).double()
            assert float((out[r] - want).norm() / want.norm()) < 2.0 ** -20, (length, r)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_workspace_of_the_largest_call_serves_the_smaller(D, dtype):
    """A server keeps one workspace, of its most drafts and its widest table."""
    B, H, G, ps, wide = 9, 2, 8, 16, 80
    cache = L.KVCache(1, wide, ps, H, D, dtype=dtype, k=torch.randn((1, wide, ps, H, D), device="cuda").to(dtype),
                      v=torch.randn((1, wide, ps, H, D), device="cuda").to(dtype))
    ws = torch.empty(L.lin_state_attn_workspace(cache, batch=B, n_q=16, num_q_heads=H * G, max_pages=wide),
                     dtype=torch.uint8, device="cuda")
    for b, n, pages in [(9, 16, 80), (9, 1, 80), (9, 2, 80), (9, 4, 80), (9, 8, 80), (1, 1, 80), (9, 4, 16), (9, 4, 17),
                        (3, 3, 4), (9, 1, 1)]:
        q = torch.randn((b, n, H * G, D), device="cuda").to(dtype)
        table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(b, pages).contiguous()
        length = torch.full((b,), pages * ps - 3, dtype=torch.int32, device="cuda")
        for out_dtype in (BF, F32):
            outs = [torch.empty(q.shape, dtype=out_dtype, device="cuda") for _ in range(2)]
            for out, w in zip(outs, (ws, None)):
                L.lin_state_attn_decode(cache, layer=0, q=q, out=out, page_table=table, kv_len=length, workspace=w)
            assert torch.equal(*outs)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq", [2, 64])
def test_strides_of_single_requests_and_tokens_are_not_used(dtype, Hq):
    """One request of one token, a cache of one layer and page: any strides there."""
    gen = torch.Generator(device="cuda").manual_seed(Hq)
    k, v = (torch.randn((1, 1, 16, 1, 64), generator=gen, device="cuda").to(dtype) for _ in range(2))
    q, new = (torch.randn((1, 1, h, 64), generator=gen, device="cuda").to(dtype) for h in (Hq, 1))
    want = torch.empty_like(q)

    def attend(k, v, q, new, out):
        cache = L.KVCache(1, 1, 16, 1, 64, dtype=dtype, k=k, v=v)
        L.lin_state_kv_append(cache, layer=0, k=new, v=new, page_table=i32(0)[None], pos=i32(9))
        L.lin_state_attn_decode(cache, layer=0, q=q, out=out, page_table=i32(0)[None], kv_len=i32(10))
        return out

    want = attend(k, v, q, new, torch.empty_like(q))
    odd = [torch.as_strided(t, t.shape, (3, 5, *t.stride()[2:])) for t in (k, v, q, new)]
    assert torch.equal(attend(*odd, torch.empty_like(q)), want)


@pytest.mark.parametrize("n", [1, 4])
def test_the_longest_request_and_one_token_more(n):
    """2^31 - 65536 tokens, whose table names one page of 65,536 tokens over and
    over: the output is that page's mean, as all keys are 0, to the 2^31 / 608 / 16
    additions of a group of warps that rounds each by 2^-24 at most, below 2^-6. One
    token more is left out."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    k = torch.zeros((1, 1, 65536, 1, 64), dtype=BF, device="cuda")
    v = torch.randn(k.shape, generator=gen, device="cuda").abs().to(BF)
    cache = L.KVCache(1, 1, 65536, 1, 64, dtype=BF, k=k, v=v)
    q = torch.randn((1, n, 8, 64), generator=gen, device="cuda").to(BF)
    table = torch.zeros((1, 32768), dtype=torch.int32, device="cuda")
    for length, want in ((2 ** 31 - 65536, v.double().mean((0, 1, 2, 3))), (2 ** 31 - 65535, None)):
        out = torch.full(q.shape, 7.0, dtype=F32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        L.lin_state_attn_decode(cache, layer=0, q=q, out=out, page_table=table, kv_len=i32(length), status=status)
        assert L.lin_state_read_status(status) == (0 if want is not None else L.LIN_ST_BAD_SEQLEN)
        if want is None:
            assert bool((out == 7.0).all())
        else:
            assert bool(((out - want).abs() <= want * 2.0 ** -6).all())



def shift_of_bf16_outputs(D, n, G, length):
    """Mean of (output - correctly rounded output) / output for requests that share
    one sequence, so that each stays in one piece. Values of one sign, channels of
    different sizes, so that outputs lie anywhere between two bf16 values: what an
    accumulation loses shows in full as outputs that round to the neighbour."""
    B = 304
    gen = torch.Generator(device="cuda").manual_seed(D + n)
    k, v = (torch.randn((1, length // 64, 64, 1, D), generator=gen, device="cuda") for _ in range(2))
    size = 2.0 ** torch.rand(D, generator=gen, device="cuda")
    k, v = k.to(BF), ((v.abs() + 1) * size).to(BF)
    q = torch.randn((B, n, G, D), generator=gen, device="cuda").to(BF)
    out = torch.empty_like(q)
    table = torch.arange(length // 64, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    L.lin_state_attn_decode(L.KVCache(1, length // 64, 64, 1, D, dtype=BF, k=k, v=v), layer=0, q=q, out=out,
                            page_table=table, kv_len=torch.full((B,), length, dtype=torch.int32, device="cuda"))
    hidden = torch.arange(length, device="cuda") > length - n + torch.arange(n, device="cuda")[:, None]
    off = []
    for r in range(0, B, 38):
        s = torch.einsum("jhd,td->jht", q[r].double(), k.reshape(length, D).double()) * D ** -0.5
        want = torch.softmax(s.masked_fill(hidden[:, None], -torch.inf), -1) @ v.reshape(length, D).double()
        off.append(((out[r].double() - want.to(BF).double()) / want).mean())
    return abs(float(torch.stack(off).mean()))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", [(1, 8), (2, 8)])
def test_bf16_outputs_lose_nothing_over_a_long_piece(D, n, G):
    """Up to 16 rows: sums that are rounded to nearest shift nothing, and weights
    in two parts less than 2^-17; another 2^-17 for chance. (A sum that cut off with every
    16 tokens took 2^-12 over half as many.)"""
    assert shift_of_bf16_outputs(D, n, G, 1 << 18) < 2.0 ** -16


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G", [(4, 8), (8, 8), (8, 16)])
def test_bf16_outputs_of_many_rows_lose_little_over_a_long_piece(D, n, G):
    """More than 16 rows: a run of 32,768 tokens is 4,096 products of 16 tokens, two to
    each, that lose a unit of the sum's last place at most: 4,096 x 2^-23 = 2^-11,
    whatever the length. (Over 262,144 tokens at a stretch 128 rows lost 2^-9.)"""
    assert shift_of_bf16_outputs(D, n, G, 1 << 18) < 2.0 ** -11


@pytest.mark.parametrize("D,n,G", [(64, 8, 8), (128, 4, 8), (256, 16, 8)])
def test_runs_of_a_long_piece_beside_short_requests(D, n, G):
    """Whole items of several runs, items that begin and end in a range, and
    requests without work, against 64 bits, with the bound of the other
    tests; a bad tree is left out although its runs leave sums."""
    long, ps = 70001, 64
    pages = -(-long // ps)
    gen = torch.Generator(device="cuda").manual_seed(D)
    k, v = (torch.randn((1, pages, ps, 1, D), generator=gen, device="cuda").to(BF) for _ in range(2))
    lens = [long, 3, 32768, 32769 + n, -1, 0, 65536, 40000] + [long] * 300
    bad = {7, 200}
    q = torch.randn((len(lens), n, G, D), generator=gen, device="cuda").to(BF)
    out = torch.full_like(q, 7.0)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(len(lens), -1).contiguous()
    parent = torch.arange(-1, n - 1, dtype=torch.int32, device="cuda").expand(len(lens), -1).contiguous()
    for r in bad:
        parent[r, 1] = 5 if n > 5 else 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lin_state_attn_decode(L.KVCache(1, pages, ps, 1, D, dtype=BF, k=k, v=v), layer=0, q=q, out=out, page_table=table,
                            kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"), parent=parent, status=status)
    assert L.lin_state_read_status(status) == L.LIN_ST_BAD_TREE
    for r in [0, 1, 2, 3, 4, 5, 6, 7, 8, 100, 200, 307]:
        if lens[r] < 0 or r in bad:
            assert bool((out[r] == 7.0).all())
            continue
        kk, vv = (t.reshape(-1, D)[:lens[r]].double() for t in (k, v))
        s = torch.einsum("jhd,td->jht", q[r].double(), kk) * D ** -0.5
        hidden = torch.arange(lens[r], device="cuda") > lens[r] - n + torch.arange(n, device="cuda")[:, None]
        p = torch.softmax(s.masked_fill(hidden[:, None], -torch.inf), -1).nan_to_num(0.0)
        want, reach = p @ vv, p @ vv.abs()
        spread = float((q[r].double().abs().reshape(-1, D) @ kk.abs().T).max()) * D ** -0.5 if lens[r] else 0.0
        inner = 2 * spread * (D + 16) * 2.0 ** -24 + (lens[r] + 16) * 2.0 ** -24 + 2.0 ** -16
        assert bool(((out[r].double() - want).abs() <= 2.0 ** -8 * want.abs() + reach * inner).all()), r


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B", [20, 38, 39, 100])
def test_short_requests_of_few_rows_in_any_batch(D, B):
    """17 to 32 rows over at most 256 tokens, on both sides of the batch from which
    heads of 256 take another kernel; the last requests as in a batch of their own."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(-1, 241, B)]
    cache, table, gen = make_cache(lens, 16, 2, D, BF, seed=B)
    q = queries(B, 3, 16, 2, D, BF, gen)
    assert table.shape[1] * 16 <= 256
    out = check_attn(cache, table, q, lens, BF)
    few = check_attn(cache, table[-4:].contiguous(), q[-4:], lens[-4:], BF)
    seen = torch.tensor(lens[-4:], device="cuda") >= 0
    assert bool((out[-4:][seen].float() - few[seen].float()).abs().max() < 2.0 ** -6)


@pytest.mark.parametrize("dtype,n,G", [(BF, 2, 4), (BF, 8, 8), (F32, 4, 8)])
@pytest.mark.parametrize("B", [3, 70])
def test_a_split_request_that_is_left_out(dtype, n, G, B):
    """A bad tree and a length past the table in requests that are cut over several
    ranges, few of many parts and many of few: their outputs stay as they are, and the
    other requests' are those of a batch without fault, bit for bit."""
    pages, ps = 100, 64
    gen = torch.Generator(device="cuda").manual_seed(B + n)
    k, v = (torch.randn((1, pages, ps, 1, 64), generator=gen, device="cuda").to(dtype) for _ in range(2))
    cache = L.KVCache(1, pages, ps, 1, 64, dtype=dtype, k=k, v=v)
    q = torch.randn((B, n, G, 64), generator=gen, device="cuda").to(dtype)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    length = torch.full((B,), pages * ps - 7, dtype=torch.int32, device="cuda")
    length[2] = -1
    tree = torch.arange(-1, n - 1, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()

    def attend(length, tree, status_want):
        out = torch.full_like(q, 7.0)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        L.lin_state_attn_decode(cache, layer=0, q=q, out=out, page_table=table, kv_len=length, parent=tree, status=status)
        assert L.lin_state_read_status(status) == status_want
        return out

    want = attend(length, tree, 0)
    assert bool((want[2] == 7.0).all())
    bad_tree, too_long = tree.clone(), length.clone()
    bad_tree[1, 1], too_long[2] = 1, pages * ps + 1
    out = attend(too_long, bad_tree, L.LIN_ST_BAD_TREE | L.LIN_ST_BAD_SEQLEN)
    want[1] = 7.0
    assert torch.equal(out, want)
