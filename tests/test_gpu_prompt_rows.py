"""Chunk attention: a row's output goes by its own query and what it sees, whatever the
rows beside it hold. Outputs are compared bit for bit with those of a call in which the
other rows are ordinary, which are looked over against the fp64 oracle."""

import numpy as np
import pytest
import torch

import linear_attention_state_chunked_gb300 as L
from tests.test_gpu_prompt import BF, F32, check_chunk, chunk_inputs, i32

pytestmark = pytest.mark.gpu


def room(q, table, page_size, two):
    """The table, or one so wide that requests of many rows go in items of two row tiles."""
    if not two:
        return table.cuda()
    wide = torch.full((table.shape[0], -(-(1 << 26) // (q.shape[0] * q.shape[1] * page_size)) + table.shape[1]), 1 << 30,
                      dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    return wide.cuda()


def attend(cache, table, q, cu, lens, dtype):
    out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lin_state_attn_chunk(cache, layer=0, q=q, out=out, page_table=table, cu_seqlens=i32(cu), kv_len=i32(lens), status=status)
    return out, L.lin_state_read_status(status)


def growing(D, B, n, cached, dtype, ps=16):
    """B requests over the same pages, so many that a CTA goes through whole items. Scores that
    grow along the keys by more than 2^120 in weight, from the first tile on."""
    cache, table, q, cu, lens = chunk_inputs([cached], [n], ps, 4, 2, D, dtype, seed=D)
    t = torch.arange(lens[0])
    pages = table[0, t // ps].long().cuda()
    for h in range(2):
        key = torch.zeros(lens[0], D)
        key[:, 0] = (1.0 + t / 20.0) * (1.0 if h == 0 else (t % 3 == 0).float())
        cache.k[0][pages, (t % ps).cuda(), h] = key.to(dtype).cuda()
    gen = torch.Generator().manual_seed(1)
    q = torch.randn((n, 4, D), generator=gen)
    q[:, :, 0] = torch.rand((n, 4), generator=gen) * 60 - 20
    return cache, table.repeat(B, 1), q.to(dtype).cuda().repeat(B, 1, 1), np.arange(B + 1) * n, lens * B


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("what", [float("nan"), -float("inf")])
@pytest.mark.parametrize("dtype,D,B,n,cached", [(BF, 64, 70, 200, 900), (BF, 64, 160, 200, 900), (BF, 128, 70, 200, 900),
                                                (BF, 128, 160, 200, 900), (BF, 256, 140, 100, 900), (BF, 256, 160, 100, 900),
                                                (BF, 128, 60, 3, 5000), (F32, 64, 60, 90, 900), (F32, 256, 60, 20, 900)])
def test_a_query_that_is_no_number_leaves_its_neighbours_alone(dtype, D, B, n, cached, what, two):
    """One head of one token of each request whose scores are all NaN, or all -infinity, so that
    its row never has a maximum: the rows beside it, whose scores grow, give the bits of the
    call without. Items cut into ranges (the smaller batches), and whole ones by the counter."""
    cache, table, q, cu, lens = growing(D, B, n, cached, dtype)
    if B < 160 and what != what and not two:
        check_chunk(cache, table, q, cu, lens, dtype)
    table = room(q, table, 16, two)
    plain, _ = attend(cache, table, q, cu, lens, dtype)
    assert torch.isfinite(plain).all()
    for token in {0, n // 2, n - 1}:
        for head in (0, 1):  # (of the first kv head, whose keys' first channel is positive)
            x = q.clone()
            x[token::n, head, 0] = what
            out, status = attend(cache, table, x, cu, lens, dtype)
            assert status == 0
            other = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
            other[token::n, head] = False
            assert torch.equal(out[other], plain[other]), (token, head)
            if what != what:
                assert torch.isnan(out[token::n, head]).all()


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("D,ps", [(64, 16), (64, 7), (128, 16), (128, 9), (256, 16), (256, 5)])
def test_values_that_are_no_number_beside_pages_that_are_none(D, ps, two):
    """Tiles that are looked over, with infinities and NaN on some pages and others that are
    not to be read: rows before the values keep their bits, rows that see them do not pass
    for finite, and what lies on no page counts for nothing."""
    cache, table, q, cu, lens = chunk_inputs([40, 0], [150, 290], ps, 4, 2, D, BF, seed=D + ps)
    bad = [-1, cache.num_pages, 1 << 30, -(1 << 31)]
    for r in (0, 1):
        for k, page in enumerate(range(50 // ps, lens[r] // ps, 60 // ps)):
            table[r, page] = bad[k % 4]
    wide = room(q, table, ps, two)
    plain, status = attend(cache, wide, q, cu, lens, BF)
    assert status == L.LIN_ST_BAD_PAGE and torch.isfinite(plain).all()
    check_chunk(cache, table, q, cu, lens, BF, status_want=L.LIN_ST_BAD_PAGE)
    # one visible from token 100 (or the next that has a page) on, and one later
    first = []
    for r in (0, 1):
        for at in (100, lens[r] - 20):
            t = next(t for t in range(at, lens[r]) if 0 <= table[r, t // ps] < cache.num_pages)
            cache.v[0, table[r, t // ps], t % ps] = float("nan") if at == 100 else float("inf")
            if at == 100:
                first.append(t)
    wild, status = attend(cache, wide, q, cu, lens, BF)
    assert status == L.LIN_ST_BAD_PAGE
    for r, cached in ((0, 40), (1, 0)):
        row = int(cu[r]) + first[r] - cached  # whose query is the first to see it
        assert torch.equal(wild[cu[r]:row], plain[cu[r]:row])
        assert not torch.isfinite(wild[row:cu[r + 1]]).any()
