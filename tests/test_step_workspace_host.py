"""One attention workspace, sized for the largest call, serves the smaller ones.
CPU only: sizes alone."""

import ctypes

import pytest

import linear_attention_state_chunked_gb300 as L
from tests.test_step_host import attn_args, cache_desc

ROWS = [1, 2, 3, 4, 8, 16, 17, 32]     # query tokens
PAGES = [0, 1, 3, 4, 5, 16, 17, 64, 1000, 100000]


def size(c, **kw):
    return L.lib.lin_state_attn_workspace(ctypes.byref(c), ctypes.byref(attn_args(**kw)))


@pytest.mark.parametrize("dt", [L.LIN_BF16, L.LIN_F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ps", [16, 64])
@pytest.mark.parametrize("H,Hq", [(1, 1), (2, 16), (1, 40), (8, 32)])
def test_the_size_never_shrinks(dt, D, ps, H, Hq):
    c = cache_desc(ps=ps, H=H, D=D, dt=dt)
    for b0, b1 in ((1, 1), (1, 3), (3, 64), (64, 64), (64, 700)):
        for n0, n1 in [(a, b) for a in ROWS for b in ROWS if a <= b]:
            for p0, p1 in zip(PAGES, PAGES[1:]):
                small = [size(c, batch=b0, n_q=n0, num_q_heads=Hq, max_pages=p0, out_dtype=o)
                         for o in (L.LIN_BF16, L.LIN_F32)]
                large = [size(c, batch=b1, n_q=n1, num_q_heads=Hq, max_pages=p1, out_dtype=o)
                         for o in (L.LIN_BF16, L.LIN_F32)]
                assert 0 < max(small) <= min(large), (b0, b1, n0, n1, p0, p1)


def test_more_query_heads_need_no_less():
    c = cache_desc(H=2)
    sizes = [size(c, batch=64, num_q_heads=2 * g, n_q=1, max_pages=128) for g in range(1, 200)]
    assert sizes == sorted(sizes)
