"""Decode-step operators on the GPU at the edges of their contract: calls in
which nothing is attended, NaN and infinities that are visible, long sums,
workspaces kept for a largest call."""

import pytest
import torch

import linear_attention_state_chunked_gb300 as L

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
