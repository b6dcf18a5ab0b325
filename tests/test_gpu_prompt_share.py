"""Chunk attention: how a batch's work is shared out goes by its lengths, not by the room
that the call has: a few rows over a long cache in a captured call with room for many
prompts, or beside them."""

import numpy as np
import pytest
import torch

import linear_attention_state_chunked_gb300 as L
from tests.test_gpu_prompt import BF, check_chunk, chunk_inputs, i32

pytestmark = pytest.mark.gpu


class Call:
    """A captured call over a cache of random values, with room for `room` rows."""

    def __init__(self, new, cached, room, Hq, Hkv, D, ps=64):
        lens = [a + b for a, b in zip(new, cached)]
        need = [-(-n // ps) for n in lens]
        table = torch.full((len(new), max(need)), -1, dtype=torch.int32)
        for r, k in enumerate(need):
            table[r, :k] = torch.arange(k, dtype=torch.int32) + sum(need[:r])
        gen = torch.Generator(device="cuda").manual_seed(0)
        k, v = (torch.randn((1, sum(need), ps, Hkv, D), generator=gen, device="cuda").to(BF) for _ in range(2))
        self.cache = L.KVCache(1, sum(need), ps, Hkv, D, k=k, v=v)
        q = torch.randn((room, Hq, D), generator=gen, device="cuda").to(BF)
        self.out = torch.zeros_like(q)
        size = L.lin_state_attn_chunk_workspace(self.cache, batch=len(new), tokens=room, num_q_heads=Hq, max_pages=max(need))
        args = dict(layer=0, q=q, out=self.out, page_table=table.cuda(), cu_seqlens=i32(np.concatenate([[0], np.cumsum(new)])),
                    kv_len=i32(lens), workspace=torch.empty(size, dtype=torch.uint8, device="cuda"))
        L.lin_state_attn_chunk(self.cache, **args)
        torch.cuda.synchronize()
        self.args, self.graph = args, torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            for _ in range(5):
                L.lin_state_attn_chunk(self.cache, **args)

    def us(self):
        """Of the quickest of some replays."""
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        best = float("inf")
        for _ in range(6):
            start.record()
            self.graph.replay()
            end.record()
            torch.cuda.synchronize()
            best = min(best, start.elapsed_time(end) * 200)
        return best


def test_room_for_many_prompts_does_not_leave_a_long_request_to_a_few_blocks():
    """64 tokens after 100,000, in a call of their own and in one with room for 32,768 rows,
    where the four items must be cut as well: the work is the same, and the time was
    about 20 times as long where they were not."""
    own, roomy = (Call([64], [100000], room, 16, 2, 128) for room in (64, 32768))
    assert roomy.us() < 4 * own.us()
    # other items (the room chooses their rows), so other sums: two bf16 roundings and the weights'
    a, b = own.out.double(), roomy.out[:64].double()
    assert float((a - b).norm() / b.norm()) < 2.0 ** -7
    assert not roomy.out[64:].any()


@pytest.mark.parametrize("at", [0, 8])
def test_one_long_request_does_not_outlast_the_prompts_beside_it(at):
    """A single token after 128,000 before or behind 8 prompts of 2,048 tokens: no longer than twice
    the prompts and the token in calls of their own (about seven times, where one block had
    all its keys)."""
    new, cached = [2048] * 8, [0] * 8
    alone, token = Call(new, cached, 8 * 2048, 16, 2, 128), Call([1], [128000], 1, 16, 2, 128)
    new.insert(at, 1)
    cached.insert(at, 128000)
    both = Call(new, cached, 16 * 2048, 16, 2, 128)
    assert both.us() < 2 * (alone.us() + token.us())


@pytest.mark.parametrize("D,Hq,Hkv,ps", [(64, 8, 8, 16), (128, 16, 4, 64), (256, 16, 4, 8)])
@pytest.mark.parametrize("where", ["first", "last", "both", "none"])
def test_batches_with_room_and_long_requests(D, Hq, Hkv, ps, where):
    """Room for more than four items to a CTA: short prompts with requests of a few tokens over
    a cache many times their length, so that items are cut, and without, so that they are not."""
    rng = np.random.default_rng(D)
    cached = rng.integers(0, 200, 60).tolist()
    new = rng.choice([0, 1, 2, 63, 64, 65, 130, 260], 60).tolist()
    cached[7], new[7] = -1, 0
    if where in ("first", "both"):
        cached[0], new[0] = 9000, 3
    if where in ("last", "both"):
        cached[-1], new[-1] = 12000, 1
    m = (256 if D < 256 else 128) // (Hq // Hkv)
    rows = int(4.5 * 152 / Hkv * m)
    x = chunk_inputs(cached, new, ps, Hq, Hkv, D, BF, seed=D, spare=max(0, rows - sum(new)))
    check_chunk(*x, BF)


def test_a_captured_call_goes_from_one_way_to_the_other():
    """Replays whose lengths leave items whole, cut them, and leave them whole again, each with
    what the one before left in the workspace: the bits of an eager call with another."""
    T, B, ps, H, D = 9760, 40, 16, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    wide = 30400 // ps
    k, v = (torch.randn((1, wide, ps, H, D), generator=gen, device="cuda").to(BF) for _ in range(2))
    cache = L.KVCache(1, wide, ps, H, D, k=k, v=v)
    table = torch.arange(wide, dtype=torch.int32, device="cuda").repeat(B, 1)  # (requests may share pages)
    q = torch.randn((T, 8 * H, D), generator=gen, device="cuda").to(BF)
    cu, lens = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.full((B,), -1, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    size = L.lin_state_attn_chunk_workspace(cache, batch=B, tokens=T, num_q_heads=8 * H, max_pages=wide)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    args = dict(layer=0, q=q, page_table=table, cu_seqlens=cu, kv_len=lens)
    L.lin_state_attn_chunk(cache, out=out, workspace=work, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lin_state_attn_chunk(cache, out=out, workspace=work, **args)
    even = ([244] * B, [100] * B)
    long = ([3] + [0] * (B - 2) + [200], [30000] + [0] * (B - 2) + [20000])
    mixed = ([240] * (B - 1) + [1], [100] * (B - 1) + [30000])
    for new, cached in (even, long, even, mixed, long, ([0] * B, [5] * B), even):
        cu.copy_(i32(np.concatenate([[0], np.cumsum(new)])))
        lens.copy_(i32([a + b for a, b in zip(new, cached)]))
        out.zero_()
        graph.replay()
        again = torch.zeros_like(out)
        L.lin_state_attn_chunk(cache, out=again, workspace=torch.full_like(work, 255), **args)
        assert torch.equal(out, again)
        assert out[:sum(new)].any(-1).all() and not out[sum(new):].any()
