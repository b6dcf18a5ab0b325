"""A small hybrid model reads ragged prompts in chunks and goes on by single tokens, on
the library's calls: the model of hybrid_decode.py with rotary positions in its
full-attention layer and pages given out on the device.

    python examples/hybrid_prompt.py [--batch 3] [--chunk 128] [--steps 8]

A chunk of a batch of prompts, packed: lin_state_kv_plan gives each request its pages,
and every token its position and its row of the cache, once for all layers; linear
layers run lin_state_prefill, the full layer lin_state_rope (which appends) and
lin_state_attn_chunk. A step of one token is the same with lin_state_decode and
lin_state_attn_decode. Weights and prompts are random.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_state_chunked_gb300 as L  # noqa: E402
from examples.hybrid_decode import BF, DIM, HEADS, KV_HEADS, PAGE, Q_HEADS, VOCAB, HybridModel  # noqa: E402


class HybridPromptModel(HybridModel):
    def __init__(self, batch, max_tokens, seed=0, device="cuda"):
        super().__init__(batch, max_tokens, seed, device)
        self.inv_freq, self.rope_scale = L.rope_frequencies(DIM, 10000.0, device=device)
        # pages in any order, none of them given to a request yet
        self.free = self.table.reshape(-1).clone()
        self.used = 0
        self.table.fill_(-1)

    def _plan(self, n_new, rows):
        """Pages for n_new[r] more tokens of every request, and the rows' places."""
        i32 = dict(dtype=torch.int32, device=self.device)
        plan = dict(cu_seqlens=torch.empty(self.batch + 1, **i32), kv_len=torch.empty(self.batch, **i32),
                    position=torch.empty(rows, **i32), slot=torch.empty(rows, dtype=torch.int64, device=self.device))
        taken = torch.zeros(1, **i32)
        L.lin_state_kv_plan(page_size=PAGE, num_pages=self.cache.num_pages, length=self.pos, n_new=n_new,
                            page_table=self.table, free_pages=self.free[self.used:], taken=taken, status=self.status, **plan)
        self.used += int(taken)
        return plan

    def _rope(self, p, layer, y, plan):
        qkv = (y @ p["qkv"].T).view(-1, Q_HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], 1)
        L.lin_state_rope(self.cache, layer=layer, q=q, k=k, v=v, q_out=q, position=plan["position"], slot=plan["slot"],
                         inv_freq=self.inv_freq, scale=self.rope_scale, status=self.status)
        return q

    def _run(self, tokens, core):
        """Logits of the packed tokens; core(p, layer, y) is a layer's core."""
        h = self.embed[tokens].float()
        y = torch.empty(h.shape, dtype=BF, device=self.device)
        L.lin_state_block_norm(x=h, w_pre=self.norm_in, y=y)
        at = {"linear": 0, "full": 0}
        for p in self.layers:
            out = core(p, at[p["kind"]], y)
            at[p["kind"]] += 1
            y = self._tail(p, out, y, h)
        return (y @ self.head.T).float()

    def prompt(self, tokens, n_new):
        """Reads n_new[r] tokens of each request, packed in `tokens`. A request's chunks
        but its last are multiples of 64 tokens, as the linear layers' states take them.
        Returns the logits of every token."""
        T = tokens.shape[0]
        new = torch.tensor(n_new, dtype=torch.int32, device=self.device)
        if sum(n_new) != T:
            raise ValueError(f"{sum(n_new)} tokens by n_new, {T} given")
        plan = self._plan(new, T)
        warm = (self.pos > 0).to(torch.int64)
        prefix = torch.where(new > 0, self.pos, 0)  # a request that gets nothing may have any length

        def core(p, layer, y):
            if p["kind"] == "linear":
                g, beta = self._gates(p, y)
                out = torch.empty((T, HEADS, DIM), dtype=BF, device=self.device)
                L.lin_state_prefill(self.pool, layer=layer, x=y @ p["qkv"].T, conv_w=p["conv"], g=g, beta=beta, out=out,
                                    cu_seqlens=plan["cu_seqlens"], prefix_len=prefix, slot=self.slots,
                                    has_initial_state=warm, gate_mode=L.LIN_GATE_PER_HEAD, status=self.status)
                return out
            q = self._rope(p, layer, y, plan)
            out = torch.empty((T, Q_HEADS, DIM), dtype=BF, device=self.device)
            L.lin_state_attn_chunk(self.cache, layer=layer, q=q, out=out, page_table=self.table,
                                   cu_seqlens=plan["cu_seqlens"], kv_len=plan["kv_len"], status=self.status)
            return out

        logits = self._run(tokens, core)
        self.pos += new
        return logits

    def step(self, tokens):
        """One more token of every request."""
        B = self.batch
        plan = self._plan(torch.ones(B, dtype=torch.int32, device=self.device), B)

        def core(p, layer, y):
            if p["kind"] == "linear":
                return self._linear(p, layer, y, 1, False)
            q = self._rope(p, layer, y, plan).unflatten(0, (B, 1))
            out = torch.empty((B, 1, Q_HEADS, DIM), dtype=BF, device=self.device)
            L.lin_state_attn_decode(self.cache, layer=layer, q=q, out=out, page_table=self.table, kv_len=plan["kv_len"],
                                    status=self.status, workspace=self._attn_workspace(1))
            return out

        logits = self._run(tokens, core)
        self.pos += 1
        return logits


def chunks(lengths, size):
    """Tokens of each request in successive chunks of up to `size`."""
    done = [0] * len(lengths)
    while any(d < n for d, n in zip(done, lengths)):
        new = [min(size, n - d) for d, n in zip(done, lengths)]
        yield done, new
        done = [d + x for d, x in zip(done, new)]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=3)
    ap.add_argument("--chunk", type=int, default=128)
    ap.add_argument("--steps", type=int, default=8)
    args = ap.parse_args()
    if args.chunk < 64 or args.chunk % 64:
        ap.error("--chunk: a multiple of 64")
    lengths = [100 + 90 * r for r in range(args.batch)]
    gen = torch.Generator().manual_seed(0)
    prompts = [torch.randint(VOCAB, (n,), generator=gen).cuda() for n in lengths]
    model = HybridPromptModel(args.batch, max(lengths) + args.steps + 1)
    last = torch.zeros(args.batch, dtype=torch.long, device="cuda")
    for done, new in chunks(lengths, args.chunk):
        packed = torch.cat([p[d:d + n] for p, d, n in zip(prompts, done, new)])
        logits = model.prompt(packed, new)
        for r, part in enumerate(logits.split(new)):
            if len(part):
                last[r] = part[-1].argmax()
    said = [last]
    for _ in range(args.steps):
        said.append(model.step(said[-1]).argmax(-1))
    assert L.lin_state_read_status(model.status) == 0
    print("prompts of", lengths, "tokens; said:", torch.stack(said, 1).tolist())
    print("pages in use:", model.used, "of", model.free.numel())


if __name__ == "__main__":
    main()
