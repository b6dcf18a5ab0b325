"""A small hybrid model's decode loop on the library's calls: three
linear-attention (GDN) layers to one full-attention layer, with
steps of one token and a verify of a few drafts.

    python examples/hybrid_decode.py [--steps 8] [--batch 4]

Every layer: norm, projections (torch matmuls), core, gated output norm, output
projection, residual and the next layer's norm. The cores and the norms are the
library's calls: lin_state_prefill / lin_state_decode over the state pool in
linear layers, lin_state_kv_append / lin_state_attn_decode over the paged cache
in the full layer, lin_state_block_norm everywhere. Weights are random.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_state_chunked_gb300 as L  # noqa: E402

BF = torch.bfloat16
HEADS, DIM = 4, 128               # linear heads and head size
Q_HEADS, KV_HEADS = 8, 2          # full attention
HIDDEN, VOCAB, PAGE = 512, 1000, 16
LAYERS = ("linear", "linear", "linear", "full")


class HybridModel:
    def __init__(self, batch, max_tokens, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)

        def w(*shape, std=None):
            std = shape[-1] ** -0.5 if std is None else std
            return (torch.randn(shape, generator=gen) * std).to(device, BF)

        self.batch, self.device = batch, device
        C = 3 * HEADS * DIM
        self.embed = w(VOCAB, HIDDEN, std=1.0)
        self.head = w(VOCAB, HIDDEN)
        self.norm_in = w(HIDDEN, std=0.1) + 1
        self.layers = []
        for i, kind in enumerate(LAYERS):
            width = (HEADS if kind == "linear" else Q_HEADS) * DIM
            p = {"kind": kind, "gate": w(width, HIDDEN), "out": w(HIDDEN, width),
                 "core_norm": w(DIM, std=0.1) + 1, "next_norm": w(HIDDEN, std=0.1) + 1}
            if kind == "linear":
                p.update(qkv=w(C, HIDDEN), conv=w(C, 4, std=0.5), decay=w(HEADS, HIDDEN), beta=w(HEADS, HIDDEN))
            else:
                p.update(qkv=w((Q_HEADS + 2 * KV_HEADS) * DIM, HIDDEN))
            self.layers.append(p)
        n_linear = LAYERS.count("linear")
        self.pool = L.StatePool(n_linear, batch + 1, HEADS, DIM, state_dtype=torch.float32, device=device)
        self.slots = torch.arange(1, batch + 1, dtype=torch.int32, device=device)
        wide = -(-max_tokens // PAGE)
        self.cache = L.KVCache(LAYERS.count("full"), batch * wide + 1, PAGE, KV_HEADS, DIM, device=device)
        # any assignment of pages does; page 0 stays free
        self.table = (torch.randperm(batch * wide, generator=gen).to(torch.int32) + 1).view(batch, wide).to(device)
        self.pos = torch.zeros(batch, dtype=torch.int32, device=device)  # committed tokens
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.workspace = None

    def _attn_workspace(self, n):
        need = L.lin_state_attn_workspace(self.cache, batch=self.batch, n_q=n, num_q_heads=Q_HEADS,
                                          max_pages=self.table.shape[1])
        if self.workspace is None or self.workspace.numel() < need:
            self.workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        return self.workspace

    def _gates(self, p, y):
        g = -torch.nn.functional.softplus(y @ p["decay"].T).float()  # log decay, one per head
        return g.contiguous(), torch.sigmoid(y @ p["beta"].T).float().contiguous()

    def _linear(self, p, layer, y, n, verify):
        """Core of a linear layer over [batch][n] tokens: a step in place, or n
        drafts whose states are not kept (commit replays the accepted ones)."""
        B = self.batch
        x = (y @ p["qkv"].T).view(B, n, -1)
        g, beta = self._gates(p, y)
        g, beta = g.view(B, n, HEADS), beta.view(B, n, HEADS)
        out = torch.empty((B, n, HEADS, DIM), dtype=BF, device=self.device)
        L.lin_state_decode(self.pool, layer=layer, x=x, conv_w=p["conv"], g=g, beta=beta, out=out,
                           slot=self.slots, pos=self.pos, gate_mode=L.LIN_GATE_PER_HEAD, status=self.status)
        if verify:
            p["replay"] = (x, g, beta)
        return out

    def _full(self, p, layer, y, n, parent=None):
        B = self.batch
        qkv = (y @ p["qkv"].T).view(B, n, Q_HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], 2)
        L.lin_state_kv_append(self.cache, layer=layer, k=k, v=v, page_table=self.table, pos=self.pos,
                              status=self.status)
        out = torch.empty((B, n, Q_HEADS, DIM), dtype=BF, device=self.device)
        L.lin_state_attn_decode(self.cache, layer=layer, q=q, out=out, page_table=self.table,
                                kv_len=self.pos + n, parent=parent, status=self.status,
                                workspace=self._attn_workspace(n))
        return out

    def _tail(self, p, core, y, h):
        """Gated output norm, projection, residual and the next layer's norm."""
        rows = core.reshape(h.shape[0], -1)
        act = "silu" if p["kind"] == "linear" else "sigmoid"
        t = torch.empty(rows.shape, dtype=BF, device=self.device)
        L.lin_state_block_norm(x=rows, gate=y @ p["gate"].T, gate_act=act, w_post=p["core_norm"], h_out=t)
        nxt = torch.empty_like(y)
        L.lin_state_block_norm(x=t @ p["out"].T, residual=h, w_pre=p["next_norm"], h_out=h, y=nxt)
        return nxt

    def forward(self, tokens, verify=False):
        """tokens [batch][n] -> logits [batch][n][vocab]. n == 1 is a step (the
        linear states move on); n > 1 drafts are verified and nothing but the
        cache's rows past pos changes."""
        B, n = tokens.shape
        h = self.embed[tokens.reshape(-1)].float()  # the residual stream stays in fp32
        y = torch.empty(h.shape, dtype=BF, device=self.device)
        L.lin_state_block_norm(x=h, w_pre=self.norm_in, y=y)
        at = {"linear": 0, "full": 0}
        for p in self.layers:
            core = (self._linear(p, at["linear"], y, n, verify) if p["kind"] == "linear"
                    else self._full(p, at["full"], y, n))
            at[p["kind"]] += 1
            y = self._tail(p, core, y, h)
        return (y @ self.head.T).view(B, n, VOCAB).float()

    def step(self, tokens):
        logits = self.forward(tokens[:, None])[:, 0]
        self.pos += 1
        return logits

    def verify(self, drafts):
        """Two drafts or more: one would be a step, which moves the linear states."""
        if drafts.shape[1] < 2:
            raise ValueError(f"a verify takes 2 drafts or more, got {drafts.shape[1]}: one token is a step")
        return self.forward(drafts, verify=True)

    def commit(self, accept_len):
        """Keep the first accept_len[r] drafts of the last verify: the linear
        layers replay them; the cache holds them already."""
        at = 0
        for p in self.layers:
            if p["kind"] == "linear":
                x, g, beta = p["replay"]
                L.lin_state_replay_commit(self.pool, layer=at, x=x, conv_w=p["conv"], g=g, beta=beta,
                                          slot=self.slots, pos=self.pos, accept_len=accept_len,
                                          gate_mode=L.LIN_GATE_PER_HEAD, status=self.status)
                at += 1
        self.pos += accept_len


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--batch", type=int, default=4)
    args = ap.parse_args()
    if args.steps < 1:
        ap.error("--steps: 1 or more, for drafts to verify")
    model = HybridModel(args.batch, 4 * args.steps + 8)
    token = torch.arange(args.batch, device="cuda") % VOCAB
    said = [token]
    for _ in range(args.steps):
        token = model.step(token).argmax(-1)
        said.append(token)
    # drafts: what greedy decoding would say if it repeated its last tokens
    drafts = torch.stack([token] + said[-4:-1], 1)
    best = model.verify(drafts).argmax(-1)
    good = (best[:, :-1] == drafts[:, 1:]).long().cumprod(1).sum(1)
    accept = (good + 1).to(torch.int32)  # the first draft is the token itself
    model.commit(accept)
    assert L.lin_state_read_status(model.status) == 0
    print("tokens of request 0:", [int(t[0]) for t in said])
    print("accepted drafts:", accept.tolist(), "positions:", model.pos.tolist())


if __name__ == "__main__":
    main()
