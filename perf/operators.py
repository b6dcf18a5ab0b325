"""What a decode step of a hybrid model needs beside the linear-attention state
path, as cases to be timed and compared:

* ``append``: new keys and values go into a paged key-value cache (one token, a
  whole prompt, or the accepted path of a draft tree);
* ``attn``: attention of one new token, or of a chain or tree of draft tokens,
  over that cache;
* ``norm``: the norm after a block with its gate, the scaled residual, and the
  norm before the next block, in one pass.

``run`` computes a case with elementary torch operations, or, where ``own`` is
true, with this repository's calls; ``exact`` is the definition in 64 bits.
"""

import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one user's chat turn: latency is all that counts
        _attn("attn_one", B=1, n=1, Hq=16, Hkv=2, D=128, lo=1000, hi=1000, page=64),
        # a full serving batch of 256 requests, 1k to 16k tokens each
        _attn("attn_batch", B=256, n=1, Hq=16, Hkv=2, D=128, lo=1024, hi=16384, page=64),
        # a single long document, heads-first pages
        _attn("attn_long", B=1, n=1, Hq=32, Hkv=8, D=128, lo=131071, hi=131071, page=16, layout="hnd"),
        # four drafts in a chain to verify; wide heads, pages that end inside a tile
        _attn("attn_verify4", B=64, n=4, Hq=16, Hkv=2, D=256, lo=200, hi=8000, page=48),
        # a tree of eight drafts over a 32-bit cache, lengths from the drafts alone upwards
        _attn("attn_tree8_f32", B=32, n=8, Hq=12, Hkv=4, D=64, lo=8, hi=4000, page=37, dtype="f32", tree=True),
        # the decode step's own tokens of 256 requests
        _append("append_step", B=256, n=1, Hkv=2, D=128, lo=64, hi=2048, page=64),
        # eight prompts of up to 4096 tokens written at once
        _append("append_prompt", B=8, n=4096, Hkv=8, D=128, lo=0, hi=500, page=16, layout="hnd"),
        # the accepted paths of 256 draft trees
        _append("append_tree8_f32", B=256, n=8, Hkv=4, D=64, lo=8, hi=2000, page=37, dtype="f32", tree=True),
        # a linear-attention layer's gated output norm (32 heads of 128), one token
        _norm("norm_gated_one", T=1, C=4096, group=128, x="f32", res="", gate="silu", pre=False),
        # the same over a prompt batch of 8 x 4096 tokens
        _norm("norm_gated_prompt", T=32768, C=4096, group=128, x="f32", res="", gate="silu", pre=False),
        # norm after a block, gate, layer scale and residual, norm before the next one: a batch's step
        _norm("norm_block_step", T=256, C=2048, group=2048, x="bf16", res="f32", gate="sigmoid", pre=True, chan=True),
        # an odd width without a norm after the block, a ragged batch of tokens
        _norm("norm_residual_odd", T=4097, C=1533, group=0, x="bf16", res="bf16", gate="", pre=True),
    ]


def _attn(name, B, n, Hq, Hkv, D, lo, hi, page, dtype="bf16", tree=False, layout="nhd"):
    c = {"op": "attn", "B": B, "n": n, "Hq": Hq, "Hkv": Hkv, "D": D, "lo": lo, "hi": hi, "page": page,
         "dtype": dtype, "tree": tree, "layout": layout}
    return {"name": name, **c} if name else c


def _append(name, B, n, Hkv, D, lo, hi, page, dtype="bf16", tree=False, layout="nhd"):
    c = {"op": "append", "B": B, "n": n, "Hkv": Hkv, "D": D, "lo": lo, "hi": hi, "page": page,
         "dtype": dtype, "tree": tree, "layout": layout}
    return {"name": name, **c} if name else c


def _norm(name, T, C, group, x, res, gate, pre, chan=False):
    """group 0: no norm after the block; res "": no residual; chan: a scale per channel."""
    c = {"op": "norm", "T": T, "C": C, "group": group, "x": x, "res": res, "gate": gate, "pre": pre, "chan": chan}
    return {"name": name, **c} if name else c


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([16, 64, _log_int(rng, 8, 200)])
    layout = rng.choice(["nhd", "hnd"])
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "attn":
        G = rng.choice([1, 3, 4, 8])
        n = rng.choice([1, 1, 4, rng.randint(2, 8)])
        tree = n > 1 and rng.random() < 0.5
        hi = _log_int(rng, 16, 131072)
        lo = rng.choice([hi, max(n, hi // 8), n])
        # no more padded cache bytes than a quarter of the largest listed case's
        most = int(1.0e9 // (hi * Hkv * D * 2 * ES[dtype]))
        B = _log_int(rng, 1, max(1, min(256, most)))
        return _attn("", B, n, Hkv * G, Hkv, D, lo, hi, page, dtype, tree, layout)
    if op == "append":
        tree = rng.random() < 0.3
        n = rng.randint(2, 8) if tree else _log_int(rng, 1, 4096)
        B = _log_int(rng, 1, max(1, min(256, 16384 // n)))
        most = int(5.0e8 // (B * Hkv * D * ES[dtype]))  # a pool of 1 GB at most, beside the prompts
        return _append("", B, n, Hkv, D, rng.choice([0, 8]), _log_int(rng, 64, max(65, min(4000, most))),
                       page, dtype, tree, layout)
    C = rng.choice([D * rng.randint(1, 32), _log_int(rng, 65, 8191)])
    T = _log_int(rng, 1, max(1, min(32768, 60_000_000 // C)))
    group = rng.choice([0, C, D if C % D == 0 else C])
    gate = rng.choice(["silu", "sigmoid", ""])
    res = rng.choice(["bf16", "f32", ""])
    pre = rng.random() < 0.6 or (group == 0 and gate == "" and res == "")
    return _norm("", T, C, group, dtype, res, gate, pre, res != "" and rng.random() < 0.5)


# ---- inputs -------------------------------------------------------------------

def _tree(rng, n):
    """Parents of one request's drafts, -1 for a child of the last committed token."""
    return [rng.randint(max(-1, j - 4), j - 1) for j in range(n)]


def _lengths(case, seed):
    rng = random.Random(seed * 7919 + 17)
    return [rng.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _trees(case, seed):
    rng = random.Random(seed * 104729 + 5)
    return [_tree(rng, case["n"]) for _ in range(case["B"])]


def _accepted(case, seed):
    """append: tokens written of each request, and a tree's last accepted node."""
    rng = random.Random(seed * 31337 + 3)
    n = case["n"]
    if case["tree"]:
        return None, [rng.randint(-1, n - 1) for _ in range(case["B"])]
    return [rng.randint((n + 1) // 2, n) for _ in range(case["B"])], None


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        _prepare_norm(case, gen, s)
        return s
    B, n, Hkv, D, page, dt = (case[k] for k in ("B", "n", "Hkv", "D", "page", "dtype"))
    lens = _lengths(case, seed)
    most = case["hi"] + (n if case["op"] == "append" else 0)
    wide = -(-most // page)  # page table entries of a request
    need = [-(-(x + (n if case["op"] == "append" else 0)) // page) for x in lens]
    # page 0 stays free; a pool that is appended to has room for every request at its longest
    pages = (B * wide if case["op"] == "append" else sum(need)) + 1
    ids = torch.randperm(pages - 1, generator=gen, device="cuda").to(torch.int32) + 1
    at = torch.full((B, wide), -1, dtype=torch.int32)
    for r, k in enumerate(need):
        at[r, :k] = torch.arange(sum(need[:r]), sum(need[:r]) + k, dtype=torch.int32)
    at = at.cuda()
    s["page_table"] = torch.where(at >= 0, ids[at.clamp_min(0).long()], at) if pages > 1 else at
    shape = (1, pages, page, Hkv, D) if case["layout"] == "nhd" else (1, pages, Hkv, page, D)
    caches = []
    for _ in range(2):
        c = torch.randn(shape, generator=gen, device="cuda", dtype=DT[dt])
        caches.append(c if case["layout"] == "nhd" else c.transpose(2, 3))
    s["k_cache"], s["v_cache"] = caches
    # one projection's rows hold the query, key and value heads side by side
    Hq = case.get("Hq", 0)
    rows = torch.randn((B, n, Hq + 2 * Hkv, D), generator=gen, device="cuda", dtype=DT[dt])
    s["q"], s["k"], s["v"] = rows[:, :, :Hq] * 1, rows[:, :, Hq:Hq + Hkv], rows[:, :, Hq + Hkv:]
    if Hq:
        rows[:, :, :Hq] *= 1.5  # scores spread over a few units, as a trained head's do
        s["q"] = rows[:, :, :Hq]
    s["len"] = torch.tensor(lens, dtype=torch.int32).cuda()
    s["parent"] = torch.tensor(_trees(case, seed), dtype=torch.int32).cuda() if case["tree"] else None
    s["n_tok"] = s["accept_node"] = None
    if case["op"] == "append":
        count, node = _accepted(case, seed)
        if count is not None:
            s["n_tok"] = torch.tensor(count, dtype=torch.int32).cuda() if n > 1 else None
        if node is not None:
            s["accept_node"] = torch.tensor(node, dtype=torch.int32).cuda()
    if own:
        import linear_attention_state_chunked_gb300 as L
        s["cache"] = L.KVCache(1, pages, page, Hkv, D, dtype=DT[dt], k=s["k_cache"], v=s["v_cache"])
        if case["op"] == "attn":
            s["out"] = torch.empty((B, n, Hq, D), dtype=DT[dt], device="cuda")
            size = L.lin_state_attn_workspace(s["cache"], batch=B, n_q=n, num_q_heads=Hq, max_pages=wide)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


def _prepare_norm(case, gen, s):
    T, C, group = case["T"], case["C"], case["group"]
    xt = DT[case["x"]]

    def make(shape, dtype, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std + mean).to(dtype)

    s["x"] = make((T, C), xt, 0.7)
    s["gate"] = make((T, C), torch.bfloat16) if case["gate"] else None
    s["w_post"] = make((group,), torch.bfloat16, 0.1, 1.0) if group else None
    s["residual"] = make((T, C), DT[case["res"]], 3.0) if case["res"] else None
    s["scale"] = 0.25 if case["res"] else 1.0
    s["scale_w"] = make((C,), torch.bfloat16, 0.2, 1.0) if case["chan"] else None
    s["w_pre"] = make((C,), torch.bfloat16, 0.1, 1.0) if case["pre"] else None
    s["h_dtype"] = DT[case["res"]] if case["res"] else torch.bfloat16
    if own:
        s["h_out"] = torch.empty((T, C), dtype=s["h_dtype"], device="cuda")
        s["y"] = torch.empty((T, C), dtype=torch.bfloat16, device="cuda") if case["pre"] else None


# ---- one pass --------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"attn": _own_attn, "append": _own_append, "norm": _own_norm}[op](s)
    return {"attn": _plain_attn, "append": _plain_append, "norm": _plain_norm}[op](s)


def _own_attn(s):
    import linear_attention_state_chunked_gb300 as L
    L.lin_state_attn_decode(s["cache"], layer=0, q=s["q"], out=s["out"], page_table=s["page_table"],
                            kv_len=s["len"], parent=s["parent"], workspace=s["workspace"])
    return s["out"]


def _own_append(s):
    import linear_attention_state_chunked_gb300 as L
    L.lin_state_kv_append(s["cache"], layer=0, k=s["k"], v=s["v"], page_table=s["page_table"], pos=s["len"],
                          n_tok=s["n_tok"], parent=s["parent"], accept_node=s["accept_node"])
    return s["k_cache"], s["v_cache"]


def _own_norm(s):
    import linear_attention_state_chunked_gb300 as L
    L.lin_state_block_norm(x=s["x"], gate=s["gate"], gate_act=s["case"]["gate"] or None, w_post=s["w_post"],
                           residual=s["residual"], scale=s["scale"], scale_w=s["scale_w"], w_pre=s["w_pre"],
                           h_out=s["h_out"], y=s["y"])
    return [s["h_out"]] + ([s["y"]] if s["y"] is not None else [])


def _ancestors(parent):
    """[B][n][n] truth values: draft d is draft j or one of its ancestors."""
    B, n = parent.shape
    eye = torch.eye(n + 1, dtype=torch.bool, device=parent.device)
    see = torch.zeros((B, n + 1, n + 1), dtype=torch.bool, device=parent.device)
    for j in range(n):  # row n stands for "no parent"
        up = torch.where(parent[:, j] < 0, n, parent[:, j]).long()
        see[:, j] = see[torch.arange(B, device=parent.device), up] | eye[j]
    return see[:, :n, :n]


def _plain_attn(s):
    c = s["case"]
    B, n, Hq, Hkv, D, page = (c[k] for k in ("B", "n", "Hq", "Hkv", "D", "page"))
    G, wide = Hq // Hkv, s["page_table"].shape[1]
    keys = wide * page
    some = max(1, min(B, (1 << 29) // (keys * Hkv * max(D, G * n))))  # requests at a time
    if c["tree"]:
        see = _ancestors(s["parent"])
    else:
        see = torch.ones((n, n), dtype=torch.bool, device="cuda").tril().expand(B, n, n)
    out = []
    for r in range(0, B, some):
        ids = s["page_table"][r:r + some].clamp_min(0)
        b = ids.shape[0]
        k = s["k_cache"][0][ids].reshape(b, keys, Hkv, D).float()
        v = s["v_cache"][0][ids].reshape(b, keys, Hkv, D).float()
        q = s["q"][r:r + some].float().reshape(b, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(b, Hkv, n * G, D)
        score = torch.matmul(q, k.permute(0, 2, 3, 1)).reshape(b, Hkv, n, G, keys) * D ** -0.5
        draft = torch.arange(keys, device="cuda") - (s["len"][r:r + some, None] - n)  # [b][keys]
        seen = see[r:r + some].gather(2, draft.clamp(0, n - 1).long()[:, None].expand(b, n, keys))
        ok = (draft < 0)[:, None] | ((draft < n)[:, None] & seen)
        score = score.masked_fill(~ok[:, None, :, None], -math.inf)
        top = score.amax(-1, keepdim=True).clamp_min(-1e30)
        p = torch.exp(score - top)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.reshape(b, Hkv, n * G, keys), v.permute(0, 2, 1, 3)).reshape(b, Hkv, n, G, D)
        o = torch.where(total > 0, o / total, torch.zeros_like(o))
        out.append(o.permute(0, 2, 1, 3, 4).reshape(b, n, Hq, D).to(DT[c["dtype"]]))
    return torch.cat(out)


def _plain_append(s):
    c = s["case"]
    B, n, page = c["B"], c["n"], c["page"]
    if c["tree"]:
        # rank of a node on the accepted path, counted from the root
        see = _ancestors(s["parent"])
        node = s["accept_node"].long()
        on = see[torch.arange(B, device="cuda"), node.clamp_min(0)] & (node >= 0)[:, None]
        rank = on.long().cumsum(1) - 1
    else:
        rank = torch.arange(n, device="cuda").expand(B, n)
        on = rank < s["n_tok"][:, None] if s["n_tok"] is not None else torch.ones_like(rank, dtype=torch.bool)
    at = s["len"][:, None].long() + rank
    r, j = torch.nonzero(on, as_tuple=True)
    at = at[r, j]
    page_id = s["page_table"][r, at // page].long()
    s["k_cache"][0][page_id, at % page] = s["k"][r, j]
    s["v_cache"][0][page_id, at % page] = s["v"][r, j]
    return s["k_cache"], s["v_cache"]


def _plain_norm(s):
    c = s["case"]
    T, C, group = c["T"], c["C"], c["group"]
    t = s["x"].float()
    if group:
        t = t.reshape(T, C // group, group)
        t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * s["w_post"].float()
        t = t.reshape(T, C)
    if c["gate"]:
        z = s["gate"].float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        t = t * (z * sig if c["gate"] == "silu" else sig)
    if s["scale_w"] is not None:
        t = t * s["scale_w"].float()
    h = s["residual"].float() + s["scale"] * t if s["residual"] is not None else s["scale"] * t
    out = [h.to(s["h_dtype"])]
    if c["pre"]:
        out.append((h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["w_pre"].float()).to(torch.bfloat16))
    return out


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    """Bytes read and written once, and products and sums; lengths at their mean."""
    if case["op"] == "norm":
        T, C = case["T"], case["C"]
        n = T * C
        b = n * ES[case["x"]] + (2 * n if case["gate"] else 0)
        b += 2 * n * ES[case["res"]] if case["res"] else 2 * n
        b += (2 * n if case["pre"] else 0) + 2 * case["group"] + (2 * C if case["pre"] else 0) + (2 * C if case["chan"] else 0)
        return {"bytes": b, "flops": 12 * n}
    B, n, Hkv, D, es = case["B"], case["n"], case["Hkv"], case["D"], ES[case["dtype"]]
    mean = (case["lo"] + case["hi"]) / 2
    if case["op"] == "append":
        # a path holds about half a tree's nodes at most, a chain three quarters of its tokens
        tokens = B * (1 if n == 1 else n * (0.25 if case["tree"] else 0.75))
        return {"bytes": tokens * Hkv * D * es * 4 + 8 * B, "flops": 0}
    Hq = case["Hq"]
    keys = B * mean
    return {"bytes": keys * Hkv * D * 2 * es + 2 * B * n * Hq * D * es + 4 * keys / case["page"] + 4 * B,
            "flops": 4 * keys * n * Hq * D}


# ---- the definition in 64 bits ---------------------------------------------------------

def exact(case, seed):
    if case["op"] == "append":
        return None  # a copy: nothing is computed
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    n, Hq, Hkv, D, page = (case[k] for k in ("n", "Hq", "Hkv", "D", "page"))
    trees = _trees(case, seed) if case["tree"] else None
    out = torch.zeros((case["B"], n, Hq, D), dtype=torch.float64, device="cuda")
    for r, length in enumerate(_lengths(case, seed)):
        t = torch.arange(length, device="cuda")
        where = s["page_table"][r].long()[t // page]
        k = s["k_cache"][0, where, t % page].double()  # [length][Hkv][D]
        v = s["v_cache"][0, where, t % page].double()
        hidden = torch.zeros((n, length), dtype=torch.bool)
        for j in range(n):
            path = {j}
            up = j
            while trees is not None and up >= 0:
                path.add(up)
                up = trees[r][up]
            if trees is None:
                path = set(range(j + 1))
            for d in range(n):
                if d not in path and 0 <= length - n + d < length:
                    hidden[j, length - n + d] = True
        hidden = hidden.cuda()
        for h in range(Hkv):
            q = s["q"][r, :, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].double()  # [n][G][D]
            z = (q.reshape(-1, D) @ k[:, h].T / math.sqrt(D)).reshape(n, -1, length)
            z = z.masked_fill(hidden[:, None], -math.inf)
            w = torch.softmax(z, -1)
            out[r, :, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)] = (w.reshape(-1, length) @ v[:, h]).reshape(n, -1, D)
    return out


def _exact_norm(case, s):
    C, group = case["C"], case["group"]
    rows_h, rows_y = [], []
    for a in range(0, case["T"], 4096):
        t = s["x"][a:a + 4096].double()
        if group:
            t = torch.cat([p / (p.pow(2).sum(1, keepdim=True) / group + 1e-6).sqrt() * s["w_post"].double()
                           for p in t.split(group, 1)], 1)
        if case["gate"]:
            z = s["gate"][a:a + 4096].double()
            t = t * torch.sigmoid(z) * (z if case["gate"] == "silu" else 1.0)
        t = t * s["scale"]
        if case["chan"]:
            t = t * s["scale_w"].double()
        if s["residual"] is not None:
            t = t + s["residual"][a:a + 4096].double()
        rows_h.append(t)
        if case["pre"]:
            rows_y.append(t / (t.pow(2).sum(1, keepdim=True) / C + 1e-6).sqrt() * s["w_pre"].double())
    return [torch.cat(rows_h)] + ([torch.cat(rows_y)] if case["pre"] else [])
