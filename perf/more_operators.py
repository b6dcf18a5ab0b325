"""What a prompt of a hybrid model needs of its full-attention layers, whole or in
chunks, beside the linear-attention state path, as cases to be timed and compared:

* ``plan``: block tables, positions and slot maps of a batch's new tokens, from the
  requests' lengths and a list of free pages;
* ``rope``: rotary positions of the new queries and keys, with keys and values going
  into the paged key-value cache;
* ``chunk``: causal attention of each request's newest tokens (one, a few, a whole
  prompt) over its pages.

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
        # the next token's place of each of 256 running requests
        _plan("plan_step", B=256, lo=1, hi=1, c_lo=64, c_hi=16384, page=64),
        # 64 chunks of prompts, new and continued, small pages
        _plan("plan_chunks", B=64, lo=1, hi=2048, c_lo=0, c_hi=8192, page=16),
        # one decode step's queries and keys of 256 requests
        _rope("rope_step", T=256, Hq=16, Hkv=2, D=128, rot=128, style="half", page=64, far=16384),
        # a prompt batch of 8 x 4096 tokens
        _rope("rope_prompt", T=32768, Hq=16, Hkv=2, D=128, rot=128, style="half", page=64, far=4096),
        # part of the head in interleaved pairs, positions far out in a long context, 32 bits
        _rope("rope_part_f32", T=4097, Hq=12, Hkv=4, D=64, rot=24, style="pairs", page=37, far=1000003, dtype="f32",
              layout="hnd"),
        # one user's next message: 64 tokens after 1,000
        _chunk("chunk_one", B=1, lo=64, hi=64, c_lo=1000, c_hi=1000, Hq=16, Hkv=2, D=128, page=64),
        # a prompt batch of 8 x 4096 tokens, nothing cached
        _chunk("chunk_prompt", B=8, lo=4096, hi=4096, c_lo=0, c_hi=0, Hq=16, Hkv=2, D=128, page=64),
        # a chunk of 2,048 tokens at the end of a long document, heads-first pages
        _chunk("chunk_long", B=1, lo=2048, hi=2048, c_lo=129000, c_hi=129000, Hq=32, Hkv=8, D=128, page=16, layout="hnd"),
        # ragged continuations, some of a single token, wide heads, pages that end inside a tile
        _chunk("chunk_ragged", B=64, lo=1, hi=512, c_lo=200, c_hi=8000, Hq=16, Hkv=2, D=256, page=48),
        # the few tokens that a prefix cache did not hold, of 32 requests
        _chunk("chunk_tails", B=32, lo=1, hi=16, c_lo=1024, c_hi=16384, Hq=16, Hkv=2, D=128, page=64),
        # as many key-value heads as query heads, narrow heads
        _chunk("chunk_heads64", B=4, lo=1500, hi=2500, c_lo=0, c_hi=3000, Hq=8, Hkv=8, D=64, page=16),
        # 32 bits, ragged, odd pages
        _chunk("chunk_f32", B=8, lo=1, hi=300, c_lo=0, c_hi=2000, Hq=12, Hkv=4, D=64, page=37, dtype="f32"),
    ]


def _plan(name, B, lo, hi, c_lo, c_hi, page, tree=False):
    """B requests of c_lo .. c_hi cached tokens and lo .. hi new ones; tree: drafts."""
    c = {"op": "plan", "B": B, "lo": lo, "hi": hi, "c_lo": c_lo, "c_hi": c_hi, "page": page, "tree": tree}
    return {"name": name, **c} if name else c


def _rope(name, T, Hq, Hkv, D, rot, style, page, far, dtype="bf16", layout="nhd", scale=1.0):
    """T tokens at positions below `far`; the first `rot` channels of a head are turned."""
    c = {"op": "rope", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "style": style, "page": page, "far": far,
         "dtype": dtype, "layout": layout, "scale": scale}
    return {"name": name, **c} if name else c


def _chunk(name, B, lo, hi, c_lo, c_hi, Hq, Hkv, D, page, dtype="bf16", layout="nhd"):
    """lo .. hi new tokens after c_lo .. c_hi cached ones."""
    c = {"op": "chunk", "B": B, "lo": lo, "hi": hi, "c_lo": c_lo, "c_hi": c_hi, "Hq": Hq, "Hkv": Hkv, "D": D,
         "page": page, "dtype": dtype, "layout": layout}
    return {"name": name, **c} if name else c


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "rope", "plan"])
    page = rng.choice([16, 64, _log_int(rng, 8, 200)])
    if op == "plan":
        tree = rng.random() < 0.3
        hi = rng.randint(2, 32) if tree else _log_int(rng, 1, 4096)
        B = _log_int(rng, 1, min(1024, 131072 // hi))
        c_hi = _log_int(rng, 1, 16384)
        return _plan("", B, hi if tree else rng.choice([hi, 1, 0]), hi, rng.choice([0, c_hi]), c_hi, page, tree)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    layout = rng.choice(["nhd", "hnd"])
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 3, 4, 8])
    if op == "rope":
        T = _log_int(rng, 1, max(1, 75_000_000 // ((Hq + 2 * Hkv) * D * (1 if dtype == "bf16" else 2))))
        return _rope("", min(T, 32768), Hq, Hkv, D, rng.choice([D, D // 2, 2 * rng.randint(1, D // 2)]),
                     rng.choice(["half", "pairs"]), page, _log_int(rng, 100, 2_000_000), dtype, layout,
                     rng.choice([1.0, 1.25]))
    hi = _log_int(rng, 1, 4096)
    c_hi = _log_int(rng, 1, 131072)
    # no more products than a quarter of the largest listed case (32 bits: an eighth of that), a cache of 1 GB
    most = (1e12 if dtype == "bf16" else 1.2e11) / (4.0 * hi * (c_hi + hi) * Hq * D)
    B = _log_int(rng, 1, max(1, min(256, int(most), int(1.0e9 // ((c_hi + hi) * Hkv * D * 2 * ES[dtype])))))
    if most < 1:
        hi = max(1, int(hi * most))
    return _chunk("", B, rng.choice([hi, 1, (hi + 1) // 2]), hi, rng.choice([0, c_hi, c_hi // 2]), c_hi, Hq, Hkv, D,
                  page, dtype, layout)


# ---- inputs -------------------------------------------------------------------

def _sizes(case, seed):
    """Cached and new tokens of each request."""
    rng = random.Random(seed * 7919 + 17)
    return ([rng.randint(case["c_lo"], case["c_hi"]) for _ in range(case["B"])],
            [rng.randint(case["lo"], case["hi"]) for _ in range(case["B"])])


def _trees(case, seed):
    """Parents of each request's drafts, -1 for a child of the last committed token."""
    rng = random.Random(seed * 104729 + 5)
    return [[rng.randint(max(-1, j - 4), j - 1) for j in range(case["hi"])] for _ in range(case["B"])]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _pages(need, wide, gen):
    """Shuffled page ids: a table with need[r] entries in row r (-1 behind them), and how many pages there are."""
    total = sum(need)
    ids = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    first = torch.tensor([sum(need[:r]) for r in range(len(need))], device="cuda")
    col = torch.arange(wide, device="cuda")
    at = (first[:, None] + col).clamp_max(max(total - 1, 0))
    have = col < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(have, ids[at], -1) if total else torch.full((len(need), wide), -1, device="cuda")
    return table.to(torch.int32), total


def _cache(case, pages, gen):
    page, Hkv, D, dt = case["page"], case["Hkv"], case["D"], DT[case["dtype"]]
    shape = (1, pages, page, Hkv, D) if case["layout"] == "nhd" else (1, pages, Hkv, page, D)
    kv = [torch.randn(shape, generator=gen, device="cuda", dtype=dt) for _ in range(2)]
    return kv if case["layout"] == "nhd" else [x.transpose(2, 3) for x in kv]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    {"plan": _prepare_plan, "rope": _prepare_rope, "chunk": _prepare_chunk}[case["op"]](case, seed, gen, s)
    return s


def _prepare_plan(case, seed, gen, s):
    B, page = case["B"], case["page"]
    cached, new = _sizes(case, seed)
    have = [-(-c // page) for c in cached]
    wide = -(-(case["c_hi"] + case["hi"]) // page)
    s["page_table"], used = _pages(have, wide, gen)
    need = sum(-(-(c + n) // page) for c, n in zip(cached, new)) - used
    s["num_pages"] = used + need + 10
    s["free_pages"] = used + torch.randperm(need + 10, generator=gen, device="cuda").to(torch.int32)
    s["length"], s["n_new"] = _i32(cached), _i32(new)
    s["parent"] = _i32(_trees(case, seed)) if case["tree"] else None
    # a captured step keeps room for the most tokens, so the last rows stay empty
    rows = B * case["hi"]
    s["cu_seqlens"] = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["position"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
    s["slot"] = torch.zeros(rows, dtype=torch.int64, device="cuda")
    s["taken"] = torch.zeros(1, dtype=torch.int32, device="cuda")


def _prepare_rope(case, seed, gen, s):
    T, Hq, Hkv, D, rot, page = (case[k] for k in ("T", "Hq", "Hkv", "D", "rot", "page"))
    dt = DT[case["dtype"]]
    pages = -(-T // page) + 1
    s["k_cache"], s["v_cache"] = _cache(case, pages, gen)
    # one projection's rows hold the query, key and value heads side by side
    rows = torch.randn((T, Hq + 2 * Hkv, D), generator=gen, device="cuda").to(dt)
    s["q"], s["k"], s["v"] = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    s["position"] = torch.randint(case["far"], (T,), generator=gen, device="cuda", dtype=torch.int32)
    # whole pages in any order, rows of a page one after another
    ids = torch.randperm(pages, generator=gen, device="cuda")
    t = torch.arange(T, device="cuda")
    s["slot"] = ids[t // page] * page + t % page
    s["inv_freq"] = (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()
    s["q_out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
    if own:
        import linear_attention_state_chunked_gb300 as L
        s["cache"] = L.KVCache(1, pages, page, Hkv, D, dtype=dt, k=s["k_cache"], v=s["v_cache"])


def _prepare_chunk(case, seed, gen, s):
    B, Hq, Hkv, D, page = (case[k] for k in ("B", "Hq", "Hkv", "D", "page"))
    dt = DT[case["dtype"]]
    cached, new = _sizes(case, seed)
    wide = -(-(case["c_hi"] + case["hi"]) // page)
    s["page_table"], pages = _pages([-(-(c + n) // page) for c, n in zip(cached, new)], wide, gen)
    s["k_cache"], s["v_cache"] = _cache(case, pages, gen)
    T = B * case["hi"]  # a captured step has room for the most tokens: the rows behind the last one's stay as they are
    rows = torch.randn((T, Hq + 2 * Hkv, D), generator=gen, device="cuda").to(dt)
    rows[:, :Hq] *= 1.5  # scores spread over a few units, as a trained head's do
    s["q"] = rows[:, :Hq]
    s["cu_seqlens"] = _i32([sum(new[:r]) for r in range(B + 1)])
    s["kv_len"] = _i32([c + n for c, n in zip(cached, new)])
    if own:
        import linear_attention_state_chunked_gb300 as L
        s["cache"] = L.KVCache(1, pages, page, Hkv, D, dtype=dt, k=s["k_cache"], v=s["v_cache"])
        s["out"] = torch.zeros((T, Hq, D), dtype=dt, device="cuda")
        size = L.lin_state_attn_chunk_workspace(s["cache"], batch=B, tokens=T, num_q_heads=Hq, max_pages=wide)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")


# ---- one pass --------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"plan": _own_plan, "rope": _own_rope, "chunk": _own_chunk}[op](s)
    return {"plan": _plain_plan, "rope": _plain_rope, "chunk": _plain_chunk}[op](s)


def _own_plan(s):
    import linear_attention_state_chunked_gb300 as L
    tree = s["parent"] is not None
    L.lin_state_kv_plan(page_size=s["case"]["page"], num_pages=s["num_pages"], length=s["length"],
                        n_new=None if tree else s["n_new"], parent=s["parent"], page_table=s["page_table"],
                        free_pages=s["free_pages"], taken=s["taken"], cu_seqlens=s["cu_seqlens"], kv_len=s["kv_len"],
                        position=s["position"], slot=s["slot"])
    return [s[k] for k in ("page_table", "taken", "cu_seqlens", "kv_len", "position", "slot")]


def _own_rope(s):
    import linear_attention_state_chunked_gb300 as L
    L.lin_state_rope(s["cache"], layer=0, q=s["q"], k=s["k"], v=s["v"], position=s["position"], slot=s["slot"],
                     inv_freq=s["inv_freq"], scale=s["case"]["scale"], interleaved=s["case"]["style"] == "pairs",
                     q_out=s["q_out"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_chunk(s):
    import linear_attention_state_chunked_gb300 as L
    L.lin_state_attn_chunk(s["cache"], layer=0, q=s["q"], out=s["out"], page_table=s["page_table"],
                           cu_seqlens=s["cu_seqlens"], kv_len=s["kv_len"], workspace=s["workspace"])
    return s["out"]


def _plain_plan(s):
    page, table = s["case"]["page"], s["page_table"]
    length, n = s["length"].long(), s["n_new"].long()
    have = (length + page - 1) // page
    need = (length + n + page - 1) // page - have
    before = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device="cuda")
    rank = col - have[:, None]  # of a page among the request's new ones
    fresh = s["free_pages"][(before[:, None] + rank).clamp(0, s["free_pages"].numel() - 1)]
    table.copy_(torch.where((rank >= 0) & (rank < need[:, None]), fresh, table))
    cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
    t = torch.arange(s["position"].numel(), device="cuda")
    r = torch.searchsorted(cu[1:], t, right=True)
    live = r < n.numel()
    r = r.clamp_max(n.numel() - 1)
    j = t - cu[r]
    at = torch.where(live, length[r] + j, 0)
    slot = table[r, at // page] * page + at % page
    place = at
    if s["parent"] is not None:
        # a draft's depth: how many steps up its path ends
        up = torch.where(live, j, -1)
        place = length[r]
        for _ in range(s["parent"].shape[1] - 1):
            up = torch.where(up >= 0, s["parent"][r, up.clamp_min(0)].long(), -1)
            place = place + (up >= 0)
    position = torch.where(live, place, -1).to(torch.int32)
    return [table, need.sum().reshape(1).to(torch.int32), cu.to(torch.int32), (length + n).to(torch.int32), position,
            torch.where(live, slot, -1)]


def _turn(x, cos, sin, rot, style):
    if style == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)


def _plain_rope(s):
    c = s["case"]
    angle = s["position"].double()[:, None] * s["inv_freq"].double()  # far positions: 64 bits
    cos = (angle.cos() * c["scale"]).float()[:, None]
    sin = (angle.sin() * c["scale"]).float()[:, None]
    s["q_out"].copy_(_turn(s["q"].float(), cos, sin, c["rot"], c["style"]))
    k = _turn(s["k"].float(), cos, sin, c["rot"], c["style"]).to(DT[c["dtype"]])
    page, row = s["slot"] // c["page"], s["slot"] % c["page"]
    s["k_cache"][0][page, row] = k
    s["v_cache"][0][page, row] = s["v"]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_chunk(s):
    c = s["case"]
    B, n, Hq, Hkv, D, page = (c[k] for k in ("B", "hi", "Hq", "Hkv", "D", "page"))
    G, wide = Hq // Hkv, s["page_table"].shape[1]
    keys = wide * page
    out = torch.zeros((s["q"].shape[0], Hq, D), dtype=DT[c["dtype"]], device="cuda")
    new = (s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).long()
    # requests padded to the longest, as many (request, kv head) pairs at a time as give 2^30 scores
    pairs = max(1, (1 << 30) // (G * n * keys))
    heads, some = min(Hkv, pairs), max(1, pairs // Hkv)
    j, t = torch.arange(n, device="cuda"), torch.arange(keys, device="cuda")
    for r in range(0, B, some):
        ids = s["page_table"][r:r + some].clamp_min(0)
        b, m, length = ids.shape[0], new[r:r + some], s["kv_len"][r:r + some].long()
        mine = j < m[:, None]  # [b][n]
        row = (s["cu_seqlens"][r:r + b, None] + j)[mine]
        ok = t <= (length - m)[:, None, None] + j[:, None]  # [b][n][keys]
        for h in range(0, Hkv, heads):
            hs = min(heads, Hkv - h)
            k = s["k_cache"][0][:, :, h:h + hs][ids].reshape(b, keys, hs, D).permute(0, 2, 3, 1).float()
            v = s["v_cache"][0][:, :, h:h + hs][ids].reshape(b, keys, hs, D).permute(0, 2, 1, 3).float()
            q = torch.zeros((b, n, hs * G, D), device="cuda")
            q[mine] = s["q"][row, h * G:(h + hs) * G].float()
            q = q.reshape(b, n, hs, G, D).permute(0, 2, 3, 1, 4).reshape(b, hs, G * n, D)
            p = torch.matmul(q, k).reshape(b, hs, G, n, keys).mul_(D ** -0.5)
            p.masked_fill_(~ok[:, None, None], -math.inf)
            p.sub_(p.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(p.reshape(b, hs, G * n, keys), v).reshape(b, hs, G, n, D) / p.sum(-1, keepdim=True)
            out[row, h * G:(h + hs) * G] = o.permute(0, 3, 1, 2, 4).reshape(b, n, hs * G, D)[mine].to(out.dtype)
    return out


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    """Bytes read and written once, and products and sums; lengths at their mean."""
    if case["op"] == "rope":
        T, Hq, Hkv, D, es = case["T"], case["Hq"], case["Hkv"], case["D"], ES[case["dtype"]]
        return {"bytes": T * ((Hq + 2 * Hkv) * D * es * 2 + 12) + 2 * case["rot"],
                "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    B, lo, hi = case["B"], case["lo"], case["hi"]
    n, cached = (lo + hi) / 2, (case["c_lo"] + case["c_hi"]) / 2
    if case["op"] == "plan":
        fresh = B * n / case["page"]
        return {"bytes": B * (20 + (4 * hi if case["tree"] else 0)) + B * hi * 12 + fresh * 8, "flops": 0}
    Hq, Hkv, D, es = case["Hq"], case["Hkv"], case["D"], ES[case["dtype"]]
    square = (lo * lo + lo * hi + hi * hi) / 3  # mean of n^2
    return {"bytes": B * (2 * n * Hq * D * es + (cached + n) * (2 * Hkv * D * es + 4 / case["page"]) + 8),
            "flops": 4 * Hq * D * B * (n * cached + square / 2 + n / 2)}


# ---- the definition in 64 bits ---------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "rope": _exact_rope, "chunk": _exact_chunk}[case["op"]](case, seed, s)


def _exact_plan(case, seed, s):
    page = case["page"]
    table, free = s["page_table"].tolist(), s["free_pages"].tolist()
    rows = s["position"].numel()
    taken, cu, kv_len, position, slot = 0, [0], [], [], []
    trees = _trees(case, seed) if case["tree"] else None
    for r, (cached, n) in enumerate(zip(*_sizes(case, seed))):
        depth = []
        for j in range(n):
            at = cached + j
            if at % page == 0:
                table[r][at // page] = free[taken]
                taken += 1
            up = trees[r][j] if trees else j - 1
            depth.append(0 if up < 0 else depth[up] + 1)
            position.append(cached + depth[j])
            slot.append(table[r][at // page] * page + at % page)
        kv_len.append(cached + n)
        cu.append(cu[-1] + n)
    blank = [-1] * (rows - len(slot))
    return [_i32(table), _i32([taken]), _i32(cu), _i32(kv_len), _i32(position + blank),
            torch.tensor(slot + blank, dtype=torch.int64).cuda()]


def _exact_rope(case, seed, s):
    half = case["rot"] // 2
    i = torch.arange(half, device="cuda")
    first, second = (i, i + half) if case["style"] == "half" else (2 * i, 2 * i + 1)
    turn = torch.polar(torch.full((case["T"], half), case["scale"], dtype=torch.float64, device="cuda"),
                       s["position"].double()[:, None] * s["inv_freq"].double())[:, None]

    def rotated(x):
        x = x.double()
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    caches = [s["k_cache"].double(), s["v_cache"].double()]
    for cache, rows in zip(caches, (rotated(s["k"]), s["v"].double())):
        cache[0, s["slot"] // case["page"], s["slot"] % case["page"]] = rows
    return [rotated(s["q"])] + caches


def _exact_chunk(case, seed, s):
    Hq, Hkv, D, page = (case[k] for k in ("Hq", "Hkv", "D", "page"))
    cached, new = _sizes(case, seed)
    if 4.0 * Hq * D * sum(n * (c + n) for c, n in zip(cached, new)) > 8e12:
        return None
    out, at = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for r, (c, n) in enumerate(zip(cached, new)):
        t = torch.arange(c + n, device="cuda")
        where = s["page_table"][r].long()[t // page]
        for h in range(Hkv):
            k = s["k_cache"][0, where, t % page, h].double()
            v = s["v_cache"][0, where, t % page, h].double()
            for j in range(0, n, 512):
                m = min(512, n - j)
                q = s["q"][at + j:at + j + m, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].double()
                z = torch.einsum("jgd,td->jgt", q, k) / math.sqrt(D)
                later = t > torch.arange(c + j, c + j + m, device="cuda")[:, None]
                w = torch.softmax(z.masked_fill(later[:, None], -math.inf), -1)
                out[at + j:at + j + m, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)] = torch.einsum("jgt,td->jgd", w, v)
        at += n
    return out
