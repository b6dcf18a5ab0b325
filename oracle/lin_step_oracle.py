"""Plain fp64 CPU oracle of the decode-step operators (include/lin_step.h):
the paged cache append, decode attention and the norms around a block, token by
token and row by row, with numpy. Imported by tests only."""

import math

import numpy as np


def tree_ok(parent):
    return all(-1 <= p < j for j, p in enumerate(parent))


def path_to(parent, node):
    """The nodes from the root to `node`, root first."""
    out = []
    while node >= 0:
        out.append(node)
        node = parent[node]
    return out[::-1]


def locate(page_table_row, t, page_size, num_pages):
    """(page, row) of token t, or None where the page id is out of range."""
    page = int(page_table_row[t // page_size])
    return (page, t % page_size) if 0 <= page < num_pages else None


def kv_append(cache_k, cache_v, k, v, page_table, pos, n_tok=None, parent=None, accept_node=None):
    """cache_k / cache_v [pages][page_size][H][D], changed in place."""
    pages, ps = cache_k.shape[:2]
    B, n = k.shape[:2]
    for r in range(B):
        if pos[r] < 0:
            continue
        if parent is not None:
            if not tree_ok(parent[r]) or not -1 <= accept_node[r] < n:
                continue
            rows = path_to(parent[r], accept_node[r])
        else:
            count = n if n_tok is None else n_tok[r]
            if not 0 <= count <= n:
                continue
            rows = range(count)
        for rank, j in enumerate(rows):
            t = int(pos[r]) + rank
            if t >= page_table.shape[1] * ps:
                continue
            at = locate(page_table[r], t, ps, pages)
            if at is not None:
                cache_k[at], cache_v[at] = k[r, j], v[r, j]


def attn_decode(cache_k, cache_v, q, page_table, kv_len, scale, parent=None):
    """(out, reach, spread): out [B][n][Hq][D], NaN where a request is left out.
    reach = sum_t p_t |v_t| and spread = max_t scale sum_i |q_i k_ti| bound how
    far roundings inside the sums may move an output."""
    pages, ps, Hkv, D = cache_k.shape
    B, n, Hq, _ = q.shape
    G = Hq // Hkv
    out = np.full((B, n, Hq, D), np.nan)
    reach = np.zeros((B, n, Hq, D))
    spread = np.zeros((B, n, Hq, 1))
    for r in range(B):
        length = int(kv_len[r])
        if length < 0 or length > page_table.shape[1] * ps or (parent is not None and not tree_ok(parent[r])):
            continue
        where = [locate(page_table[r], t, ps, pages) for t in range(length)]
        base = length - n
        for j in range(n):
            mine = set(path_to(parent[r], j)) if parent is not None else set(range(j + 1))
            seen = [w for t, w in enumerate(where) if w is not None and (t < base or t - base in mine)]
            if not seen:
                out[r, j] = 0.0
                continue
            pg, row = np.array([w[0] for w in seen]), np.array([w[1] for w in seen])
            for h in range(Hq):
                k, v = cache_k[pg, row, h // G], cache_v[pg, row, h // G]
                s = scale * (k @ q[r, j, h])
                p = np.exp(s - s.max())
                p /= p.sum()
                out[r, j, h] = p @ v
                reach[r, j, h] = p @ np.abs(v)
                spread[r, j, h] = abs(scale) * (np.abs(k) @ np.abs(q[r, j, h])).max()
    return out, reach, spread


def block_norm(x, gate=None, act=None, w_post=None, residual=None, scale=1.0, scale_w=None, w_pre=None,
               eps=1e-6):
    """(t, h, y) as fp64 arrays; t is the scaled block output that h adds to
    the residual, y None without w_pre."""
    T, C = x.shape
    t = np.array(x, np.float64)
    if w_post is not None:
        g = len(w_post)
        for c in range(0, C, g):
            part = t[:, c:c + g]
            t[:, c:c + g] = part / np.sqrt((part ** 2).mean(1, keepdims=True) + eps) * w_post
    if gate is not None:
        sig = np.array([[1.0 / (1.0 + math.exp(-z)) if z > -700 else 0.0 for z in row] for row in gate])
        t = t * sig * (gate if act == "silu" else 1.0)
    t = t * scale * (1.0 if scale_w is None else scale_w)
    h = t if residual is None else residual + t
    y = None
    if w_pre is not None:
        y = h / np.sqrt((h ** 2).mean(1, keepdims=True) + eps) * w_pre
    return t, h, y
