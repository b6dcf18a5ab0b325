"""Plain fp64 CPU oracle of the prompt operators (include/lin_prompt.h): block tables
and slot maps, rotary positions and attention of packed new tokens over a paged cache,
with numpy. Imported by tests only."""

import numpy as np

from oracle.lin_step_oracle import locate, path_to, tree_ok

BAD_SEQLEN, BAD_TREE, BAD_PAGE, NO_PAGES = 8, 256, 512, 1024


def kv_plan(length, n_new, page_table, page_size, num_pages, tokens, free_pages=None, parent=None):
    """(table, taken, cu, kv_len, position, slot, status) token by token."""
    table = np.array(page_table)
    B, wide = table.shape
    position, slot = np.full(tokens, -1), np.full(tokens, -1, np.int64)
    cu, kv_len, status, used, taken = [0], [], 0, 0, 0
    for r in range(B):
        have, n = int(length[r]), int(n_new[r])
        if have < 0:
            kv_len.append(-1)
            cu.append(cu[-1])
            continue
        bad = 0
        if n < 0:
            n, bad = 0, BAD_SEQLEN
        if have + n > wide * page_size:
            bad |= BAD_SEQLEN
        if parent is not None and not tree_ok(parent[r]):
            bad |= BAD_TREE
        start = cu[-1]
        cu.append(start + n)
        need = 0
        if not bad and free_pages is not None:
            need = -(-(have + n) // page_size) + (-have // page_size)
        if not bad and start + n > tokens:
            bad = BAD_SEQLEN
        if not bad and need and used + need > len(free_pages):
            bad = NO_PAGES
        status |= bad
        if bad:
            kv_len.append(-1)
            used += need
            continue
        kv_len.append(have + n)
        first = -(-have // page_size)
        for i in range(need):
            table[r, first + i] = free_pages[used + i]
        used += need
        if need:
            taken = used
        for j in range(n):
            t = have + j
            position[start + j] = t if parent is None else have + len(path_to(parent[r], j)) - 1
            at = locate(table[r], t, page_size, num_pages)
            if at is None:
                status |= BAD_PAGE
            else:
                slot[start + j] = at[0] * page_size + at[1]
    return table, taken, np.array(cu), np.array(kv_len), position, slot, status


def rope(x, position, inv_freq, scale=1.0, interleaved=False):
    """(turned, reach): x [T][heads][D]; reach bounds |x| + |y| of each channel's pair."""
    y, reach = np.array(x, np.float64), np.abs(np.array(x, np.float64))
    half = len(inv_freq)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    # products of up to 55 bits: reduced exactly, as fractions, where a double rounds
    from fractions import Fraction
    two_pi = 2 * Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    table = {}
    angle = np.zeros((len(position), half))
    for t, pos in enumerate(position):
        for k, f in enumerate(inv_freq):
            key = (int(pos), float(f))
            if key not in table:
                z = Fraction(int(pos)) * Fraction(float(f))
                table[key] = float(z - two_pi * (z // two_pi))
            angle[t, k] = table[key]
    cos, sin = np.cos(angle)[:, None], np.sin(angle)[:, None]
    p, q = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = scale * (p * cos - q * sin), scale * (q * cos + p * sin)
    reach[..., a] = reach[..., b] = abs(scale) * (np.abs(p) + np.abs(q))
    return y, reach


def attn_chunk(cache_k, cache_v, q, page_table, cu, kv_len, scale):
    """(out, reach, spread): out [T][Hq][D], NaN in rows that are left as they are;
    reach = sum_t p_t |v_t| and spread = max_t scale sum_i |q_i k_ti| bound how far
    roundings inside the sums may move an output."""
    pages, ps, Hkv, D = cache_k.shape
    T, Hq, _ = q.shape
    G = Hq // Hkv
    out, reach, spread = np.full((T, Hq, D), np.nan), np.zeros((T, Hq, D)), np.zeros((T, Hq, 1))
    for r in range(len(kv_len)):
        length, a, b = int(kv_len[r]), int(cu[r]), int(cu[r + 1])
        if length < 0 or length > page_table.shape[1] * ps or a < 0 or b < a or b > T:
            continue
        n = b - a
        where = [locate(page_table[r], t, ps, pages) for t in range(length)]
        live = np.array([w is not None for w in where], bool)
        pg = np.array([w[0] if w else 0 for w in where], int)
        row = np.array([w[1] if w else 0 for w in where], int)
        pos = length - n + np.arange(n)
        see = live[None, :] & (np.arange(length)[None, :] <= pos[:, None])  # [n][length]
        any_ = see.any(1)
        out[a:b] = 0.0
        if not any_.any():
            continue
        for h in range(Hq):
            k, v = cache_k[pg, row, h // G], cache_v[pg, row, h // G]
            used = see.any(0)
            k, v = np.where(used[:, None], k, 0.0), np.where(used[:, None], v, 0.0)
            x = q[a:b, h]
            s = np.where(see, scale * (x @ k.T), -np.inf)
            p = np.zeros_like(s)
            top = s[any_].max(1, keepdims=True)
            p[any_] = np.exp(s[any_] - top)
            p[any_] /= p[any_].sum(1, keepdims=True)
            out[a:b, h], reach[a:b, h] = p @ v, p @ np.abs(v)
            spread[a:b, h, 0] = np.where(see, abs(scale) * (np.abs(x) @ np.abs(k).T), 0.0).max(1)
    return out, reach, spread
