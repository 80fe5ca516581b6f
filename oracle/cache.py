"""fp64 definition of the paged key/value cache calls, in numpy.

Plain loops over requests, heads and tokens; shares no code with the GPU path.
Pages hold page_size consecutive tokens of one request; token j of request b is
at place j % page_size of page table[b][j // page_size].
"""

from __future__ import annotations

import math

import numpy as np


def plan(ctx, new, held, table, free, count, page_size, total):
    """(slots, q_offsets, kv_lens, held, count, table, free) after a plan, or
    the status code of a plan that hands out nothing.  Lists of ints in."""
    table, stack = [list(r) for r in table], list(free[:count])
    width, pool = (len(table[0]) if table else 0), len(free)
    if any(c < 0 or n < 0 or h < 0 or h > width or c + n > width * page_size for c, n, h in zip(ctx, new, held)):
        return 6
    if sum(new) > total or not 0 <= count <= pool:
        return 6
    want = [-(-(c + n) // page_size) for c, n in zip(ctx, new)]
    for b, w in enumerate(want):
        stack += table[b][w:held[b]]
    if len(stack) > pool:
        return 6
    if sum(max(0, w - h) for w, h in zip(want, held)) > len(stack):
        return 8
    free = list(free)
    pushed = list(stack)
    for b, w in enumerate(want):
        for i in range(held[b], w):
            table[b][i] = stack.pop()
    for i in range(count, len(stack)):
        free[i] = pushed[i]
    slots, offsets = [], [0]
    for b, n in enumerate(new):
        for t in range(ctx[b], ctx[b] + n):
            page = table[b][t // page_size]
            slots.append(page * page_size + t % page_size if 0 <= page < pool else -1)
        offsets.append(offsets[-1] + n)
    slots += [-1] * (total - len(slots))
    return slots, offsets, [c + n for c, n in zip(ctx, new)], want, len(stack), table, free


def act(name, x):
    if name == "gelu":
        return x * 0.5 * np.vectorize(math.erfc)(-x / math.sqrt(2))  # (1 + erf has no digit left below -8)
    return x / (1 + np.exp(-x))


def attend(q, k_cache, v_cache, table, q_off, kv_lens, name, scale, bias=None, window=0, mask=None, depths=None):
    """fp64 (out, lse, size, score_err, vsum) of the attention from the new tokens:
    `size` is sum |P||V| per output, `vsum` sum |V| over the seen tokens and
    `score_err` the row's largest sum |q||k| scale, for tolerances.  Rows
    behind q_off[-1] are NaN."""
    total, heads, d = q.shape
    kv_heads, page = k_cache.shape[2], k_cache.shape[1]
    out = np.full((total, heads, d), np.nan)
    size, vsum = np.full_like(out, np.nan), np.full_like(out, np.nan)
    lse, dot = np.full((heads, total), np.nan), np.full((heads, total), np.nan)
    for b, length in enumerate(kv_lens):
        lo, hi = q_off[b], q_off[b + 1]
        ctx = length - (hi - lo)
        place = [(table[b][j // page], j % page) for j in range(length)]
        depth = [int(depths[lo + t]) if depths is not None else t for t in range(hi - lo)]
        pos = np.array(list(range(ctx)) + [ctx + x for x in depth])
        for t in range(hi - lo):
            sees = np.ones(length, bool)
            for u in range(hi - lo):
                sees[ctx + u] = u <= t if mask is None else bool((int(mask[lo + t][u // 32]) >> (u % 32)) & 1)
            apart = ctx + depth[t] - pos
            if window:
                sees &= np.abs(apart) < window
            js = np.nonzero(sees)[0]
            for h in range(heads):
                if not len(js):
                    out[lo + t, h], size[lo + t, h], vsum[lo + t, h] = 0.0, 0.0, 0.0
                    lse[h, lo + t], dot[h, lo + t] = -np.inf, 0.0
                    continue
                pg, at = np.array([place[j] for j in js]).T
                k = k_cache[pg, at, h // (heads // kv_heads)]
                v = v_cache[pg, at, h // (heads // kv_heads)]
                x = scale * (k @ q[lo + t, h])
                dot[h, lo + t] = scale * np.max(np.abs(k) @ np.abs(q[lo + t, h]))
                if bias is not None:
                    reach = (bias.shape[1] - 1) // 2
                    x = x + bias[h][np.clip(apart[js], -reach, reach) + reach]
                if name == "softmax":
                    top = np.max(x)
                    p = np.exp(x - top)
                    lse[h, lo + t] = top + np.log(np.sum(p))
                    p = p / np.sum(p)
                else:
                    p = act(name, x)
                out[lo + t, h] = p @ v
                size[lo + t, h] = np.abs(p) @ np.abs(v)
                vsum[lo + t, h] = np.sum(np.abs(v), axis=0)
    return out, lse, size, dot, vsum
