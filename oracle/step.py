"""fp64 definitions of the calls around the attention, in numpy: norms with
rotation and their gradients, verification of drafted tokens, 4-bit rows.

Plain loops and textbook formulas; shares no code with the GPU path.
"""

from __future__ import annotations

import math

import numpy as np


def pair_columns(pairs, interleaved):
    i = np.arange(pairs)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)


def rotate(x, pos, freq, interleaved, back=False):
    """x [rows, heads, d] with every pair turned by pos * freq (back: the other way)."""
    a, b = pair_columns(len(freq), interleaved)
    t = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freq, np.float64)
    c, s = np.cos(t), np.sin(t) * (-1 if back else 1)
    y = np.array(x, np.float64)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def norm(x, w, eps):
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * (1.0 if w is None else w)


def norm_rotate(x, pos, freq, w, eps, interleaved):
    return rotate(x if eps is None else norm(x, w, eps), pos, freq, interleaved)


def norm_rotate_bwd(dy, x, pos, freq, w, eps, interleaved):
    """(dx, dw, size): size is what an element's sum adds up, for tolerances."""
    g = rotate(dy, pos, freq, interleaved, back=True)
    if eps is None:
        return g, None, np.abs(g)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    h = x * r
    dh = g if w is None else g * w
    size = r * (np.abs(dh) + np.abs(h) * np.mean(np.abs(dh * h), -1, keepdims=True))
    return r * (dh - h * np.mean(dh * h, -1, keepdims=True)), np.sum(g * h, (0, 1)), size


def positions(offsets, rows):
    """Places within the segments; -1 behind the last."""
    pos = np.full(rows, -1, np.int64)
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        pos[lo:hi] = np.arange(hi - lo)
    return pos


def verify(target, tokens, offsets, uniforms, draft=None, parents=None):
    """(accepted, next, places), a request at a time.  target and draft hold
    fp32 values as float64.  Entries of target below zero, infinite or NaN count as 0."""
    accepted, following, places = [], [], np.full(len(tokens), -1, np.int64)
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        if lo == hi:
            accepted.append(0)
            following.append(-1)
            continue
        children = [[] for _ in range(hi - lo)]
        for t in range(1, hi - lo):
            up = t - 1 if parents is None else parents[lo + t]
            if 0 <= up < t and 0 <= tokens[lo + t] < target.shape[1]:
                children[up].append(t)
        at, n = 0, 0
        while True:
            places[lo + at] = n
            n += 1
            p, gone, step = target[lo + at], set(), None
            counts = lambda x: float(p[x]) if 0 < p[x] < math.inf else 0.0  # noqa: E731
            for t in children[at]:
                x, u = tokens[lo + t], float(uniforms[lo + t])
                if draft is not None:
                    stays = u * float(draft[lo + t][x]) < counts(x) > 0
                else:
                    stays = x not in gone and u * (1 - math.fsum(counts(g) for g in gone)) < counts(x)
                if stays:
                    step = t
                    break
                gone.add(x)
            if step is None:
                break
            at = step
        rest = np.array(p)
        if draft is not None:
            if at + 1 < hi - lo:
                q = draft[lo + at + 1]
                with np.errstate(invalid="ignore"):
                    rest = (p.astype(np.float32) - q.astype(np.float32)).astype(np.float64)
        else:
            rest[list(gone)] = 0.0
        accepted.append(n)
        following.append(draw(rest, uniforms[lo]))
        if following[-1] < 0:
            following[-1] = draw(p, uniforms[lo])
    return accepted, following, places


def draw(weights, u):
    w = np.where((weights > 0) & np.isfinite(weights), weights, 0.0)
    total = math.fsum(w)
    if total == 0:
        return -1
    some = np.nonzero(w)[0]
    run = 0.0
    for i in some:
        run = math.fsum((run, w[i]))
        if run > u * total:
            return int(i)
    return int(some[-1])


def bf16(x):
    """float32 rounded to bf16, halves to even."""
    with np.errstate(all="ignore"):
        bits = np.asarray(x, np.float32).view(np.uint32)
    odd = (bits >> 16) & 1
    out = ((bits + 0x7FFF + odd) & np.uint32(0xFFFF0000)).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(x), out, np.asarray(x, np.float32))


def quantise(x):
    """(codes, step, middle) of heads [..., d], by the definition's fp32 steps."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
        step = bf16((hi - lo) / np.float32(15))
        middle = bf16(lo + np.float32(8) * step)
        c = np.where(step > 0, np.rint((x - middle) / step), np.float32(0))
    return (np.clip(c, -8, 7) + 8).astype(np.int64), step[..., 0], middle[..., 0]


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(codes):
    c = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],))
    c[..., 0::2], c[..., 1::2] = codes & 15, codes >> 4
    return c


def values(codes, scales):
    """What codes [..., d / 2] with scales [..., 2] (step, middle) stand for, in fp64."""
    return scales[..., 1:] + scales[..., :1] * (unpack(codes) - 8)
