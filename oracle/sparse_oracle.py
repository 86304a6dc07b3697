"""Plain numpy oracle of the bounds of a paged cache's pages, of the choice of
blocks by them and of the attention over chosen blocks.  Written from the
definitions alone; shares no code with the HIP path.  Test infrastructure only.

A cache is a dict as in kv_oracle."""
from __future__ import annotations

import math

import numpy as np

from oracle import kv_oracle as K


def _exponent(amax: float) -> int:
    """The smallest e >= -100 with amax * 2^-e <= 127."""
    e = -100
    while math.ldexp(amax, -e) > 127:
        e += 1
    return e


def n_blocks(start, page_size, width):
    return min(max(int(start), 0) // page_size, width)


def bounds(cache, codes, scale, table, start, end):
    """codes int [n_pages, heads, 2, dim] and scale [n_pages, heads], changed in place."""
    n_pages, heads, page_size, _ = cache["k"].shape
    for r in range(len(start)):
        if end[r] <= max(int(start[r]), 0):
            continue
        for b in range(n_blocks(start[r], page_size, len(table[r])), n_blocks(end[r], page_size, len(table[r]))):
            p = int(table[r][b])
            if not 0 <= p < n_pages:
                continue
            for h in range(heads):
                k = cache["k"][p, h]
                if cache["k_scale"] is not None:
                    k = k * K.scale_value(cache["k_scale"][p, h])[:, None]
                k = np.where(np.abs(k) > np.finfo(np.float32).max, np.inf, k)   # a value is read in fp32
                if not np.isfinite(k).all():
                    codes[p, h], scale[p, h] = 0, 255
                    continue
                e = _exponent(np.abs(k).max())
                codes[p, h, 0] = np.floor(np.ldexp(k.min(0), -e))
                codes[p, h, 1] = np.ceil(np.ldexp(k.max(0), -e))
                scale[p, h] = e + 127


def query_codes(q):
    """q [group, dim] float64 -> whole numbers."""
    if not np.isfinite(q).all():
        return np.zeros(q.shape, dtype=np.int64)
    return np.rint(np.ldexp(q, -_exponent(np.abs(q).max()))).astype(np.int64)


def select(q, codes, scale, n_pages, page_size, table, start, offsets, take, n_first, n_last, out):
    """q [n_rows, q_heads, dim] float64; fills out [n_rows, heads, take]."""
    heads = codes.shape[1]
    group = q.shape[1] // heads
    for r in range(len(start)):
        blocks = n_blocks(start[r], page_size, len(table[r]))
        for row in range(int(offsets[r]), int(offsets[r + 1])):
            for h in range(heads):
                c = query_codes(q[row, h * group:(h + 1) * group])
                ranked = []
                for b in range(blocks):
                    p = int(table[r][b])
                    if b < n_first or b >= blocks - n_last:
                        score = (2, 0.0)
                    elif not 0 <= p < n_pages or scale[p, h] == 255:
                        score = (1, 0.0)
                    else:
                        edge = np.where(c > 0, codes[p, h, 1].astype(np.int64), codes[p, h, 0].astype(np.int64))
                        score = (0, math.ldexp(int((c * edge).sum(1).max()), int(scale[p, h]) - 127))
                    ranked.append((-score[0], -score[1], b))
                chosen = sorted(b for _, _, b in sorted(ranked)[:take])
                out[row, h] = chosen + [-1] * (take - len(chosen))


def sparse_attention(q, cache, table, start, offsets, blocks, mask, scale, out):
    """As kv_oracle.tree_attention, over the positions of blocks [n_rows, heads,
    take], the tail and the nodes.  Returns (spread, reach)."""
    n_pages, heads, page_size, _ = cache["k"].shape
    group = q.shape[1] // heads
    spread, reach = np.zeros_like(out), np.zeros(out.shape[:2])
    for r in range(len(start)):
        n, a = int(offsets[r + 1] - offsets[r]), int(start[r])
        full = n_blocks(a, page_size, len(table[r]))
        for i in range(n):
            row = int(offsets[r]) + i
            for g in range(heads):
                named = [b for before, b in zip([-1, *blocks[row, g][:-1]], blocks[row, g]) if 0 <= b < full and b > before]
                pos = [b * page_size + s for b in named for s in range(page_size)]
                pos += list(range(full * page_size, a))
                pos += [a + j for j in range(n) if K.sees(mask, int(offsets[r]), i, j)]
                if not pos:
                    out[row, g * group:(g + 1) * group] = 0.0
                    continue
                kk = np.stack([K.row_at(cache, "k", table[r], t)[g] for t in pos])
                vv = np.stack([K.row_at(cache, "v", table[r], t)[g] for t in pos])
                for h in range(g * group, (g + 1) * group):
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = scale * (kk @ q[row, h])
                        w = np.exp(s - s.max())
                        w = w / w.sum()
                        out[row, h] = w @ vv
                        spread[row, h] = w @ np.abs(vv)
                        reach[row, h] = scale * (np.abs(kk) @ np.abs(q[row, h])).max()
    return spread, reach
