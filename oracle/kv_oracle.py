"""Plain numpy oracle (float64) of the paged KV cache and of the attention of
drafted nodes over it.  Written from the definitions alone; shares no code with
the HIP path.  Test infrastructure only.

A cache is a dict: k, v [n_pages, heads, page_size, dim] hold the codes' values
in float64, k_scale, v_scale [n_pages, heads, page_size] the scale bytes (None
for a bf16 cache)."""
from __future__ import annotations

import numpy as np

TOP = {"e4m3": 448.0, "i8": 127.0}
MIN_EXP = -100


def nearest_code(y: np.ndarray, kind: str) -> np.ndarray:
    """Float64 to the nearest value of the 8-bit type, ties to even (|y| <= the
    type's top).  e4m3: 3 fraction bits, smallest normal 2^-6, step 2^-9 below."""
    if kind == "i8":
        return np.rint(y)
    with np.errstate(divide="ignore"):
        e = np.maximum(np.floor(np.log2(np.abs(y))), -6.0)
    step = np.exp2(e - 3)
    return np.rint(y / step) * step


def quantise_rows(x: np.ndarray, kind: str):
    """x [..., dim] float64 -> (codes' values, scale bytes) of an 8-bit cache."""
    finite = np.isfinite(x).all(-1)
    safe = np.where(finite[..., None], x, 0.0)
    amax = np.abs(safe).max(-1)
    e = np.full(amax.shape, MIN_EXP, dtype=np.int64)
    for i in np.ndindex(amax.shape):
        while amax[i] * 2.0 ** -float(e[i]) > TOP[kind]:
            e[i] += 1
    codes = nearest_code(safe * np.exp2(-e.astype(np.float64))[..., None], kind)
    return codes, np.where(finite, e + 127, 255).astype(np.uint8)


def scale_value(b: np.ndarray) -> np.ndarray:
    return np.where(b == 255, np.nan, np.exp2(b.astype(np.float64) - 127))


def place(cache, table_row, t):
    """(page, slot) of a position, or None where it has no page in the pool."""
    n_pages, _, page_size, _ = cache["k"].shape
    if t < 0 or t // page_size >= len(table_row):
        return None
    page = int(table_row[t // page_size])
    return (page, t % page_size) if 0 <= page < n_pages else None


def write(cache, kind, k, v, table, start, offsets):
    """k, v [n_rows, heads, dim] float64 (already bf16 values for a bf16 cache)."""
    for r in range(len(start)):
        for i in range(int(offsets[r + 1] - offsets[r])):
            at = place(cache, table[r], int(start[r]) + i)
            if at is None:
                continue
            for name, x in (("k", k), ("v", v)):
                row = x[offsets[r] + i]
                if kind == "bf16":
                    cache[name][at[0], :, at[1]] = row
                else:
                    cache[name][at[0], :, at[1]], cache[name + "_scale"][at[0], :, at[1]] = quantise_rows(row, kind)


def row_at(cache, name, table_row, t):
    """The values [heads, dim] at a position, NaN where it has no page."""
    at = place(cache, table_row, t)
    if at is None:
        return np.full(cache[name].shape[1::2], np.nan)
    codes = cache[name][at[0], :, at[1]]
    if cache[name + "_scale"] is None:
        return codes
    return codes * scale_value(cache[name + "_scale"][at[0], :, at[1]])[:, None]


def read(cache, table, start, offsets, outs):
    for r in range(len(start)):
        for i in range(int(offsets[r + 1] - offsets[r])):
            for name, out in zip("kv", outs):
                out[offsets[r] + i] = row_at(cache, name, table[r], int(start[r]) + i)


def commit(cache, table, start, paths, path_lens):
    for r in range(len(start)):
        for i in range(min(int(path_lens[r]), paths.shape[1])):
            src, dst = place(cache, table[r], int(start[r] + paths[r, i])), place(cache, table[r], int(start[r]) + i)
            if paths[r, i] < i or src is None or dst is None:
                continue
            for name in ("k", "v", "k_scale", "v_scale"):
                if cache[name] is not None:
                    cache[name][dst[0], :, dst[1]] = cache[name][src[0], :, src[1]].copy()


def sees(mask, offset, i, j):
    """Whether node i sees node j; mask uint64 [n_rows, words] or None (chain)."""
    return j <= i if mask is None else bool((int(mask[offset + i, j // 64]) >> (j % 64)) & 1)


def tree_attention(q, cache, table, start, offsets, mask, scale, out):
    """q [n_rows, q_heads, dim] float64; fills out (float64) at the rows of the
    batch.  Returns (sum_j w_j |v_j|, largest scale * sum_d |q_d k_d| over the
    seen positions) per output row, which error bounds are built from."""
    heads = cache["k"].shape[1]
    group = q.shape[1] // heads
    spread = np.zeros_like(out)
    reach = np.zeros(out.shape[:2])
    for r in range(len(start)):
        n, a = int(offsets[r + 1] - offsets[r]), int(start[r])
        if n == 0:
            continue
        keys = np.stack([row_at(cache, "k", table[r], t) for t in range(a + n)])
        vals = np.stack([row_at(cache, "v", table[r], t) for t in range(a + n)])
        for i in range(n):
            row = int(offsets[r]) + i
            seen = np.array([t < a or sees(mask, int(offsets[r]), i, t - a) for t in range(a + n)], dtype=bool)
            for h in range(q.shape[1]):
                if not seen.any():
                    out[row, h] = 0.0
                    continue
                kk, vv = keys[seen, h // group], vals[seen, h // group]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (kk @ q[row, h])
                    w = np.exp(s - s.max())
                    w = w / w.sum()
                    out[row, h] = w @ vv
                    spread[row, h] = w @ np.abs(vv)
                    reach[row, h] = scale * (np.abs(kk) @ np.abs(q[row, h])).max()
    return spread, reach
