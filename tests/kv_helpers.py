"""Batches, caches and masks for the KV cache tests, on the GPU and as the
oracle's float64 arrays."""
from __future__ import annotations

import numpy as np
import torch

from gpu_helpers import DEV, f64

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
DEAD = {"bf16": float("nan"), "e4m3": 0x7F, "i8": -128}       # what unwritten memory is filled with


def codes_f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to(torch.float32).to(torch.float64).cpu().numpy()


def oracle_cache(k, v, ks=None, vs=None):
    h = lambda t: None if t is None else t.cpu().numpy().copy()  # noqa: E731
    return dict(k=codes_f64(k), v=codes_f64(v), k_scale=h(ks), v_scale=h(vs))


def dead_cache(kind, n_pages, heads, page, dim):
    """k, v, k_scale, v_scale full of values that no result may depend on."""
    shape = (n_pages, heads, page, dim)
    if kind == "bf16":
        return [torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV) for _ in "kv"] + [None, None]
    raw = torch.uint8 if kind == "e4m3" else torch.int8
    codes = [torch.full(shape, DEAD[kind], dtype=raw, device=DEV).view(TYPES[kind]) for _ in "kv"]
    return codes + [torch.full(shape[:3], 255, dtype=torch.uint8, device=DEV) for _ in "kv"]


def make_plan(start, rows, page, seed=0, spare=2, pad=3):
    """(table, start, offsets as int32 GPU tensors; their numpy forms; n_pages,
    n_rows) with shuffled pages, each request's own."""
    rng = np.random.default_rng(seed)
    start, rows = np.asarray(start, dtype=np.int32), np.asarray(rows, dtype=np.int32)
    need = np.maximum(1, -(-(start + rows) // page))
    n_pages, width = int(need.sum()) + spare, int(need.max())
    order = rng.permutation(n_pages)
    table = np.full((len(start), width), -1, dtype=np.int32)   # entries past a request's pages are never read
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    offsets = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    gpu = [torch.from_numpy(x).to(DEV) for x in (table, start, offsets)]
    return gpu, (table, start, offsets), n_pages, int(offsets[-1]) + pad


def tree_mask(n_rows, offsets, words, seed=0, kind="tree"):
    """uint64 [n_rows, words]: random trees in drafting order ("tree"), every
    node ("full"), or random bits, empty rows among them ("random").  Bits past
    a request's nodes are set at random: they are ignored."""
    rng = np.random.default_rng(seed)
    bits = rng.integers(0, 2, size=(n_rows, words * 64)).astype(bool)
    for r in range(len(offsets) - 1):
        a, n = int(offsets[r]), int(offsets[r + 1] - offsets[r])
        for i in range(n):
            if kind == "full":
                bits[a + i, :n] = True
            elif kind == "random":
                bits[a + i, :n] = rng.random(n) < rng.choice([0.0, 0.1, 0.5])
            else:
                bits[a + i, :n] = bits[a + rng.integers(max(0, i - 6), i), :n] if i else False
                bits[a + i, i] = True
    return np.packbits(bits, axis=-1, bitorder="little").view(np.uint64)


def mask_tensor(mask):
    return None if mask is None else torch.from_numpy(mask.view(np.int64).copy()).to(DEV)


def rand_rows(n_rows, heads, dim, dtype, seed, packed=True):
    """[n_rows, heads, dim] as slices of a wider packed row (strided), with a
    few large channels."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((n_rows, heads + 2 if packed else heads, dim), generator=gen, device=DEV)
    x[..., :2] *= 9
    x = x.to(TYPES[dtype])
    return x[:, 1:1 + heads] if packed else x


def attention_bound(out, spread, reach, dim):
    """Largest difference of the kernel's bf16 result from the float64 one.
    With u = 2^-24 (half a step of fp32), b = 2^-8 (half a step of bf16):
      a score is off by at most (dim + 6) u reach (the dot product's additions,
      the two scalings, the difference from the maximum), so a weight, with the
      exponential's own few u, by a factor within 1 +- e, e = 2 (dim + 16) u
      reach + 16 u (numerator and sum move apart by twice as much at most);
      the weight's rounding to bf16 and the additions of weight times value are
      within (b + 4096 u) spread, and the final rounding within b |out|."""
    u, b = 2.0 ** -24, 2.0 ** -8
    e = np.expm1(2 * (2 * (dim + 16) * u * reach + 16 * u))[..., None]
    value = np.abs(out)
    first = (b + 4096 * u + e) * spread
    return (first + b * (value + first)) * 1.001 + 1e-37


__all__ = ["f64"]
