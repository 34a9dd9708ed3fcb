"""The decode-attention operators in 64 bits, from their definitions: test infrastructure that
shares nothing with the CUDA path.  A cache is a dict of numpy arrays in [page][head][slot] order:
k, v (f16 / bf16 as float64 values, or int8 quants with k_scale, v_scale), sums."""
from __future__ import annotations

import math

import numpy as np


def values(cache, name):
    """A plane's values in 64 bits."""
    x = np.asarray(cache[name], np.float64)
    if cache.get(name + "_scale") is not None:
        sc = np.asarray(cache[name + "_scale"], np.float64)
        x = x * np.repeat(sc, 32, axis=-1)
    return x


def place(pages, page_size, pos):
    """(page, slot) of the positions of one sequence."""
    pos = np.asarray(pos)
    return np.asarray(pages)[pos // page_size], pos % page_size


def attn_decode(cache, page_size, q, pages, lens, scale, window=0):
    """(o, mass, reach, weights): o [S][Hq][D]; mass = sum_i w_i |v_i| and
    reach = scale * max_i sum_d |q_d k_id|, the yardsticks of the error bound; weights: per
    sequence, [Hkv][n] sums over the group's heads, with the first position read."""
    k, v = values(cache, "k"), values(cache, "v")
    hkv = k.shape[1]
    S, hq, d = q.shape
    q = np.asarray(q, np.float64)
    group = hq // hkv
    o, mass = np.zeros((S, hq, d)), np.zeros((S, hq, d))
    reach, weights = np.zeros((S, hq)), []
    for s in range(S):
        n = int(lens[s])
        lo = max(0, n - window) if window else 0
        w_sum = np.zeros((hkv, n - lo))
        if n > lo:
            page, slot = place(pages[s], page_size, np.arange(lo, n))
            for a in range(hq):
                h = a // group
                kk, vv = k[page, h, slot], v[page, h, slot]
                x = scale * (kk @ q[s, a])
                reach[s, a] = abs(scale) * (np.abs(kk) @ np.abs(q[s, a])).max()
                w = np.exp(x - x.max())
                w /= w.sum()
                o[s, a], mass[s, a] = w @ vv, w @ np.abs(vv)
                w_sum[h] += w
        weights.append((lo, w_sum))
    return o, mass, reach, weights


def rope(x, table, pos, axis, pairs):
    """x [T][H][D] rotated, in x's own precision, each step rounded: pair i by
    table[pos[axis[i]][t]][i] = (cos, sin)."""
    y = x.copy()
    half = table.shape[1]
    for i in range(half):
        c, s = (table[pos[axis[i]], i, j].astype(x.dtype)[:, None] for j in range(2))
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, a] * s + x[:, :, b] * c
    return y


def quantise_rows(x):
    """Q8_0 rows of f32 x [...][D]: (int8 quants, f16 scales)."""
    blocks = x.astype(np.float32).reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(blocks).max(-1)
    d = np.minimum(amax / np.float32(127), np.float32(65504)).astype(np.float16)
    df = d.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(df == 0, np.float32(0), np.rint(blocks / df))
    return np.clip(q, -127, 127).astype(np.int8).reshape(x.shape), d


def evict(sums, n, keep, sink, recent):
    """Positions that stay of one kv head with the weight sums of its n rows."""
    if n <= keep:
        return list(range(n))

    def worth(i):
        w = float(sums[i])
        return math.inf if math.isnan(w) else w
    # NaN before every number, then the larger sum, then the lower position
    middle = sorted(range(sink, n - recent),
                    key=lambda i: (not math.isnan(float(sums[i])), -worth(i), i))
    return sorted([*range(sink), *middle[:keep - sink - recent], *range(n - recent, n)])
