"""Paged caches of Q4_0 rows for the tests: as kv_cases.Paged, with what no call may read poisoned."""
import numpy as np
import torch

import gguf_block_quantized_q4_gb300 as mq
from oracle import kv
from tests.kv_cases import Paged, half_ulp, tiny


class Paged4(Paged):
    def __init__(self, lens, hkv, dim, page_size, layout="hnd", sums=False, seed=0, spare=3, max_len=None,
                 scale=0.1):
        super().__init__("q8_0", lens, hkv, dim, page_size, layout, sums, seed, spare, max_len)
        g = torch.Generator().manual_seed(seed + 1)
        for name in ("k", "v"):
            shape = self.host[name].shape
            n = torch.randint(0, 256, (*shape[:3], dim // 2), generator=g, dtype=torch.int16).to(torch.uint8)
            # scales of both signs, in the places of the poisoned cache's numbers
            dead = np.isnan(self.host[name + "_scale"])
            sc = (torch.randn((*shape[:3], dim // 32), generator=g) * scale).half().numpy()
            sc[dead] = np.nan
            self.set(name, n.numpy(), sc)
        self.cache = self.wrap()

    def set(self, name, packed, scales):
        """Rows [page][head][slot] of bytes, with their scales."""
        self.host[name] = kv.unpack4(packed).astype(np.int8) - 8
        self.host[name + "_scale"] = scales
        for n, x in ((name, packed), (name + "_scale", scales)):
            t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
            self.dev[n] = t.transpose(1, 2).contiguous() if self.layout == "nhd" else t

    def wrap(self):
        d = self.dev
        if d["k"].dtype != torch.uint8:  # (called once before the rows are set)
            return None
        return mq.KVCache(mq.Q4_0, d["k"], d["v"], d["k_scale"], d["v_scale"], d.get("sums"), layout=self.layout)


def attn_bound4(p, q, ref, mass, reach, scale, window, io):
    """|o - o_exact| per element over Q4_0 rows, and the relative bound of a weight.  A block's product
    runs over four accumulation steps of products of numbers up to 8 in magnitude: each step
    loses at most 2^-22 of 8 sum |q| |d| (the tensor cores may truncate), and the query's parts
    2^-22 of it; the blocks' sums, scaled in binary32, lose 2^-23 of sum |q| |k| each.  Twice that in
    the weights' quotient; the weights' parts, exp, and the sums over tiles, warps and pieces 2^-17
    as for other rows; then the rounding to the output's type.  For bf16 activations the weights are one
    f16 part, rounded by 2^-12 of themselves, and their products with the scales once more: 2^-11 of
    mass.  And what f16 parts cannot hold of small weights: a weight p (2^7 for one that is the
    reference's, up to 2^15) and its product with a scale d below 1 (in units of `unit`, a power of two
    up to twice the largest scale) end in three roundings to steps of 2^-24, half a step each, so an
    element of a key with a number of at most 8 loses 8 * 3 * 2^-25 of 2^7 (the sum of the weights is
    at least that), which matters where the heavy keys' numbers are 0."""
    S, hq, dim = q.shape
    hkv = p.host["k"].shape[1]
    wide = np.zeros((S, hq))
    for s in range(S):
        n = p.lens_list[s]
        lo = max(0, n - window) if window else 0
        if n == lo:
            continue
        page, slot = kv.place(p.pages_host[s], p.page_size, np.arange(lo, n))
        for a in range(hq):
            d = np.abs(p.host["k_scale"][page, a // (hq // hkv), slot].astype(np.float64))
            sums = np.abs(q[s, a].astype(np.float64)).reshape(-1, 32).sum(-1)
            wide[s, a] = abs(scale) * 8 * (d @ sums).max()
    rel = 2 * (wide * 5 * 2.0 ** -22 + reach * (dim / 32 + 2) * 2.0 ** -23) + 2.0 ** -17
    unit = max(1.0, 2 * float(np.nanmax(np.abs(p.host["v_scale"].astype(np.float64)))))
    floor = np.array([24 * n * 2.0 ** -32 * unit for n in p.lens_list])[:, None, None]
    parts = 2.0 ** -11 if io == "bf16" else 0.0
    return floor + (np.expm1(rel)[..., None] + parts) * mass + half_ulp(io) * 1.01 * np.abs(ref) + tiny(io), rel
