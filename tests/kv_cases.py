"""Paged caches for the decode-attention tests: random rows on the device, with everything that a
call must not look at poisoned (NaN, infinities, page entries far outside the cache)."""
import numpy as np
import torch

import gguf_block_quantized_q4_gb300 as mq

KINDS = {"f16": mq.F16, "bf16": mq.BF16, "q8_0": mq.Q8_0}
IO = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def numpy_of(t):
    return (t.float() if t.dtype == torch.bfloat16 else t).cpu().numpy()


class Paged:
    """A cache of S sequences with `lens` rows; pages in random order."""

    def __init__(self, kind, lens, hkv, dim, page_size, layout="hnd", sums=False, seed=0,
                 spare=3, max_len=None):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.lens_list, self.page_size, self.layout = kind, list(lens), page_size, layout
        need = [-(-n // page_size) for n in lens]
        n_pages = sum(need) + spare
        self.max_len = max(max_len or 0, max(lens, default=1), 1)
        width = -(-self.max_len // page_size)
        order = torch.randperm(n_pages, generator=g)
        self.free = order[sum(need):].tolist()
        table = torch.full((len(lens), width), 0x7FFFFFFF, dtype=torch.int32)  # stale entries
        live = torch.zeros((n_pages, page_size), dtype=torch.bool)
        at = 0
        for s, n in enumerate(lens):
            own = order[at:at + need[s]]
            at += need[s]
            table[s, :need[s]] = own.int()
            for i, p in enumerate(own.tolist()):
                live[p, :min(page_size, n - i * page_size)] = True
        shape = (n_pages, hkv, page_size)
        planes = {}
        for name in ("k", "v"):
            if kind == "q8_0":
                q = torch.randint(-128, 128, (*shape, dim), generator=g, dtype=torch.int16).to(torch.int8)
                sc = (torch.randn((*shape, dim // 32), generator=g).abs() * 0.02).half()
                sc[~live[:, None, :].expand(shape)] = float("nan")
                planes[name], planes[name + "_scale"] = q, sc
            else:
                x = torch.randn((*shape, dim), generator=g).to(IO[kind])
                if name == "v":
                    x = x + 0.3
                x[~live[:, None, :].expand(shape)] = float("nan") if name == "k" else float("inf")
                planes[name] = x
        if sums:
            w = torch.rand(shape, generator=g)
            w[~live[:, None, :].expand(shape)] = float("nan")
            planes["sums"] = w
        self.host = {n: numpy_of(t) for n, t in planes.items()}
        if layout == "nhd":
            planes = {n: t.transpose(1, 2).contiguous() for n, t in planes.items()}
        self.dev = {n: t.cuda() for n, t in planes.items()}
        self.cache = self.wrap()
        self.pages, self.pages_host = table.cuda(), table.numpy()
        self.lens = torch.tensor(self.lens_list, dtype=torch.int32, device="cuda")

    def wrap(self):
        d = self.dev
        return mq.KVCache(KINDS[self.kind], d["k"], d["v"], d.get("k_scale"), d.get("v_scale"),
                          d.get("sums"), layout=self.layout)

    def read(self, name):
        """A plane from the device, as [page][head][slot]."""
        t = self.dev[name]
        return numpy_of(t.transpose(1, 2).contiguous() if self.layout == "nhd" else t)


def half_ulp(io):
    """Relative rounding error of an output of this type."""
    return {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[io]


def tiny(io):
    """Absolute rounding error near zero: half of the type's smallest subnormal, and room for
    sums that cancel in binary32."""
    return {"f32": 1e-30, "f16": 2.0 ** -25, "bf16": 1e-30}[io]


def attn_bound(dim, reach, mass, o, io):
    """|o - o_exact| per element.  A logit's error: the parts of the query hold 2^-22 of each
    product, and the dim/16 * 3 accumulation steps of the tensor cores lose at most 2^-22 of the
    running sum each (they may truncate), all times reach = scale * max_i sum |q||k_i|; twice
    that in the weights' quotient.  The weights' own parts 2^-22, exp 2^-21, sums over tiles, warps
    and pieces 2^-18, of mass = sum w|v|.  Then the rounding to the output's type."""
    rel = 2 * reach * (3 * dim / 16 + 2) * 2.0 ** -22 + 2.0 ** -17
    return np.expm1(rel)[..., None] * mass + half_ulp(io) * 1.01 * np.abs(o) + tiny(io)
