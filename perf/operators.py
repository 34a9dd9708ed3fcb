"""Cases of the decode-attention operators: rotary positions with several axes on the QKV
product's output, stored into a paged key-value cache (``rope_store``); attention of one new
token per sequence over that cache (``attn_decode``); eviction of cached rows by their
accumulated attention weight (``kv_evict``).

``run`` computes an operator in its plain form (elementary torch operations in 32 bits), or,
with ``own`` set, through the package's calls.  ``exact`` computes the same outputs in 64 bits,
apart from both.

The cache holds rows of ``head_dim`` values per (page, kv head, slot): f16, bf16, or Q8_0
(int8 quants and one f16 scale per 32 values).  Planes are [page][head][slot] ("hnd") or
[page][slot][head] ("nhd").
"""
import math
import random

import torch

own = False

IO = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROW_BYTES = {"f16": lambda d: 2 * d, "bf16": lambda d: 2 * d, "q8_0": lambda d: d + d // 32 * 2}


def _attn(name, seqs, max_len, hq, hkv, dim, cache, io="f32", page=16, layout="hnd", ragged=True,
          window=0, track=False):
    return {"name": name, "op": "attn", "seqs": seqs, "max_len": max_len, "hq": hq, "hkv": hkv,
            "dim": dim, "cache": cache, "io": io, "page": page, "layout": layout,
            "ragged": ragged, "window": window, "track": track}


def _rope(name, tokens, hq, hkv, dim, cache, io="f32", page=16, layout="hnd", rot=None, axes=1,
          style="half", weave=False, bias=True, max_pos=32768):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": hq, "hkv": hkv, "dim": dim,
            "cache": cache, "io": io, "page": page, "layout": layout, "rot": rot or dim,
            "axes": axes, "style": style, "weave": weave, "bias": bias, "max_pos": max_pos}


def _evict(name, seqs, max_len, keep, hkv, dim, cache, page=16, layout="hnd", sink=4, recent=32,
           ragged=True):
    return {"name": name, "op": "evict", "seqs": seqs, "max_len": max_len, "keep": keep,
            "hkv": hkv, "dim": dim, "cache": cache, "page": page, "layout": layout,
            "sink": sink, "recent": recent, "ragged": ragged}


def listed():
    return [
        # the first tokens of one chat on the Qwen2.5-0.5B head layout: latency is all
        _attn("attn 1x37 14/2x64 f16", 1, 37, 14, 2, 64, "f16", ragged=False),
        # a small batch of ordinary chats on the Qwen2.5-7B head layout
        _attn("attn 8x1k 28/4x128 f16", 8, 1100, 28, 4, 128, "f16"),
        # a full serving batch of unlike lengths, one slot of it idle, on the quantised cache
        _attn("attn 64x8k 28/4x128 q8_0", 64, 8192, 28, 4, 128, "q8_0", page=32),
        # one long document: few rows, all of the length to split
        _attn("attn 1x131072 28/4x128 bf16", 1, 131072, 28, 4, 128, "bf16", io="bf16", page=64,
              ragged=False),
        # a batch whose cache will be evicted from: the weights are summed too
        _attn("attn 32x4k 32/8x128 f16 track", 32, 4001, 32, 8, 128, "f16", io="f16", track=True,
              layout="nhd"),
        # one head per kv head, odd page size, sliding window that starts inside a page
        _attn("attn 5x2k 12/12x96 q8_0 window", 5, 2047, 12, 12, 96, "q8_0", page=24,
              window=1000, track=True),
        # one decode step of a batch of eight
        _rope("rope 8 28/4x128 f16", 8, 28, 4, 128, "f16"),
        # prefill of image patches: time, height and width axes in contiguous sections
        _rope("rope 4096 28/4x128 f16 3 axes", 4096, 28, 4, 128, "f16", axes=3),
        # prefill into the quantised cache, half of each head rotated, neighbouring pairs,
        # axes woven through the pairs
        _rope("rope 1023 32/8x128 q8_0 woven", 1023, 32, 8, 128, "q8_0", io="bf16", rot=64,
              axes=3, style="pairs", weave=True, bias=False, page=32, layout="nhd"),
        # two short chats just over their budget
        _evict("evict 2x300 to 256 2x64 f16", 2, 300, 256, 2, 64, "f16"),
        # a batch brought back to half of its length
        _evict("evict 16x4k to 2k 4x128 q8_0", 16, 4096, 2048, 4, 128, "q8_0", page=32),
        # one long document brought down to a quarter
        _evict("evict 1x131072 to 32768 4x128 f16", 1, 131072, 32768, 4, 128, "f16", page=64,
               recent=1024, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "evict"])
    dim = rng.choice([64, 96, 128, 128, 256])
    hq, hkv = rng.choice([(14, 2), (28, 4), (32, 8), (12, 12), (16, 1), (20, 4), (7, 7)])
    common = dict(page=rng.choice([8, 16, 24, 32, 64, 100]), layout=rng.choice(["hnd", "nhd"]))
    cache = rng.choice(["f16", "bf16", "q8_0"])
    row = 2 * hkv * ROW_BYTES[cache](dim)
    if op == "attn":
        seqs = _log(rng, 1, 64)
        max_len = max(1, min(_log(rng, 1, 131072), int(2.2e8 / (row * seqs))))
        window = 0 if rng.random() < 0.7 else _log(rng, 1, max_len)
        return _attn("x", seqs, max_len, hq, hkv, dim, cache, io=rng.choice(["f32", "f32", "f16", "bf16"]),
                     window=window, track=rng.random() < 0.3, **common)
    if op == "rope":
        tokens = _log(rng, 1, 4096 * 36 * 128 // ((hq + 2 * hkv) * dim) // 2)
        axes = rng.randint(1, 4)
        return _rope("x", tokens, hq, hkv, dim, cache, io=rng.choice(["f32", "f32", "f16", "bf16"]),
                     rot=rng.choice([dim, dim, dim // 2]), axes=axes, style=rng.choice(["half", "pairs"]),
                     weave=axes > 1 and rng.random() < 0.5, bias=rng.random() < 0.5,
                     max_pos=rng.choice([4096, 32768, 131072]), **common)
    seqs = _log(rng, 1, 16)
    max_len = max(16, min(_log(rng, 16, 131072), int(2.2e8 / (row * seqs))))
    keep = _log(rng, 8, max_len)
    sink, recent = rng.randint(0, min(4, keep // 4)), rng.randint(0, keep // 4)
    return _evict("x", seqs, max_len, keep, hkv, dim, cache, sink=sink, recent=recent, **common)


# ---- inputs -----------------------------------------------------------------------------


def _lens(c):
    """The sequences' lengths: the same for every seed, so that work() knows them."""
    n, top = c["seqs"], c["max_len"]
    if not c["ragged"]:
        return [top] * n
    r = random.Random(n * 1000003 + top)
    lens = [r.randint(1, top) for _ in range(n)]
    lens[r.randrange(n)] = top
    if n >= 5 and c["op"] == "attn":
        lens[(lens.index(top) + 1) % n] = 0  # an idle slot of the batch
    return lens


def _planes(c, n_pages, g, dev):
    """The cache's planes: k, v (and the scales of Q8_0), as [page][head][slot] or
    [page][slot][head] rows of dim values.  Rows that no sequence holds have values too."""
    hkv, ps, d = c["hkv"], c["page"], c["dim"]
    shape = (n_pages, hkv, ps) if c["layout"] == "hnd" else (n_pages, ps, hkv)
    p = {}
    for name in ("k", "v"):
        if c["cache"] == "q8_0":
            p[name] = torch.randint(-127, 128, (*shape, d), generator=g, device=dev, dtype=torch.int8)
            p[name + "_scale"] = (torch.randn((*shape, d // 32), generator=g, device=dev).abs() * 0.01
                                  + 0.001).half()
        else:
            x = torch.randn((*shape, d), generator=g, device=dev, dtype=torch.float32)
            p[name] = (x if name == "k" else x + 0.25).to(IO[c["cache"]])
    return p


def _inputs(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    s = {"case": c}
    hkv, ps, d = c["hkv"], c["page"], c["dim"]
    if c["op"] == "rope":
        n = c["tokens"]
        n_pages = -(-n // ps) + 2
        s.update(_planes(c, n_pages, g, dev))
        pages = torch.randperm(n_pages, generator=g, device=dev)
        i = torch.arange(n, device=dev)
        s["slot"] = pages[i // ps] * ps + i % ps
        s["qkv"] = torch.randn((n, (c["hq"] + 2 * hkv) * d), generator=g, device=dev).to(IO[c["io"]])
        s["bias"] = torch.randn((c["hq"] + 2 * hkv) * d, generator=g, device=dev) if c["bias"] else None
        half = c["rot"] // 2
        freq = 1e6 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        if c["weave"]:
            s["axis"] = [k % c["axes"] for k in range(half)]
        else:  # the first axis gets what is left over
            share = half // (c["axes"] + 1) if c["axes"] > 1 else 0
            s["axis"] = [max(0, min(c["axes"] - 1, (k - (half - share * (c["axes"] - 1))) // max(share, 1) + 1))
                         if c["axes"] > 1 else 0 for k in range(half)]
        ang = torch.arange(c["max_pos"], device=dev, dtype=torch.float64)[:, None] * freq
        s["table"] = torch.stack([ang.cos(), ang.sin()], -1).float()
        base = int(torch.randint(0, max(1, c["max_pos"] - n), (1,), generator=g, device=dev))
        grid = [i // 1024, i // 32 % 32, i % 32, i % 7]
        s["pos"] = torch.stack([(base + (i if c["axes"] == 1 else grid[a])) % c["max_pos"]
                                for a in range(c["axes"])]).int()
        return s
    lens = _lens(c)
    used = -(-c["max_len"] // ps)
    need = [-(-n // ps) for n in lens]
    new = -(-c["keep"] // ps) if c["op"] == "evict" else 0
    n_old = sum(need)
    s.update(_planes(c, n_old + new * c["seqs"] + 1, g, dev))
    # each sequence's pages lie anywhere in the pool; entries past its length are stale
    order = torch.randperm(n_old, generator=g, device=dev) if n_old else torch.zeros(1, device=dev, dtype=torch.int64)
    first = torch.tensor([sum(need[:k]) for k in range(len(need))], device=dev)
    at = (first[:, None] + torch.arange(used, device=dev)).clamp(max=max(n_old - 1, 0))
    s["pages"] = order[at].int().contiguous()
    s["lens"] = torch.tensor(lens, device=dev, dtype=torch.int32)
    shape = s["k"].shape[:-1]
    if c["op"] == "attn":
        # some keys lie along their queries: the weights are uneven, as trained ones are
        s["q"] = (torch.randn((c["seqs"], c["hq"], d), generator=g, device=dev) * 2).to(IO[c["io"]])
        s["sums"] = torch.rand(shape, generator=g, device=dev) if c["track"] else None
        return s
    s["sums"] = torch.rand(shape, generator=g, device=dev).pow(8) * 20
    # a share of equal sums, as rows have that no query has looked at
    s["sums"][torch.rand(shape, generator=g, device=dev) < 0.1] = 0.0
    s["n_old"] = n_old
    s["new_pages"] = (n_old + torch.randperm(new * c["seqs"], generator=g, device=dev)).int().view(c["seqs"], new)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # what a serving program keeps: the cache object, the rotation, the workspace
        import gguf_block_quantized_q4_gb300 as mq
        mq.init(0)
        kind = {"f16": mq.F16, "bf16": mq.BF16, "q8_0": mq.Q8_0}[case["cache"]]
        s["cache"] = mq.KVCache(kind, s["k"], s["v"], s.get("k_scale"), s.get("v_scale"),
                                s.get("sums"), layout=case["layout"])
        if case["op"] == "rope":
            s["rope"] = mq.Rope(s["table"], s["axis"], pairs=case["style"] == "pairs")
        if case["op"] == "attn":
            s["ws"] = mq.attn_workspace(s["cache"], case["seqs"], case["hq"], case["max_len"], case["track"])
    return s


# ---- the plain forms ----------------------------------------------------------------------


def _flat(s, name):
    """Rows of a plane and of its scales in one index."""
    return s[name].view(-1, s[name].shape[-1])


def _row_index(c, page, head, slot):
    if c["layout"] == "hnd":
        return (page * c["hkv"] + head) * c["page"] + slot
    return (page * c["page"] + slot) * c["hkv"] + head


def _values(s, name, rows):
    x = _flat(s, name)[rows].float()
    if s["case"]["cache"] == "q8_0":
        sc = _flat(s, name + "_scale")[rows].float()
        x = (x.unflatten(-1, (-1, 32)) * sc[..., None]).flatten(-2)
    return x


def _seq_rows(s, c, pages, length):
    """Row index of each (sequence, kv head, position), [S][Hkv][length]."""
    pos = torch.arange(length, device="cuda")
    page = pages.long()[:, pos // c["page"]]
    head = torch.arange(c["hkv"], device="cuda")
    return _row_index(c, page[:, None, :], head[None, :, None], (pos % c["page"])[None, None, :])


def _run_attn(s, c):
    n, d, group = c["max_len"], c["dim"], c["hq"] // c["hkv"]
    rows = _seq_rows(s, c, s["pages"], n)
    pos, lens = torch.arange(n, device="cuda"), s["lens"].long()[:, None]
    seen = pos < lens
    if c["window"]:
        seen = seen & (pos >= lens - c["window"])
    seen = seen[:, None, None, :]
    q = s["q"].float().view(c["seqs"], c["hkv"], group, d)
    w = torch.matmul(q, _values(s, "k", rows).transpose(-1, -2)) * (1.0 / math.sqrt(d))
    w = torch.where(seen, w, -math.inf)
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(-1, keepdim=True)
    w = w / torch.where(total == 0, 1.0, total)
    v = torch.where(seen[:, 0, :, :, None], _values(s, "v", rows), 0.0)
    o = torch.matmul(w, v).to(s["q"].dtype).view(c["seqs"], c["hq"], d)
    if not c["track"]:
        return {"o": o}
    # a row belongs to one sequence: what the others' stale page entries name gets nothing
    s["sums"].view(-1).index_add_(0, rows.flatten(), w.sum(2).flatten())
    return {"o": o, "sums": s["sums"]}


def _run_rope(s, c):
    n, d, half = c["tokens"], c["dim"], c["rot"] // 2
    x = s["qkv"].float()
    if s["bias"] is not None:
        x = x + s["bias"]
    x = x.view(n, -1, d)
    rotated, v = x[:, :c["hq"] + c["hkv"]], x[:, c["hq"] + c["hkv"]:]
    pair = torch.arange(half, device="cuda")
    at = s["table"][s["pos"].long()[torch.tensor(s["axis"], device="cuda")].T, pair]  # [n][half][2]
    cos, sin = at[:, None, :, 0], at[:, None, :, 1]
    rot, rest = rotated[..., :2 * half], rotated[..., 2 * half:]
    if c["style"] == "half":
        a, b = rot[..., :half], rot[..., half:]
        rot = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    rotated = torch.cat([rot, rest], -1)
    q = rotated[:, :c["hq"]].to(s["qkv"].dtype)
    slot = s["slot"][:, None]
    rows = _row_index(c, slot // c["page"], torch.arange(c["hkv"], device="cuda"), slot % c["page"])
    out = {"q": q}
    for name, y in (("k", rotated[:, c["hq"]:]), ("v", v)):
        if c["cache"] == "q8_0":
            blocks = y.unflatten(-1, (-1, 32))
            sc = (blocks.abs().amax(-1) / torch.full((), 127.0, device="cuda")).half()
            by = sc.float()[..., None]
            quants = torch.where(by == 0, 0.0, torch.round(blocks / by)).clamp(-127, 127)
            _flat(s, name)[rows] = quants.to(torch.int8).flatten(-2)
            _flat(s, name + "_scale")[rows] = sc
        else:
            _flat(s, name)[rows] = y.to(s[name].dtype)
        out[name] = _shown(s, name, 0)
    return out


def _shown(s, name, first):
    """A plane from page `first` on, as the values it stands for."""
    x = s[name][first:]
    if s["case"]["cache"] == "q8_0":
        return x.unflatten(-1, (-1, 32)) * s[name + "_scale"][first:][..., None]  # f16
    return x


def _run_evict(s, c):
    n, keep = c["max_len"], c["keep"]
    rows = _seq_rows(s, c, s["pages"], n)
    pos, lens = torch.arange(n, device="cuda"), s["lens"].long()[:, None]
    valid = pos < lens
    safe = valid & ((pos < c["sink"]) | (pos >= lens - c["recent"]) | (lens <= keep))
    rank = torch.where(safe[:, None], math.inf, s["sums"].view(-1)[rows])
    rank = torch.where(valid[:, None], rank, -math.inf)
    top = min(keep, n)
    kept = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :top]
    count = lens.clamp(max=keep)
    place = torch.arange(top, device="cuda")
    live = (place < count)[:, None].expand(kept.shape)
    kept = torch.where(live, kept, n).sort(-1).values  # in order, what is empty last
    src = torch.gather(rows, 2, kept.clamp(max=n - 1))
    dst = _seq_rows(s, c, s["new_pages"], top)
    for name in ("k", "v", "k_scale", "v_scale", "sums"):
        if s.get(name) is not None:
            plane = s[name].view(-1, s[name].shape[-1]) if name != "sums" else s[name].view(-1, 1)
            plane[dst] = torch.where(live[..., None], plane[src], plane[dst])
    out = torch.full((c["seqs"], c["hkv"], keep), -1, dtype=torch.int32, device="cuda")
    out[..., :top] = torch.where(live, kept, -1).int()
    return _evicted(s, out, count[:, 0].int())


def _evicted(s, kept, count):
    first = s["n_old"]
    return {"kept": kept, "lens": count, "k": _shown(s, "k", first), "v": _shown(s, "v", first),
            "sums": s["sums"][first:]}


def _run_own(s, c):
    import gguf_block_quantized_q4_gb300 as mq
    if c["op"] == "attn":
        o = mq.attn_decode(s["cache"], s["q"], s["pages"], s["lens"], c["max_len"], window=c["window"],
                           track=c["track"], ws=s["ws"])
        return {"o": o, "sums": s["sums"]} if c["track"] else {"o": o}
    if c["op"] == "rope":
        q = mq.rope_store(s["cache"], s["rope"], s["qkv"], s["pos"], s["slot"], c["hq"], bias=s["bias"])
        return {"q": q, "k": _shown(s, "k", 0), "v": _shown(s, "v", 0)}
    kept, count = mq.kv_evict(s["cache"], s["pages"], s["lens"], c["max_len"], s["new_pages"],
                              c["keep"], sink=c["sink"], recent=c["recent"])
    return _evicted(s, kept, count)


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    return {"attn": _run_attn, "rope": _run_rope, "evict": _run_evict}[c["op"]](state, c)


def work(case):
    c = case
    row = ROW_BYTES[c["cache"]](c["dim"])
    if c["op"] == "rope":
        size = torch.empty(0, dtype=IO[c["io"]]).element_size()
        n, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["dim"]
        return {"bytes": n * ((2 * hq + 2 * hkv) * d * size + 2 * hkv * row + c["rot"] * 4 + c["axes"] * 4 + 8),
                "flops": n * (hq + hkv) * c["rot"] * 3}
    lens = _lens(c)
    if c["op"] == "attn":
        keys = sum(min(n, c["window"]) if c["window"] else n for n in lens)
        size = torch.empty(0, dtype=IO[c["io"]]).element_size()
        return {"bytes": keys * c["hkv"] * (2 * row + (8 if c["track"] else 0)) + 2 * c["seqs"] * c["hq"] * c["dim"] * size,
                "flops": 4 * keys * c["hq"] * c["dim"]}
    kept = sum(min(n, c["keep"]) for n in lens)
    looked = sum(n for n in lens if n > c["keep"])
    return {"bytes": c["hkv"] * (looked * 4 + kept * (4 * row + 8 + 4)), "flops": c["hkv"] * looked}


# ---- 64 bits --------------------------------------------------------------------------------


def _row64(s, c, name, page, head, slot):
    """Rows of one kv head in 64 bits, by their place in the plane as it is laid out."""
    at = (page, head, slot) if c["layout"] == "hnd" else (page, slot, head)
    x = s[name][at].double()
    if c["cache"] == "q8_0":
        x = x * s[name + "_scale"][at].double().repeat_interleave(32, -1)
    return x


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "rope":
        return _exact_rope(c, s)
    lens = _lens(c)
    group = c["hq"] // c["hkv"] if c["op"] == "attn" else 1
    if c["op"] == "attn":
        o = torch.zeros((c["seqs"], c["hq"], c["dim"]), dtype=torch.float64, device="cuda")
        sums = s["sums"].double() if c["track"] else None
        for b, n in enumerate(lens):
            lo = max(0, n - c["window"]) if c["window"] else 0
            pos = torch.arange(lo, n, device="cuda")
            page, slot = s["pages"][b].long()[pos // c["page"]], pos % c["page"]
            for h in range(c["hkv"] if n else 0):
                k, v = (_row64(s, c, name, page, h, slot) for name in ("k", "v"))
                q = s["q"][b, h * group:(h + 1) * group].double()
                w = torch.softmax(q @ k.T / math.sqrt(c["dim"]), -1)
                o[b, h * group:(h + 1) * group] = w @ v
                if c["track"]:
                    sums[(page, h, slot) if c["layout"] == "hnd" else (page, slot, h)] += w.sum(0)
        return {"o": o, "sums": sums} if c["track"] else {"o": o}
    # eviction: chosen one by one, copied as stored
    k, v = ((s[n].double() if c["cache"] != "q8_0" else s[n].double() * s[n + "_scale"].double()
             .repeat_interleave(32, -1)) for n in ("k", "v"))
    sums = s["sums"].double()
    for b, n in enumerate(lens):
        for h in range(c["hkv"]):
            pos = torch.arange(n, device="cuda")
            page, slot = s["pages"][b].long()[pos // c["page"]], pos % c["page"]
            src = (page, h, slot) if c["layout"] == "hnd" else (page, slot, h)
            kept = list(range(n))
            if n > c["keep"]:
                middle = range(c["sink"], n - c["recent"])
                w = s["sums"][src].tolist()
                best = sorted(middle, key=lambda i: (-w[i], i))[:c["keep"] - c["sink"] - c["recent"]]
                kept = sorted([*range(c["sink"]), *best, *range(n - c["recent"], n)])
            kept = torch.tensor(kept, device="cuda", dtype=torch.int64)
            to = torch.arange(len(kept), device="cuda")
            to = (s["new_pages"][b].long()[to // c["page"]], to % c["page"])
            dst = (to[0], h, to[1]) if c["layout"] == "hnd" else (to[0], to[1], h)
            src = tuple(x[kept] if torch.is_tensor(x) else x for x in src)
            for plane in (k, v, sums):
                plane[dst] = plane[src]
    return {"kept": None, "lens": None, "k": k[s["n_old"]:], "v": v[s["n_old"]:], "sums": sums[s["n_old"]:]}


def _exact_rope(c, s):
    x = s["qkv"].double()
    if s["bias"] is not None:
        x = x + s["bias"].double()
    x = x.view(c["tokens"], -1, c["dim"])
    half, y = c["rot"] // 2, x.clone()
    for i in range(half):
        cs = s["table"][s["pos"][s["axis"][i]].long(), i].double()[:, None]
        a, b = (i, i + half) if c["style"] == "half" else (2 * i, 2 * i + 1)
        n = c["hq"] + c["hkv"]
        y[:, :n, a] = x[:, :n, a] * cs[..., 0] - x[:, :n, b] * cs[..., 1]
        y[:, :n, b] = x[:, :n, a] * cs[..., 1] + x[:, :n, b] * cs[..., 0]
    out = {"q": y[:, :c["hq"]]}
    page, slot = s["slot"] // c["page"], s["slot"] % c["page"]
    for j, name in enumerate(("k", "v")):
        plane = s[name].double()
        if c["cache"] == "q8_0":
            plane = plane * s[name + "_scale"].double().repeat_interleave(32, -1)
        for h in range(c["hkv"]):
            r = y[:, c["hq"] + j * c["hkv"] + h]
            if c["cache"] == "q8_0":
                blocks = r.reshape(c["tokens"], -1, 32)
                d = (blocks.abs().amax(-1, keepdim=True) / 127).half().double()
                r = (torch.round(blocks / d).clamp(-127, 127) * d).nan_to_num(0.0).flatten(1)
            plane[(page, h, slot) if c["layout"] == "hnd" else (page, slot, h)] = r
        out[name] = plane
    return out
