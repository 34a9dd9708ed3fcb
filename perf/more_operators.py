"""Cases of a decoding step's operators beside those of ``operators.py``: norms of the query and key
heads with the rotation and the store in one pass (``norm``); attention of one new token per
sequence over a paged cache of 4-bit rows (``attn``); sampling of the next token from logits
(``sample``).

``run`` computes an operator in its plain form (elementary torch operations in 32 bits; in 64 where a
sum or a value next to a border decides), or, with ``own`` set, through the package's calls.
``exact`` computes the same outputs in 64 bits, apart from both.

The cache holds rows of ``head_dim`` values per (page, kv head, slot): f16, bf16, Q8_0 (int8 quants
and one f16 scale per 32 values) or Q4_0 (two values a byte: byte j of a block of 32 holds n of value j in
its low and of value 16 + j in its high half, value = scale (n - 8)).  Planes are [page][head][slot]
("hnd") or [page][slot][head] ("nhd").
"""
import math
import random

import torch

own = False

IO = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROW_BYTES = {"f16": lambda d: 2 * d, "bf16": lambda d: 2 * d, "q8_0": lambda d: d + d // 32 * 2,
             "q4_0": lambda d: d // 2 + d // 32 * 2}


def _attn(name, seqs, max_len, hq, hkv, dim, io="f32", page=16, layout="hnd", ragged=True, window=0,
          track=False):
    return {"name": name, "op": "attn", "seqs": seqs, "max_len": max_len, "hq": hq, "hkv": hkv,
            "dim": dim, "cache": "q4_0", "io": io, "page": page, "layout": layout, "ragged": ragged,
            "window": window, "track": track}


def _norm(name, tokens, hq, hkv, dim, cache, io="f32", page=16, layout="hnd", rot=None, axes=1,
          style="half", bias=False, max_pos=32768):
    return {"name": name, "op": "norm", "tokens": tokens, "hq": hq, "hkv": hkv, "dim": dim,
            "cache": cache, "io": io, "page": page, "layout": layout, "rot": rot or dim, "axes": axes,
            "style": style, "bias": bias, "max_pos": max_pos}


def _sample(name, rows, vocab, kind, io="f32", masked=0.0):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "kind": kind, "io": io,
            "masked": masked}


def listed():
    return [
        # the first tokens of one chat on the Qwen2.5-0.5B head layout: latency is all
        _attn("attn 1x37 14/2x64", 1, 37, 14, 2, 64, ragged=False),
        # a small batch of ordinary chats on the Qwen2.5-7B head layout
        _attn("attn 8x1k 28/4x128", 8, 1100, 28, 4, 128),
        # a full serving batch of unlike lengths, one slot of it idle
        _attn("attn 64x8k 28/4x128", 64, 8192, 28, 4, 128, page=32),
        # one long document, bf16 activations: few rows, all of the length to split
        _attn("attn 1x131072 28/4x128 bf16", 1, 131072, 28, 4, 128, io="bf16", page=64, ragged=False),
        # one head per kv head, odd page size, a window that starts inside a page, weights summed
        _attn("attn 5x2k 12/12x96 window track", 5, 2047, 12, 12, 96, io="f16", page=24, window=1000,
              track=True, layout="nhd"),
        # one decode step of a batch of eight into the 4-bit cache
        _norm("norm 8 16/8x128 q4_0", 8, 16, 8, 128, "q4_0"),
        # prefill into the 4-bit cache
        _norm("norm 4096 32/8x128 q4_0", 4096, 32, 8, 128, "q4_0", page=32),
        # a shorter prefill, 16-bit all through: half of each head rotated, neighbouring pairs, two axes
        _norm("norm 1023 12/12x96 bf16 half", 1023, 12, 12, 96, "bf16", io="bf16", rot=48, axes=2,
              style="pairs", bias=True, layout="nhd", page=24),
        # one chat's next token with the usual filters
        _sample("sample 1x151936 top-k top-p", 1, 151936, "usual"),
        # a serving batch whose requests each have settings of their own, some of them greedy
        _sample("sample 64x151936 mixed", 64, 151936, "mixed"),
        # top-p alone over a smaller vocabulary, of which a grammar has masked most
        _sample("sample 16x32003 top-p masked", 16, 32003, "top_p", io="bf16", masked=0.9),
        # many samples at plain temperature with a min-p floor, as in a rollout
        _sample("sample 256x151936 min-p", 256, 151936, "min_p"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "norm", "sample"])
    if op == "sample":
        vocab = _log(rng, 2, 262144)
        rows = max(1, min(_log(rng, 1, 256), 256 * 151936 // vocab // 2))
        return _sample("x", rows, vocab, rng.choice(["usual", "mixed", "top_p", "min_p", "mixed"]),
                       io=rng.choice(["f32", "f32", "f16", "bf16"]), masked=rng.choice([0.0, 0.0, 0.5, 0.99]))
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    hq, hkv = rng.choice([(14, 2), (28, 4), (32, 8), (12, 12), (16, 1), (20, 4), (7, 7), (16, 8)])
    common = dict(page=rng.choice([8, 16, 24, 32, 64, 100]), layout=rng.choice(["hnd", "nhd"]),
                  io=rng.choice(["f32", "f32", "f16", "bf16"]))
    if op == "attn":
        row = 2 * hkv * ROW_BYTES["q4_0"](dim)
        seqs = _log(rng, 1, 64)
        max_len = max(1, min(_log(rng, 1, 131072), int(1.2e8 / (row * seqs))))
        window = 0 if rng.random() < 0.7 else _log(rng, 1, max_len)
        return _attn("x", seqs, max_len, hq, hkv, dim, window=window, track=rng.random() < 0.3, **common)
    tokens = _log(rng, 1, 4096 * 48 * 128 // ((hq + 2 * hkv) * dim) // 2)
    return _norm("x", tokens, hq, hkv, dim, rng.choice(["q4_0", "q4_0", "q8_0", "f16", "bf16"]),
                 rot=rng.choice([dim, dim, dim // 2]), axes=rng.randint(1, 4),
                 style=rng.choice(["half", "pairs"]), bias=rng.random() < 0.5,
                 max_pos=rng.choice([4096, 32768, 131072]), **common)


# ---- inputs -----------------------------------------------------------------------------


def _lens(c):
    """The sequences' lengths: the same for every seed, so that work() knows them."""
    n, top = c["seqs"], c["max_len"]
    if not c["ragged"]:
        return [top] * n
    r = random.Random(n * 1000003 + top)
    lens = [r.randint(1, top) for _ in range(n)]
    lens[r.randrange(n)] = top
    if n >= 5:
        lens[(lens.index(top) + 1) % n] = 0  # an idle slot of the batch
    return lens


def _planes(c, n_pages, g):
    """The cache's planes: k, v and the scales of quantised rows.  Rows that no sequence holds have
    values too."""
    hkv, ps, d, dev = c["hkv"], c["page"], c["dim"], "cuda"
    shape = (n_pages, hkv, ps) if c["layout"] == "hnd" else (n_pages, ps, hkv)
    p = {}
    for name in ("k", "v"):
        if c["cache"] in ("f16", "bf16"):
            p[name] = torch.randn((*shape, d), generator=g, device=dev).to(IO[c["cache"]])
            continue
        if c["cache"] == "q8_0":
            p[name] = torch.randint(-127, 128, (*shape, d), generator=g, device=dev, dtype=torch.int8)
        else:
            p[name] = torch.randint(0, 256, (*shape, d // 2), generator=g, device=dev, dtype=torch.uint8)
        # (the scale of 4 bits has the sign that the block's largest value has not)
        sc = torch.randn((*shape, d // 32), generator=g, device=dev)
        size = 0.01 if c["cache"] == "q8_0" else 0.15
        sc = (sc.abs() + 0.1) * size * (sc.sign() if c["cache"] == "q4_0" else 1.0)
        p[name + "_scale"] = sc.half()
    return p


def _logits(c, g):
    """Logits of a trained model's kind: a wide bulk and a few likely tokens, more of them in some rows;
    tokens that a grammar has masked are -inf or the type's lowest value."""
    n, v = c["rows"], c["vocab"]
    x = torch.randn((n, v), generator=g, device="cuda") * 2.0 - 4.0
    few = min(v, 24)
    at = torch.randint(0, v, (n, few), generator=g, device="cuda")
    up = torch.rand((n, few), generator=g, device="cuda").cumsum(-1) * torch.rand((n, 1), generator=g, device="cuda")
    x.scatter_reduce_(1, at, 5.0 + up, "amax")
    x = x.to(IO[c["io"]])
    if c["masked"]:
        gone = torch.rand((n, v), generator=g, device="cuda") < c["masked"]
        gone[:, v // 2] = False
        low = torch.where(torch.arange(n, device="cuda") % 2 == 0, -math.inf, torch.finfo(IO[c["io"]]).min)
        x = torch.where(gone, low[:, None].to(x.dtype), x)
    return x.contiguous()


def _settings(c, g):
    """Temperature, top-k, top-p and min-p of each row; None: not given."""
    n, v = c["rows"], c["vocab"]
    full = lambda x, dtype=torch.float32: torch.full((n,), x, device="cuda", dtype=dtype)  # noqa: E731
    rand = lambda: torch.rand(n, generator=g, device="cuda")  # noqa: E731
    if c["kind"] == "usual":
        return {"temperature": full(0.7), "top_k": full(40, torch.int32), "top_p": full(0.95), "min_p": None}
    if c["kind"] == "top_p":
        return {"temperature": full(0.8), "top_k": None, "top_p": full(0.9), "min_p": None}
    if c["kind"] == "min_p":
        return {"temperature": full(1.1), "top_k": None, "top_p": None, "min_p": full(0.02)}
    temperature = torch.where(rand() < 0.15, 0.0, 0.3 + rand())
    top_k = torch.where(rand() < 0.4, 0.0, torch.exp(rand() * math.log(min(v, 2000.0)))).int()
    top_p = torch.where(rand() < 0.4, 1.0, rand())
    min_p = torch.where(rand() < 0.6, 0.0, rand() * 0.1)
    return {"temperature": temperature, "top_k": top_k, "top_p": top_p, "min_p": min_p}


def _inputs(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    s = {"case": c}
    if c["op"] == "sample":
        s["logits"] = _logits(c, g)
        s.update(_settings(c, g))
        s["u"] = torch.rand(c["rows"], generator=g, device=dev)
        return s
    hkv, ps, d = c["hkv"], c["page"], c["dim"]
    if c["op"] == "norm":
        n, heads = c["tokens"], c["hq"] + 2 * hkv
        n_pages = -(-n // ps) + 2
        s.update(_planes(c, n_pages, g))
        pages = torch.randperm(n_pages, generator=g, device=dev)
        i = torch.arange(n, device=dev)
        s["slot"] = pages[i // ps] * ps + i % ps
        # heads of unlike sizes, as a product's columns have
        size = torch.exp(torch.randn((1, heads, 1), generator=g, device=dev))
        s["qkv"] = (torch.randn((n, heads, d), generator=g, device=dev) * size).view(n, heads * d).to(IO[c["io"]])
        s["bias"] = torch.randn(heads * d, generator=g, device=dev) * 0.1 if c["bias"] else None
        s["wq"], s["wk"] = (0.5 + torch.rand(d, generator=g, device=dev) for _ in range(2))
        s["eps"] = 1e-6
        half = c["rot"] // 2
        freq = 1e6 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        s["axis"] = [k * c["axes"] // half for k in range(half)]
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
    n_old = sum(need)
    s.update(_planes(c, n_old + 1, g))
    # each sequence's pages lie anywhere in the pool; entries past its length are stale
    order = torch.randperm(n_old, generator=g, device=dev) if n_old else torch.zeros(1, device=dev, dtype=torch.int64)
    first = torch.tensor([sum(need[:k]) for k in range(len(need))], device=dev)
    at = (first[:, None] + torch.arange(used, device=dev)).clamp(max=max(n_old - 1, 0))
    s["pages"] = order[at].int().contiguous()
    s["lens"] = torch.tensor(lens, device=dev, dtype=torch.int32)
    s["q"] = (torch.randn((c["seqs"], c["hq"], d), generator=g, device=dev) * 2).to(IO[c["io"]])
    s["sums"] = torch.rand(s["k"].shape[:-1], generator=g, device=dev) if c["track"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # what a serving program keeps: the cache object, the rotation, the norms, the workspace
        import gguf_block_quantized_q4_gb300 as mq
        mq.init(0)
        if case["op"] == "sample":
            return s
        kind = {"f16": mq.F16, "bf16": mq.BF16, "q8_0": mq.Q8_0, "q4_0": mq.Q4_0}[case["cache"]]
        s["cache"] = mq.KVCache(kind, s["k"], s["v"], s.get("k_scale"), s.get("v_scale"),
                                s.get("sums"), layout=case["layout"])
        if case["op"] == "norm":
            s["rope"] = mq.Rope(s["table"], s["axis"], pairs=case["style"] == "pairs", n_axes=case["axes"])
            s["norm"] = mq.HeadNorm(s["wq"], s["wk"], s["eps"])
        else:
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


def _nibbles(x):
    """The numbers n of 4-bit rows, in the order of their values."""
    x = x.unflatten(-1, (-1, 16))
    return torch.cat([x & 15, x >> 4], -1)


def _seq_rows(c, pages, length):
    """Row index of each (sequence, kv head, position), [S][Hkv][length]."""
    pos = torch.arange(length, device="cuda")
    page = pages.long()[:, pos // c["page"]]
    head = torch.arange(c["hkv"], device="cuda")
    return _row_index(c, page[:, None, :], head[None, :, None], (pos % c["page"])[None, None, :])


def _values4(s, name, rows):
    n = _nibbles(_flat(s, name)[rows]).float() - 8.0
    return (n * _flat(s, name + "_scale")[rows].float()[..., None]).flatten(-2)


def _run_attn(s, c):
    n, d, group = c["max_len"], c["dim"], c["hq"] // c["hkv"]
    rows = _seq_rows(c, s["pages"], n)
    pos, lens = torch.arange(n, device="cuda"), s["lens"].long()[:, None]
    seen = pos < lens
    if c["window"]:
        seen = seen & (pos >= lens - c["window"])
    seen = seen[:, None, None, :]
    q = s["q"].float().view(c["seqs"], c["hkv"], group, d)
    w = torch.matmul(q, _values4(s, "k", rows).transpose(-1, -2)) * (1.0 / math.sqrt(d))
    w = torch.where(seen, w, -math.inf)
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(-1, keepdim=True)
    w = w / torch.where(total == 0, 1.0, total)
    o = torch.matmul(w, _values4(s, "v", rows)).to(s["q"].dtype).view(c["seqs"], c["hq"], d)
    if not c["track"]:
        return {"o": o}
    # a row belongs to one sequence: what the others' stale page entries name gets nothing
    s["sums"].view(-1).index_add_(0, rows.flatten(), w.sum(2).flatten())
    return {"o": o, "sums": s["sums"]}


def _run_norm(s, c):
    n, d, half, nq = c["tokens"], c["dim"], c["rot"] // 2, c["hq"]
    x = s["qkv"].float()
    if s["bias"] is not None:
        x = x + s["bias"]
    x = x.view(n, -1, d)
    normed, v = x[:, :nq + c["hkv"]], x[:, nq + c["hkv"]:]
    # (the mean and its root in 64 bits: a stored row is rounded to a few, and a border decides)
    by = torch.rsqrt((normed.double() ** 2).mean(-1, keepdim=True) + s["eps"]).float()
    normed = normed * by
    normed = torch.cat([normed[:, :nq] * s["wq"], normed[:, nq:] * s["wk"]], 1)
    pair = torch.arange(half, device="cuda")
    at = s["table"][s["pos"].long()[torch.tensor(s["axis"], device="cuda")].T, pair]  # [n][half][2]
    cos, sin = at[:, None, :, 0], at[:, None, :, 1]
    rot, rest = normed[..., :2 * half], normed[..., 2 * half:]
    if c["style"] == "half":
        a, b = rot[..., :half], rot[..., half:]
        rot = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    turned = torch.cat([rot, rest], -1)
    q = turned[:, :nq].to(s["qkv"].dtype)
    slot = s["slot"][:, None]
    rows = _row_index(c, slot // c["page"], torch.arange(c["hkv"], device="cuda"), slot % c["page"])
    for name, y in (("k", turned[:, nq:]), ("v", v)):
        if c["cache"] in ("f16", "bf16"):
            _flat(s, name)[rows] = y.to(s[name].dtype)
            continue
        blocks = y.unflatten(-1, (-1, 32))
        most, least = blocks.amax(-1), blocks.amin(-1)
        big = torch.where(most >= -least, most, least)
        if c["cache"] == "q8_0":
            sc = (big.abs() / torch.full((), 127.0, device="cuda")).half()
        else:
            sc = (big / torch.full((), -8.0, device="cuda")).half()
        by = sc.float()[..., None]
        quants = torch.where(by == 0, 0.0, torch.round(blocks / by))
        if c["cache"] == "q8_0":
            _flat(s, name)[rows] = quants.clamp(-127, 127).to(torch.int8).flatten(-2)
        else:
            quants = (quants + 8).clamp(0, 15).to(torch.uint8)
            _flat(s, name)[rows] = (quants[..., :16] | quants[..., 16:] << 4).flatten(-2)
        _flat(s, name + "_scale")[rows] = sc
    return {"q": q, "k": _shown(s, c, "k"), "v": _shown(s, c, "v")}


def _shown(s, c, name):
    """A plane as the values it stands for."""
    if c["cache"] in ("f16", "bf16"):
        return s[name]
    n = s[name].unflatten(-1, (-1, 32)) if c["cache"] == "q8_0" else _nibbles(s[name]).to(torch.int8) - 8
    return n * s[name + "_scale"][..., None]  # f16


def _run_sample(s, c):
    n, v = c["rows"], c["vocab"]
    x = s["logits"].float()
    x = torch.where(x.isnan(), -math.inf, x)
    order = torch.sort(x, dim=-1, descending=True, stable=True)  # equal ones by their index
    top = order.values[:, :1]
    greedy = ~(s["temperature"] > 0)[:, None]
    # (weights and sums in 64 bits: the token is where a running sum passes a border)
    by = torch.where(greedy, 1.0, s["temperature"][:, None]).double()
    diff = torch.where(order.values == top, 0.0, order.values.double() - top.double())
    w = torch.exp(diff / by)
    place = torch.arange(v, device="cuda")
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        w = torch.where((k > 0) & (place >= k), 0.0, w)
    if s["top_p"] is not None:
        p = s["top_p"][:, None].double()
        before = w.cumsum(-1) - w  # kept while what stands before does not reach the share
        w = torch.where((p < 1) & (place > 0) & (before >= p * w.sum(-1, keepdim=True)), 0.0, w)
    if s["min_p"] is not None:
        w = torch.where(w < s["min_p"][:, None].double().clamp(max=1.0), 0.0, w)
    w = torch.where(greedy, (place == 0).double(), w)
    total = w.sum(-1, keepdim=True)
    w = torch.zeros_like(w).scatter_(1, order.indices, w)  # in the tokens' order
    run_ = w.cumsum(-1)
    token = (run_ > s["u"][:, None].double() * total).int().argmax(-1)
    p = torch.gather(w, 1, token[:, None]) / total
    return {"token": token.int(), "logprob": torch.log(p)[:, 0].float()}


def _run_own(s, c):
    import gguf_block_quantized_q4_gb300 as mq
    if c["op"] == "attn":
        o = mq.attn_decode(s["cache"], s["q"], s["pages"], s["lens"], c["max_len"], window=c["window"],
                           track=c["track"], ws=s["ws"])
        return {"o": o, "sums": s["sums"]} if c["track"] else {"o": o}
    if c["op"] == "norm":
        q = mq.rope_store(s["cache"], s["rope"], s["qkv"], s["pos"], s["slot"], c["hq"], bias=s["bias"],
                          norm=s["norm"])
        return {"q": q, "k": _shown(s, c, "k"), "v": _shown(s, c, "v")}
    token, logprob = mq.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                               top_p=s["top_p"], min_p=s["min_p"])
    return {"token": token, "logprob": logprob}


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    return {"attn": _run_attn, "norm": _run_norm, "sample": _run_sample}[c["op"]](state, c)


def work(case):
    c = case
    size = torch.empty(0, dtype=IO[c["io"]]).element_size()
    if c["op"] == "sample":
        return {"bytes": c["rows"] * (c["vocab"] * size + 28), "flops": c["rows"] * c["vocab"]}
    row = ROW_BYTES[c["cache"]](c["dim"])
    if c["op"] == "norm":
        n, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["dim"]
        return {"bytes": n * ((2 * hq + 2 * hkv) * d * size + 2 * hkv * row + c["rot"] * 4 + c["axes"] * 4 + 8),
                "flops": n * (hq + hkv) * (c["rot"] * 3 + d * 4)}
    keys = sum(min(n, c["window"]) if c["window"] else n for n in _lens(c))
    return {"bytes": keys * c["hkv"] * (2 * row + (8 if c["track"] else 0)) + 2 * c["seqs"] * c["hq"] * c["dim"] * size,
            "flops": 4 * keys * c["hq"] * c["dim"]}


# ---- 64 bits --------------------------------------------------------------------------------


def _plane64(s, c, name):
    """A plane's values in 64 bits, as it is laid out."""
    if c["cache"] in ("f16", "bf16"):
        return s[name].double()
    scale = s[name + "_scale"].double().repeat_interleave(32, -1)
    if c["cache"] == "q8_0":
        return s[name].double() * scale
    x = s[name].reshape(*s[name].shape[:-1], -1, 16).int()
    return torch.stack([x % 16, x // 16], -2).flatten(-3).double().sub(8) * scale


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "norm":
        return _exact_norm(c, s)
    if c["op"] == "sample":
        return _exact_sample(c, s)
    group = c["hq"] // c["hkv"]
    o = torch.zeros((c["seqs"], c["hq"], c["dim"]), dtype=torch.float64, device="cuda")
    sums = s["sums"].double() if c["track"] else None
    k64, v64 = _plane64(s, c, "k"), _plane64(s, c, "v")
    for b, n in enumerate(_lens(c)):
        lo = max(0, n - c["window"]) if c["window"] else 0
        pos = torch.arange(lo, n, device="cuda")
        page, slot = s["pages"][b].long()[pos // c["page"]], pos % c["page"]
        for h in range(c["hkv"] if n else 0):
            at = (page, h, slot) if c["layout"] == "hnd" else (page, slot, h)
            q = s["q"][b, h * group:(h + 1) * group].double()
            w = torch.softmax(q @ k64[at].T / math.sqrt(c["dim"]), -1)
            o[b, h * group:(h + 1) * group] = w @ v64[at]
            if c["track"]:
                sums[at] += w.sum(0)
    return {"o": o, "sums": sums} if c["track"] else {"o": o}


def _exact_norm(c, s):
    n, nq, d, half = c["tokens"], c["hq"], c["dim"], c["rot"] // 2
    x = s["qkv"].double()
    if s["bias"] is not None:
        x = x + s["bias"].double()
    x = x.view(n, -1, d)
    y = x.clone()
    for h in range(nq + c["hkv"]):
        w = (s["wq"] if h < nq else s["wk"]).double()
        y[:, h] = x[:, h] * w / torch.sqrt((x[:, h] * x[:, h]).sum(-1, keepdim=True) / d + s["eps"])
    z, m = y.clone(), nq + c["hkv"]
    for i in range(half):
        cs = s["table"][s["pos"][s["axis"][i]].long(), i].double()[:, None]
        a, b = (i, i + half) if c["style"] == "half" else (2 * i, 2 * i + 1)
        z[:, :m, a] = y[:, :m, a] * cs[..., 0] - y[:, :m, b] * cs[..., 1]
        z[:, :m, b] = y[:, :m, a] * cs[..., 1] + y[:, :m, b] * cs[..., 0]
    out = {"q": z[:, :nq]}
    page, slot = s["slot"] // c["page"], s["slot"] % c["page"]
    for j, name in enumerate(("k", "v")):
        plane = _plane64(s, c, name)
        for h in range(c["hkv"]):
            r = z[:, nq + j * c["hkv"] + h]
            if c["cache"] in ("q8_0", "q4_0"):
                blocks = r.reshape(n, -1, 32)
                if c["cache"] == "q8_0":
                    dd = (blocks.abs().amax(-1, keepdim=True) / 127).half().double()
                    lo, hi = -127, 127
                else:
                    at = (blocks.abs() + (blocks > 0) * 1e-300).argmax(-1, keepdim=True)
                    dd = (blocks.gather(-1, at) / -8).half().double()
                    lo, hi = -8, 7
                r = (torch.round(blocks / dd).clamp(lo, hi) * dd).nan_to_num(0.0).flatten(1)
            plane[(page, h, slot) if c["layout"] == "hnd" else (page, slot, h)] = r
        out[name] = plane
    return out


def _exact_sample(c, s):
    """Row by row: the tokens that stay as a set, then the running sum over them."""
    token = torch.zeros(c["rows"], dtype=torch.int32, device="cuda")
    logprob = torch.zeros(c["rows"], dtype=torch.float64, device="cuda")
    given = {k: s[k].tolist() if s[k] is not None else None for k in ("temperature", "top_k", "top_p", "min_p")}
    for r, u in enumerate(s["u"].tolist()):
        x = s["logits"][r].double()
        x = torch.where(x.isnan(), -math.inf, x)
        t = given["temperature"][r]
        if t <= 0:
            token[r] = int((x == x.max()).nonzero()[0])
            continue
        w = torch.exp((x - x.max()) / t)
        left = torch.argsort(-x, stable=True)
        if given["top_k"] and 0 < given["top_k"][r] < len(left):
            left = left[:given["top_k"][r]]
        if given["top_p"] and given["top_p"][r] < 1:
            upto = torch.cumsum(w[left], 0)
            left = left[:int((upto < given["top_p"][r] * upto[-1]).sum()) + 1]
        if given["min_p"]:
            left = left[w[left] >= min(given["min_p"][r], 1.0)]
        left = left.sort().values
        upto = torch.cumsum(w[left], 0)
        i = left[int((upto <= u * upto[-1]).sum())]
        token[r], logprob[r] = int(i), torch.log(w[i] / upto[-1])
    return {"token": token, "logprob": logprob}
