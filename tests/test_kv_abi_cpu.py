"""Refusals of the paged cache's calls that need no device: the cache's description, types, head
layouts, lengths, budgets and flags are checked before anything else."""
import ctypes
import os
import subprocess
import tempfile

import pytest

import gguf_block_quantized_q4_gb300 as mq
from gguf_block_quantized_q4_gb300 import build as mqbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    mqbuild.build()
    return mq.lib()


def cache(**kw):
    hkv, ps = kw.get("n_kv_heads", 4), kw.get("page_size", 16)
    c = dict(type=mq.F16, n_kv_heads=hkv, head_dim=128, page_size=ps, n_pages=10,
             page_stride=hkv * ps, head_stride=ps, slot_stride=1)
    c.update(kw)
    return mq._KVCacheStruct(**c)


def rope(**kw):
    r = dict(max_pos=100, rot_dim=128, pairs=0, n_axes=1)
    axis = kw.pop("axis", {})
    r.update(kw)
    s = mq._RopeStruct(**r)
    for i, a in axis.items():
        s.axis[i] = a
    return s


def attn(L, c, io=0, S=1, hq=28, max_len=100, pages_ld=7, scale=0.1, window=0, flags=0):
    st = L.mq_attn_decode(ctypes.byref(c) if c is not None else None, io, None, None, None,
                          pages_ld, None, S, hq, max_len, scale, window, flags, None, 0, None)
    return mq.STATUS[st], L.mq_last_error().decode()


def store(L, c, r, io=0, ld=36 * 128, T=1, hq=28):
    st = L.mq_rope_store(ctypes.byref(c), ctypes.byref(r) if r is not None else None, io, None, ld,
                         None, None, None, None, T, hq, None)
    return mq.STATUS[st], L.mq_last_error().decode()


def evict(L, c, S=1, max_len=100, pages_ld=7, new_ld=4, keep=64, sink=0, recent=0):
    st = L.mq_kv_evict(ctypes.byref(c), None, pages_ld, None, S, max_len, None, new_ld, keep, sink,
                       recent, None, None, None)
    return mq.STATUS[st], L.mq_last_error().decode()


@pytest.mark.parametrize("kw,status,word", [
    (dict(type=mq.Q4_K), "MQ_ERR_TYPE", "cache type 12"),
    (dict(type=mq.F32), "MQ_ERR_TYPE", "cache type 0"),
    (dict(head_dim=80), "MQ_ERR_SHAPE", "head_dim=80"),
    (dict(head_dim=0), "MQ_ERR_SHAPE", "head_dim"),
    (dict(n_kv_heads=0, page_stride=1), "MQ_ERR_SHAPE", "n_kv_heads"),
    (dict(page_size=0, page_stride=1), "MQ_ERR_SHAPE", "page_size"),
    (dict(page_size=65537), "MQ_ERR_SHAPE", "page_size"),
    (dict(n_pages=0), "MQ_ERR_SHAPE", "n_pages"),
    (dict(slot_stride=0), "MQ_ERR_SHAPE", "slot_stride"),
    (dict(head_stride=15), "MQ_ERR_SHAPE", "overlap"),
    (dict(page_stride=63), "MQ_ERR_SHAPE", "overlap"),
    (dict(page_stride=1 << 60), "MQ_ERR_SHAPE", "page_stride"),
])
def test_cache_description(L, kw, status, word):
    for got in (attn(L, cache(**kw)), store(L, cache(**kw), rope()), evict(L, cache(**kw))):
        assert got[0] == status and word in got[1], got


def test_layouts_that_keep_rows_apart_pass(L):
    """(the next refusal then is the missing device or pointer)"""
    for kw in (dict(page_stride=64, head_stride=1, slot_stride=4), dict(page_stride=1000),
               dict(page_stride=1, head_stride=10 * 16, slot_stride=10),
               dict(n_kv_heads=1, head_stride=1, page_stride=16)):
        got = attn(L, cache(**kw), hq=4)
        assert got[0] in ("MQ_ERR_STATE", "MQ_ERR_CUDA", "MQ_ERR_ARG") and "stride" not in got[1], got


def test_attention_arguments(L):
    assert attn(L, None)[0] == "MQ_ERR_ARG"
    assert attn(L, cache(), io=mq.Q8_0)[0] == "MQ_ERR_TYPE"
    for hq in (0, 27, 4100):
        assert attn(L, cache(), hq=hq)[0] == "MQ_ERR_SHAPE"
    for kw in (dict(S=-1), dict(S=65536), dict(max_len=0), dict(max_len=113), dict(pages_ld=0),
               dict(window=-1), dict(flags=2), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert attn(L, cache(), **kw)[0] == "MQ_ERR_ARG", kw


def test_rotation_arguments(L):
    assert store(L, cache(), None)[0] == "MQ_ERR_ARG"
    for kw in (dict(rot_dim=0), dict(rot_dim=12), dict(rot_dim=136)):
        assert store(L, cache(), rope(**kw))[0] == "MQ_ERR_SHAPE", kw
    for kw in (dict(n_axes=0), dict(n_axes=5), dict(pairs=2), dict(axis={63: 1}), dict(max_pos=0)):
        assert store(L, cache(), rope(**kw))[0] == "MQ_ERR_ARG", kw
    assert store(L, cache(), rope(), ld=36 * 128 - 4)[0] == "MQ_ERR_SHAPE"
    assert store(L, cache(), rope(), ld=36 * 128 + 2)[0] == "MQ_ERR_ALIGN"
    assert store(L, cache(), rope(), T=-1)[0] == "MQ_ERR_ARG"
    assert store(L, cache(), rope(), io=mq.Q8_0)[0] == "MQ_ERR_TYPE"
    assert store(L, cache(), rope(), hq=30)[0] == "MQ_ERR_SHAPE"


def test_eviction_arguments(L):
    for kw in (dict(keep=0), dict(keep=65), dict(sink=-1), dict(recent=-1), dict(sink=33, recent=32),
               dict(new_ld=0), dict(max_len=113), dict(S=-1), dict(sink=1 << 62, recent=1 << 62)):
        assert evict(L, cache(), **kw)[0] == "MQ_ERR_ARG", kw


def test_structures_match_the_header():
    """The binding's structures have the sizes and offsets of include/mq.h."""
    fields = [("mq_kv_cache", f) for f, _ in mq._KVCacheStruct._fields_]
    fields += [("mq_rope", f) for f, _ in mq._RopeStruct._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "mq.h"\nint main(void) {\n'
    src += '  printf("%zu %zu\\n", sizeof(mq_kv_cache), sizeof(mq_rope));\n'
    src += "".join(f'  printf("%zu\\n", offsetof({t}, {f}));\n' for t, f in fields) + "}\n"
    with tempfile.TemporaryDirectory() as d:
        open(os.path.join(d, "s.c"), "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", os.path.join(d, "s"),
                        os.path.join(d, "s.c")], check=True)
        out = subprocess.run([os.path.join(d, "s")], check=True, capture_output=True, text=True).stdout
    got = [int(x) for x in out.split()]
    assert got[:2] == [ctypes.sizeof(mq._KVCacheStruct), ctypes.sizeof(mq._RopeStruct)]
    assert got[2:] == [getattr({"mq_kv_cache": mq._KVCacheStruct, "mq_rope": mq._RopeStruct}[t],
                               f).offset for t, f in fields]


def test_workspace_constant_matches_the_header():
    src = open(os.path.join(ROOT, "include", "mq.h")).read()
    assert f"#define MQ_ATTN_WS_ZERO {mq.ATTN_WS_ZERO}\n" in src


def test_axes_of_sections():
    assert mq.rope_axes([2, 1, 1]) == [0, 0, 1, 2]
    assert mq.rope_axes([3, 1, 2], weave=True) == [0, 1, 2, 0, 2, 0]
