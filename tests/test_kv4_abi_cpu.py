"""Refusals and structures of the 4-bit cache and of the heads' norms that need no device."""
import ctypes
import os
import subprocess
import tempfile

import pytest

import gguf_block_quantized_q4_gb300 as mq
from tests.test_kv_abi_cpu import L, ROOT, attn, cache, evict, rope, store  # noqa: F401


def norm_store(L, c, r, norm, io=0, ld=36 * 128, T=1, hq=28):
    st = L.mq_norm_rope_store(ctypes.byref(c), ctypes.byref(r), ctypes.byref(norm) if norm is not None else None,
                              io, None, ld, None, None, None, None, T, hq, None)
    return mq.STATUS[st], L.mq_last_error().decode()


def test_a_q4_0_cache_is_described(L):
    """(the next refusal is the missing device or pointer)"""
    c = cache(type=mq.Q4_0)
    norm = mq._HeadNormStruct(None, None, 1e-6)
    for got in (attn(L, c), store(L, c, rope()), evict(L, c), norm_store(L, c, rope(), norm)):
        assert got[0] in ("MQ_ERR_STATE", "MQ_ERR_CUDA", "MQ_ERR_ARG") and "type" not in got[1], got


@pytest.mark.parametrize("eps", [0.0, -1e-6, 1e-31, 2e30, float("nan"), float("inf")])
def test_epsilon_is_refused(L, eps):
    got = norm_store(L, cache(), rope(), mq._HeadNormStruct(None, None, eps))
    assert got[0] == "MQ_ERR_ARG" and "norm.eps" in got[1], got


def test_norm_arguments(L):
    assert norm_store(L, cache(), rope(), None) == ("MQ_ERR_ARG", "mq_norm_rope_store: norm is NULL")
    norm = mq._HeadNormStruct(None, None, 1e-6)
    # what mq_rope_store refuses, under this call's name
    for kw, status in ((dict(ld=36 * 128 - 4), "MQ_ERR_SHAPE"), (dict(ld=36 * 128 + 2), "MQ_ERR_ALIGN"),
                       (dict(T=-1), "MQ_ERR_ARG"), (dict(io=mq.Q8_0), "MQ_ERR_TYPE"), (dict(hq=30), "MQ_ERR_SHAPE")):
        got = norm_store(L, cache(), rope(), norm, **kw)
        assert got[0] == status and got[1].startswith("mq_norm_rope_store: "), got


def test_queries_over_the_norms_weights_are_refused(L):
    """(other blocks still read them)"""
    c, r = cache(), rope()
    for q, k in ((4096 + 28 * 128 * 4 - 4, 1 << 20), (1 << 20, 4096 - 508)):
        norm = mq._HeadNormStruct(q, k, 1e-6)
        st = L.mq_norm_rope_store(ctypes.byref(c), ctypes.byref(r), ctypes.byref(norm), 0, ctypes.c_void_p(1 << 30), 36 * 128, None, None,
                                  None, ctypes.c_void_p(4096), 1, 28, None)
        assert mq.STATUS[st] == "MQ_ERR_ARG" and "overlaps the norms" in L.mq_last_error().decode()


def test_norm_structure_matches_the_header():
    names = [f for f, _ in mq._HeadNormStruct._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "mq.h"\nint main(void) {\n'
    src += '  printf("%zu\\n", sizeof(mq_head_norm));\n'
    src += "".join(f'  printf("%zu\\n", offsetof(mq_head_norm, {f}));\n' for f in names) + "}\n"
    with tempfile.TemporaryDirectory() as d:
        open(os.path.join(d, "s.c"), "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", os.path.join(d, "s"),
                        os.path.join(d, "s.c")], check=True)
        out = subprocess.run([os.path.join(d, "s")], check=True, capture_output=True, text=True).stdout
    assert [int(x) for x in out.split()] == [ctypes.sizeof(mq._HeadNormStruct)] + [
        getattr(mq._HeadNormStruct, f).offset for f in names]
