"""mq_sample's kernel on the host, one fiber per thread (threads/device.h): the order in which threads go on is the
caller's."""
import ctypes
import os
import subprocess

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gguf_block_quantized_q4_gb300", "csrc")
HERE = os.path.join(ROOT, "tests", "threads")

# what the host's compiler cannot take, each once in the file
REPLACED = [
    ('#include "kv.cuh"\n', ""),
    ("extern __shared__ __align__(16) uint32_t totals[];", "uint32_t *const totals = static_cast<uint32_t *>(threads::dynamic());"),
    ("__shared__ __align__(16) Shared sh;", "Shared &sh = threads::shared<Shared>();"),
    ('asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(f));', "r = exp2f(f);"),
]
ORDERS = [(0, 0), (1, 0), *((which, seed) for which in (2, 3, 4, 5) for seed in (1, 2, 3))]


def build(folder):
    text = open(os.path.join(CSRC, "sample.cu")).read()
    for old, new in REPLACED:
        assert text.count(old) == 1, old
        text = text.replace(old, new)
    for name, body in (("sample.cu", text), ("mq_common.cuh", ""), ("cooperative_groups.h", ""),
                       ("sample.cuh", open(os.path.join(CSRC, "sample.cuh")).read())):
        with open(os.path.join(folder, name), "w") as f:
            f.write(body)
    lib = os.path.join(folder, "sample_host.so")
    subprocess.run(["g++", "-O2", "-U_FORTIFY_SOURCE", "-std=c++17", "-shared", "-fPIC", "-ffp-contract=off", "-I", HERE, "-I", folder,
                    f'-DSAMPLE_CU="{os.path.join(folder, "sample.cu")}"', os.path.join(HERE, "sample_host.cpp"), "-o", lib],
                   check=True, capture_output=True, text=True)
    library = ctypes.CDLL(lib)
    f = library.sample_host
    f.library = library
    p, i64 = ctypes.c_void_p, ctypes.c_int64
    f.argtypes = [ctypes.c_int, p, i64, i64, i64, p, p, p, p, p, p, p, p, ctypes.c_int, ctypes.c_uint]
    return f


def sample(f, logits, u, ranks_log=1, order=(0, 0), **given):
    """logits f32 [B][V], u and given (temperature, top_k, top_p, min_p) one per row; 2^ranks_log blocks a row."""
    B, V = logits.shape
    kept = {k: np.ascontiguousarray(v, np.int32 if k == "top_k" else np.float32) for k, v in given.items()}
    u = np.ascontiguousarray(u, np.float32)
    token, logprob = np.full(B, -7, np.int32), np.full(B, np.nan, np.float32)
    clusters = (ctypes.c_int * 5)(*(1 << 20 if i <= ranks_log else 0 for i in range(5)))

    def at(x):
        return None if x is None else x.ctypes.data
    assert logits.dtype == np.float32 and logits.strides[1] == 4
    assert f(0, at(logits), logits.strides[0] // 4 if B > 1 else V, B, V, at(u), *(at(kept.get(k)) for k in ("temperature", "top_k", "top_p", "min_p")),
             at(token), at(logprob), ctypes.addressof(clusters), *order) == 0
    return token, logprob
