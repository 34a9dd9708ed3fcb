"""Python binding of libmq, the GB300 GGUF block-quantised matmul library, with the paged
key-value cache and decode attention between its products.

Argument marshalling only: every step of the computation runs in libmq's CUDA
kernels.  PyTorch provides device memory and streams.  The C ABI
(include/mq.h) is exposed twice:

* ``lib()``: the raw ctypes library with the exact C names and signatures
  (``mq_matvec`` etc.), taking plain pointers and sizes;
* thin wrappers with the same names minus the ``mq_`` prefix that take torch
  tensors, read their data pointers and the current CUDA stream, and raise
  :class:`MQError` on a non-OK status.

There is no fallback: if libmq.so is missing or fails to load, importing the
wrappers raises.
"""
from __future__ import annotations

import ctypes
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmq.so")

Q4_0, Q4_1, Q5_0, Q5_1, Q8_0, Q4_K, Q5_K, Q6_K = 2, 3, 6, 7, 8, 12, 13, 14
F16, BF16 = 1, 30  # unquantised weights: decode matvec only
F32 = 0  # activations of rope_store / attn_decode; not a weight type
ATTN_TRACK = 1
REG_DEFAULT, REG_NO_MMQ_PLANE, REG_MMQ_FROM_DECODE_PLANE = 0, 1, 2
# (elements, bytes) per block; f16 / bf16 rows count in units of 32 elements (K % 32 == 0)
BLOCK = {Q4_0: (32, 18), Q4_1: (32, 20), Q5_0: (32, 22), Q5_1: (32, 24), Q8_0: (32, 34),
         Q4_K: (256, 144), Q5_K: (256, 176), Q6_K: (256, 210), F16: (32, 64), BF16: (32, 64)}

STATUS = ["MQ_OK", "MQ_ERR_ARG", "MQ_ERR_TYPE", "MQ_ERR_SHAPE", "MQ_ERR_PAYLOAD",
          "MQ_ERR_ALIGN", "MQ_ERR_CUDA", "MQ_ERR_OOM", "MQ_ERR_LAUNCH", "MQ_ERR_TIMEOUT",
          "MQ_ERR_STATE", "MQ_ERR_INDEX"]

# The C ABI: name -> (restype, argtypes)
_P, _I64, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
_ST = ctypes.c_int
ABI = {
    "mq_init": (_ST, [ctypes.c_int]),
    "mq_register_weight": (_ST, [ctypes.c_int, _P, _SZ, _I64, _I64, ctypes.c_uint32,
                                 ctypes.POINTER(_P)]),
    "mq_weight_free": (_ST, [_P]),
    "mq_weight_info": (_ST, [_P, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(_I64),
                             ctypes.POINTER(_I64), ctypes.POINTER(_SZ)]),
    "mq_weight_unpack": (_ST, [_P, _P, _SZ]),
    "mq_matvec": (_ST, [ctypes.c_int, _P, _P, _P, _I64, _I64, ctypes.c_int, _P]),
    "mq_act_bytes": (_SZ, [_I64, _I64]),
    "mq_quantize_act": (_ST, [_P, _P, _I64, _I64, _P]),
    "mq_mmq": (_ST, [ctypes.c_int, _P, _P, _P, _I64, _I64, _I64, _P]),
    "mq_mmq_fused": (_ST, [ctypes.c_int, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "mq_mmq_fused_static": (_ST, [ctypes.c_int, _P, _P, _P, _I64, _I64, _I64, _P]),
    "mq_matvec_host": (_ST, [ctypes.c_int, _P, _P, _P, _P, _P, _I64, _I64, ctypes.c_int, _P]),
    "mq_mmq_host": (_ST, [ctypes.c_int, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "mq_mmq_blockdots": (_ST, [ctypes.c_int, _P, _P, _P, _I64, _I64, _I64, _P]),
    "mq_register_ffn_gu": (_ST, [ctypes.c_int, _P, _P, _SZ, _I64, _I64, ctypes.c_uint32,
                                 ctypes.POINTER(_P)]),
    "mq_ffn_gu_matvec": (_ST, [ctypes.c_int, _P, _P, _P, _I64, _I64, ctypes.c_int, _P]),
    "mq_ffn_gu_mmq": (_ST, [ctypes.c_int, _P, _P, _P, _I64, _I64, _I64, _P]),
    "mq_rope_store": (_ST, [_P, _P, ctypes.c_int, _P, _I64, _P, _P, _P, _P, _I64, ctypes.c_int,
                            _P]),
    "mq_attn_workspace_bytes": (_SZ, [_P, _I64, ctypes.c_int, _I64, ctypes.c_uint32]),
    "mq_attn_decode": (_ST, [_P, ctypes.c_int, _P, _P, _P, _I64, _P, _I64, ctypes.c_int, _I64,
                             ctypes.c_float, _I64, ctypes.c_uint32, _P, _SZ, _P]),
    "mq_kv_evict": (_ST, [_P, _P, _I64, _P, _I64, _I64, _P, _I64, _I64, _I64, _I64, _P, _P, _P]),
    "mq_stream_status": (_ST, [_P]),
    "mq_last_error": (ctypes.c_char_p, []),
    "mq_status_name": (ctypes.c_char_p, [ctypes.c_int]),
}

_lib = None


class MQError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        self.name = STATUS[status] if 0 <= status < len(STATUS) else f"status {status}"
        super().__init__(f"{self.name}: {message}")


def lib():
    """Load libmq.so (built in-tree by build.py) and declare the C ABI."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m gguf_block_quantized_q4_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in ABI.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        raise MQError(status, lib().mq_last_error().decode(errors="replace"))


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def init(device: int = 0):
    _check(lib().mq_init(device))


class Weight:
    """A registered weight (library-owned device planes)."""

    def __init__(self, qtype: int, data, N: int, K: int, flags: int = REG_DEFAULT):
        import numpy as np
        buf = np.ascontiguousarray(np.frombuffer(memoryview(data), dtype=np.uint8)
                                   if not isinstance(data, np.ndarray) else data.view(np.uint8))
        h = ctypes.c_void_p()
        _check(lib().mq_register_weight(qtype, buf.ctypes.data_as(ctypes.c_void_p), buf.nbytes,
                                        N, K, flags, ctypes.byref(h)))
        self.handle = h
        self.qtype, self.N, self.K = qtype, N, K
        self.nbytes = buf.nbytes

    def info(self):
        t, n, k, b = ctypes.c_int(), _I64(), _I64(), _SZ()
        _check(lib().mq_weight_info(self.handle, ctypes.byref(t), ctypes.byref(n),
                                    ctypes.byref(k), ctypes.byref(b)))
        return t.value, n.value, k.value, b.value

    def unpack(self):
        import numpy as np
        out = np.empty(self.nbytes, dtype=np.uint8)
        _check(lib().mq_weight_unpack(self.handle, out.ctypes.data_as(ctypes.c_void_p),
                                      out.nbytes))
        return out

    def free(self):
        if self.handle:
            _free_deferred()
            _check(lib().mq_weight_free(self.handle))
            self.handle = None

    def __del__(self):
        # mq_weight_free synchronises the device, which would invalidate a stream capture in
        # progress (a weight kept alive by a reference cycle is collected whenever the
        # garbage collector runs): during a capture the handle is kept and freed later
        try:
            if getattr(self, "handle", None) and _lib is not None:
                if _capturing():
                    _deferred_frees.append(self.handle)
                else:
                    _free_deferred()
                    _lib.mq_weight_free(self.handle)
        except Exception:
            pass


_deferred_frees = []


def _capturing() -> bool:
    torch = sys.modules.get("torch")
    try:
        return bool(torch is not None and torch.cuda.is_available()
                    and torch.cuda.is_current_stream_capturing())
    except Exception:
        return False


def _free_deferred():
    """Free the weights whose collection fell inside a stream capture (none while one is
    still in progress)."""
    if not _deferred_frees or _capturing():
        return
    while _deferred_frees:
        _lib.mq_weight_free(_deferred_frees.pop())


def register_weight(qtype, data, N, K, flags=REG_DEFAULT) -> Weight:
    _free_deferred()
    return Weight(qtype, data, N, K, flags)


class FfnGuWeight(Weight):
    """A fused gate/up weight (mq_register_ffn_gu): N gate rows and N up rows."""

    def __init__(self, qtype: int, gate, up, N: int, K: int, flags: int = REG_DEFAULT):
        import numpy as np

        def as_u8(d):
            return np.ascontiguousarray(np.frombuffer(memoryview(d), dtype=np.uint8)
                                        if not isinstance(d, np.ndarray) else d.view(np.uint8))
        g, u = as_u8(gate), as_u8(up)
        if g.nbytes != u.nbytes:
            raise ValueError("gate and up payloads differ in size")
        h = ctypes.c_void_p()
        _check(lib().mq_register_ffn_gu(qtype, g.ctypes.data_as(ctypes.c_void_p),
                                        u.ctypes.data_as(ctypes.c_void_p), g.nbytes, N, K, flags,
                                        ctypes.byref(h)))
        self.handle = h
        self.qtype, self.N, self.K = qtype, N, K
        self.nbytes = 2 * g.nbytes


def register_ffn_gu(qtype, gate, up, N, K, flags=REG_DEFAULT) -> FfnGuWeight:
    _free_deferred()
    return FfnGuWeight(qtype, gate, up, N, K, flags)


# What a call makes for itself (outputs, buffers, a workspace, a copy of a strided input) it makes and
# clears under `stream`, the stream that its kernels run on (default: the current one): memory of
# the current stream's pool could have work of that stream pending, and would go back to it while the
# kernels still run.


def ffn_gu_matvec(W: FfnGuWeight, x, h=None, stream=None):
    """h[B][N] = silu(W_gate x) * (W_up x) (x: CUDA f32 [B][K] or [K])."""
    import torch
    if stream is not None and (h is None or not x.is_contiguous()):
        with torch.cuda.stream(stream):
            return ffn_gu_matvec(W, x, h)
    x2 = x.reshape(-1, W.K)
    B = x2.shape[0]
    if h is None:
        h = torch.empty((B, W.N), dtype=torch.float32, device=x.device)
    _check(lib().mq_ffn_gu_matvec(W.qtype, W.handle, _ptr(x2), _ptr(h), W.N, W.K, B,
                                  _stream(stream)))
    return h


def ffn_gu_mmq(W: FfnGuWeight, xq, M: int, h=None, stream=None):
    """h[M][N] = silu(W_gate a) * (W_up a) for the quantised activations xq."""
    import torch
    if stream is not None and h is None:
        with torch.cuda.stream(stream):
            return ffn_gu_mmq(W, xq, M)
    if h is None:
        h = torch.empty((M, W.N), dtype=torch.float32, device=xq.device)
    _check(lib().mq_ffn_gu_mmq(W.qtype, W.handle, _ptr(xq), _ptr(h), M, W.N, W.K,
                               _stream(stream)))
    return h


def matvec(W: Weight, x, y=None, stream=None):
    """y[B][N] = dequant(W) @ x[B][K]^T (x: CUDA f32 [B][K] or [K])."""
    import torch
    if stream is not None and (y is None or not x.is_contiguous()):
        with torch.cuda.stream(stream):
            return matvec(W, x, y)
    x2 = x.reshape(-1, W.K)
    B = x2.shape[0]
    if y is None:
        y = torch.empty((B, W.N), dtype=torch.float32, device=x.device)
    _check(lib().mq_matvec(W.qtype, W.handle, _ptr(x2), _ptr(y), W.N, W.K, B, _stream(stream)))
    return y


def act_bytes(M: int, K: int) -> int:
    return lib().mq_act_bytes(M, K)


def min_ld(nb: int) -> int:
    """Row stride (f16 elements) of the min-term operand: 3*nb rounded up to 8."""
    return (3 * nb + 7) // 8 * 8


def act_layout(M: int, K: int):
    """Byte offsets of the xq sections (see mq_act_bytes in mq.h)."""
    def al(v):
        return (v + 255) & ~255
    mt = (M + 127) // 128 * 128
    nb = K // 32
    o = {"qs": 0}
    o["scale"] = al(o["qs"] + M * K)
    o["bsum"] = al(o["scale"] + M * nb * 4)
    o["op"] = al(o["bsum"] + M * nb * 4)
    o["scaleT"] = al(o["op"] + M * K * 2)
    o["minT"] = al(o["scaleT"] + mt * nb * 4)
    o["amin"] = al(o["minT"] + mt * nb * 4)
    o["urow"] = al(o["amin"] + M * min_ld(nb) * 2)
    o["sync"] = al(o["urow"] + mt * 4)
    o["total"] = al(o["sync"] + 8)
    o["mt"] = mt
    return o


def act_views(xq, M: int, K: int):
    """Views (qs int8 [M][K], scale f32 [M][K/32], bsum int32 [M][K/32], op f16 [M][K])
    of an xq buffer, following the layout documented in mq.h."""
    import torch
    o = act_layout(M, K)
    nb = K // 32
    qs = xq[o["qs"]:o["qs"] + M * K].view(torch.int8).view(M, K)
    sc = xq[o["scale"]:o["scale"] + M * nb * 4].view(torch.float32).view(M, nb)
    bs = xq[o["bsum"]:o["bsum"] + M * nb * 4].view(torch.int32).view(M, nb)
    op = xq[o["op"]:o["op"] + M * K * 2].view(torch.float16).view(M, K)
    return qs, sc, bs, op


def act_views_transposed(xq, M: int, K: int):
    """Views (scaleT f32 [K/32][M], minT f32 [K/32][M]) of the transposed sections."""
    import torch
    o = act_layout(M, K)
    nb, mt = K // 32, o["mt"]
    st = xq[o["scaleT"]:o["scaleT"] + mt * nb * 4].view(torch.float32).view(nb, mt)[:, :M]
    tt = xq[o["minT"]:o["minT"] + mt * nb * 4].view(torch.float32).view(nb, mt)[:, :M]
    return st, tt


def act_views_min(xq, M: int, K: int):
    """Views (amin f16 [M][3*K/32], urow f32 [M]) of the min-term operand sections."""
    import torch
    o = act_layout(M, K)
    nb = K // 32
    ld = min_ld(nb)
    am = xq[o["amin"]:o["amin"] + M * ld * 2].view(torch.float16).view(M, ld)[:, :3 * nb]
    ur = xq[o["urow"]:o["urow"] + M * 4].view(torch.float32)
    return am, ur


def quantize_act(x, xq=None, stream=None):
    """Quantise CUDA f32 x[M][K]; returns the uint8 xq buffer."""
    import torch
    if stream is not None and xq is None:
        with torch.cuda.stream(stream):
            return quantize_act(x)
    M, K = x.shape
    if xq is None:
        xq = torch.empty(act_bytes(M, K), dtype=torch.uint8, device=x.device)
    _check(lib().mq_quantize_act(_ptr(x), _ptr(xq), M, K, _stream(stream)))
    return xq


def mmq(W: Weight, xq, M: int, y=None, stream=None):
    import torch
    if stream is not None and y is None:
        with torch.cuda.stream(stream):
            return mmq(W, xq, M)
    if y is None:
        y = torch.empty((M, W.N), dtype=torch.float32, device=xq.device)
    _check(lib().mq_mmq(W.qtype, W.handle, _ptr(xq), _ptr(y), M, W.N, W.K, _stream(stream)))
    return y


def act_buffer(M: int, K: int, device=None):
    """An xq buffer of mq_act_bytes(M, K) bytes, zero-filled (so the fused call's barrier
    count starts at zero), ready for mmq_fused as well as quantize_act."""
    import torch
    return torch.zeros(act_bytes(M, K), dtype=torch.uint8, device=device or "cuda")


def mmq_fused(W: Weight, x, xq=None, y=None, stream=None):
    """Quantise x (f32 [M][K] on the device) into xq and run the MMQ, in one kernel.
    Returns (y, xq); xq then holds what quantize_act writes."""
    import torch
    if stream is not None and (xq is None or y is None):
        with torch.cuda.stream(stream):
            return mmq_fused(W, x, xq, y)
    M = x.shape[0]
    if xq is None:
        xq = act_buffer(M, W.K, x.device)
    if y is None:
        y = torch.empty((M, W.N), dtype=torch.float32, device=x.device)
    _check(lib().mq_mmq_fused(W.qtype, W.handle, _ptr(x), _ptr(xq), _ptr(y), M, W.N, W.K,
                              _stream(stream)))
    return y, xq


def matvec_host(W: Weight, x_host, y_host, x_dev, y_dev, stream=None):
    """Decode matvec from host buffers (torch CPU tensors x_host [B][K], y_host [B][N]), all
    enqueued on the stream by one C call.  Pinned, 16-byte aligned host tensors are read and
    written by the kernels directly (x through x_dev, y straight into y_host); others are
    copied through x_dev / y_dev.  y_host is complete when the stream is."""
    B = x_host.shape[0]
    _check(lib().mq_matvec_host(W.qtype, W.handle, _ptr(x_host), _ptr(y_host), _ptr(x_dev),
                                _ptr(y_dev), W.N, W.K, B, _stream(stream)))


def mmq_host(W: Weight, x_host, y_host, x_dev, xq_dev, y_dev, stream=None):
    """Prefill (quantise + MMQ) from host buffers, as matvec_host: a pinned, 16-byte aligned
    x_host is read by the quantiser directly (else copied through x_dev); y goes out through
    y_dev and a copy."""
    M = x_host.shape[0]
    _check(lib().mq_mmq_host(W.qtype, W.handle, _ptr(x_host), _ptr(y_host), _ptr(x_dev),
                             _ptr(xq_dev), _ptr(y_dev), M, W.N, W.K, _stream(stream)))


STATIC_XQ_BYTES = 16 << 20  # the library's scratch for mmq_fused_static (MQ_STATIC_XQ_BYTES)


def mmq_fused_static(W: Weight, x, y=None, stream=None):
    """mmq_fused with the library's static scratch in place of an xq buffer (allocates
    nothing on the device; one call in flight at a time).  Returns y."""
    import torch
    if stream is not None and y is None:
        with torch.cuda.stream(stream):
            return mmq_fused_static(W, x)
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, W.N), dtype=torch.float32, device=x.device)
    _check(lib().mq_mmq_fused_static(W.qtype, W.handle, _ptr(x), _ptr(y), M, W.N, W.K,
                                     _stream(stream)))
    return y


def mmq_blockdots(W: Weight, xq, M: int, D=None, stream=None):
    import torch
    if stream is not None and D is None:
        with torch.cuda.stream(stream):
            return mmq_blockdots(W, xq, M)
    if D is None:
        D = torch.empty((M, W.N, W.K // 32), dtype=torch.int32, device=xq.device)
    _check(lib().mq_mmq_blockdots(W.qtype, W.handle, _ptr(xq), _ptr(D), M, W.N, W.K,
                                  _stream(stream)))
    return D


# ---- decode attention over a paged key-value cache ------------------------------------------


class _KVCacheStruct(ctypes.Structure):  # mq_kv_cache
    _fields_ = [("type", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_size", ctypes.c_int), ("n_pages", _I64), ("page_stride", _I64),
                ("head_stride", _I64), ("slot_stride", _I64), ("k", _P), ("v", _P),
                ("k_scale", _P), ("v_scale", _P), ("weight_sum", _P)]


class _RopeStruct(ctypes.Structure):  # mq_rope
    _fields_ = [("table", _P), ("max_pos", _I64), ("rot_dim", ctypes.c_int),
                ("pairs", ctypes.c_int), ("n_axes", ctypes.c_int), ("axis", ctypes.c_uint8 * 128)]


_IO = {}  # torch dtype -> type code of activations
_torch = _raw_current_stream = _empty_cuda = None


def _torch_setup():
    """What the calls below need of torch, looked up once."""
    global _torch, _raw_current_stream, _empty_cuda
    import torch
    _IO.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})
    # the current stream's handle without a Stream object (2.8 us less per call)
    _raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    # an output (shape, strides, dtype) on the current device, which the calls require to be the
    # cache's, straight from the allocator (3.4 us less per call) where a trial shows that its entry,
    # which is torch's own business, is there and does that
    def empty(shape, strides, dtype):
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")
    _empty_cuda = empty
    try:
        direct = torch._C._dynamo.guards._empty_strided_cuda
        trial = direct((2, 1), (1, 1), torch.int32)
        if trial.shape == (2, 1) and trial.dtype == torch.int32:
            _empty_cuda = direct
    except Exception:
        pass
    _torch = torch
    return torch


def _refuse(what):
    raise ValueError(what)


class KVCache:
    """A paged cache over the caller's planes (mq_kv_cache): k, v [page][head][slot][head_dim]
    (layout "hnd") or [page][slot][head][head_dim] ("nhd") of f16, bf16, or int8 with f16
    scales k_scale, v_scale of the same axes and head_dim / 32; sums f32 of the same axes
    without head_dim (the weight each row has gathered), or None.  The planes may be views with
    larger outer strides, the same in rows for all of them."""

    def __init__(self, kind, k, v, k_scale=None, v_scale=None, sums=None, layout="hnd"):
        torch = _torch or _torch_setup()
        if layout not in ("hnd", "nhd"):
            _refuse(f"layout {layout!r} is neither 'hnd' nor 'nhd'")
        want = {F16: torch.float16, BF16: torch.bfloat16, Q8_0: torch.int8}.get(kind)
        if want is None:
            _refuse(f"cache type {kind} is not F16, BF16 or Q8_0")
        if k.dim() != 4 or k.shape != v.shape:
            _refuse("k and v are [page][...][...][head_dim]")
        d = k.shape[3]
        planes = [("k", k, want, d), ("v", v, want, d)]
        if kind == Q8_0:
            if k_scale is None or v_scale is None:
                _refuse("a Q8_0 cache needs its scales")
            planes += [("k_scale", k_scale, torch.float16, d // 32),
                       ("v_scale", v_scale, torch.float16, d // 32)]
        if sums is not None:
            planes.append(("sums", sums, torch.float32, 1))
        # strides in rows (that of an axis of one element says nothing)
        rows = [k.stride(i) // max(d, 1) if k.shape[i] > 1 else 1 for i in range(3)]
        for name, t, dtype, width in planes:
            if not t.is_cuda or t.dtype != dtype:
                _refuse(f"{name} must be a CUDA tensor of {dtype}")
            if t.shape[:3] != k.shape[:3] or t.shape[3:] != (() if name == "sums" else (width,)):
                _refuse(f"{name} has shape {tuple(t.shape)}")
            if any(t.shape[i] != 1 and t.stride(i) != rows[i] * width for i in range(3)) or (
                    t.dim() == 4 and width > 1 and t.stride(3) != 1):
                _refuse(f"{name}: rows are not contiguous, or its strides differ from k's")
        head, slot = (1, 2) if layout == "hnd" else (2, 1)
        self.kind, self.k, self.v, self.k_scale, self.v_scale = kind, k, v, k_scale, v_scale
        self.sums, self.layout = sums, layout
        self.n_pages, self.n_kv_heads, self.page_size = k.shape[0], k.shape[head], k.shape[slot]
        self.head_dim, self.device = d, k.device
        self._device_index = k.device.index

        def ptr(t):
            return None if t is None else t.data_ptr()
        self._c = _KVCacheStruct(kind, self.n_kv_heads, d, self.page_size, self.n_pages, rows[0],
                                 rows[head], rows[slot], ptr(k), ptr(v),
                                 ptr(k_scale) if kind == Q8_0 else None,
                                 ptr(v_scale) if kind == Q8_0 else None, ptr(sums))
        self._ref = ctypes.addressof(self._c)


def kv_cache(kind, n_pages, page_size, n_kv_heads, head_dim, sums=False, layout="hnd",
             device="cuda") -> KVCache:
    """A KVCache over new zeroed planes."""
    import torch
    if kind not in (F16, BF16, Q8_0):
        _refuse(f"cache type {kind} is not F16, BF16 or Q8_0")
    outer = ((n_pages, n_kv_heads, page_size) if layout == "hnd"
             else (n_pages, page_size, n_kv_heads))
    dtype = {F16: torch.float16, BF16: torch.bfloat16, Q8_0: torch.int8}[kind]

    def plane(*shape, dtype):
        return torch.zeros(shape, dtype=dtype, device=device)
    k, v = (plane(*outer, head_dim, dtype=dtype) for _ in range(2))
    ks, vs = ((plane(*outer, head_dim // 32, dtype=torch.float16) for _ in range(2))
              if kind == Q8_0 else (None, None))
    return KVCache(kind, k, v, ks, vs, plane(*outer, dtype=torch.float32) if sums else None,
                   layout)


def rope_table(max_pos, inv_freq, scale=1.0, device="cuda"):
    """The f32 table [max_pos][len(inv_freq)][2] of scale * (cos, sin)(position * inv_freq),
    computed in 64 bits."""
    import torch
    f = torch.as_tensor(inv_freq, dtype=torch.float64, device=device)
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * f
    return (torch.stack([a.cos(), a.sin()], -1) * scale).float()


def rope_axes(sections, weave=False):
    """The axis of each pair for sections[a] pairs on axis a: contiguous, or woven (pair i on
    the axes in turn while they have pairs left)."""
    if not weave:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a, n in enumerate(left):
            if n:
                out.append(a)
                left[a] -= 1
    return out


class Rope:
    """A rotation (mq_rope): table f32 [max_pos][pairs of a head][2] (rope_table), axis: the
    position axis of each pair (default: all on axis 0); pairs: dims (2i, 2i+1) instead of
    (i, i + rot_dim/2); n_axes: the axes that positions are given on (default: up to the last one
    that a pair turns by)."""

    def __init__(self, table, axis=None, pairs=False, n_axes=None):
        torch = _torch or _torch_setup()
        if (table.dim() != 3 or table.shape[2] != 2 or not table.is_contiguous()
                or not table.is_cuda or table.dtype != torch.float32):
            _refuse("table must be a contiguous CUDA f32 tensor [max_pos][rot_dim/2][2]")
        half = table.shape[1]
        axis = bytes(half) if axis is None else bytes(axis)  # (refuses what is no small integer)
        if len(axis) != half or half > 128 or max(axis, default=0) > 3:
            _refuse("axis names one of up to 4 axes for each of at most 128 pairs")
        used = max(axis, default=0) + 1
        if n_axes is not None and not used <= n_axes <= 4:
            _refuse(f"n_axes={n_axes}: the pairs turn by {used} axes, and there are at most 4")
        self.table, self.axis, self.n_axes = table, list(axis), n_axes or used
        self._c = _RopeStruct(table.data_ptr(), table.shape[0], 2 * half, int(pairs), self.n_axes)
        ctypes.memmove(self._c.axis, axis, half)
        self._ref = ctypes.addressof(self._c)


def rope_store(cache: KVCache, rope: Rope, qkv, pos, slot, n_heads, bias=None, q=None,
               stream=None):
    """Rotate and store T tokens: qkv [T][(n_heads + 2 n_kv_heads) head_dim] (f32, f16 or bf16;
    rows may be strided), pos int32 [n_axes][T] (or [T] for one axis), slot int64 [T].  Returns
    the rotated queries [T][n_heads][head_dim]."""
    torch = _torch or _torch_setup()
    if stream is not None and q is None:
        with torch.cuda.stream(stream):
            return rope_store(cache, rope, qkv, pos, slot, n_heads, bias)
    T, width = qkv.shape
    ld, inner = qkv.stride()
    d = cache.head_dim
    io = _IO.get(qkv.dtype)
    if io is None or width != (n_heads + 2 * cache.n_kv_heads) * d or inner != 1:
        _refuse(f"qkv must be f32, f16 or bf16 [T][{(n_heads + 2 * cache.n_kv_heads) * d}] with "
                f"contiguous rows, not {qkv.dtype} {tuple(qkv.shape)}, strides {qkv.stride()}")
    if (pos.dtype != torch.int32 or not pos.is_contiguous()
            or pos.shape not in ((rope.n_axes, T), (T,) if rope.n_axes == 1 else None)):
        _refuse("pos must be contiguous int32 [n_axes][T]")
    if slot.dtype != torch.int64 or slot.shape != (T,) or not slot.is_contiguous():
        _refuse("slot must be contiguous int64 [T]")
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (width,)
                             or not bias.is_contiguous()):
        _refuse("bias must be contiguous f32, one per column of qkv")
    if q is None:
        q = _empty_cuda((T, n_heads, d), (n_heads * d, d, 1), qkv.dtype)
    elif q.dtype != qkv.dtype or q.numel() != T * n_heads * d or not q.is_contiguous():
        _refuse("q must be contiguous, of qkv's type")
    status = lib().mq_rope_store(
        cache._ref, rope._ref, io, qkv.data_ptr(), ld if T > 1 else width,
        None if bias is None else bias.data_ptr(), pos.data_ptr(), slot.data_ptr(), q.data_ptr(),
        T, n_heads, _raw_current_stream(cache._device_index) if stream is None else stream.cuda_stream)
    if status:
        _check(status)
    return q


ATTN_WS_ZERO = 4096  # bytes at a workspace's start that must be zero before its first call


def attn_workspace(cache: KVCache, n_seqs, n_heads, max_len, track=False):
    """A workspace for attn_decode calls of up to this size."""
    import torch
    n = lib().mq_attn_workspace_bytes(cache._ref, n_seqs, n_heads, max_len, int(bool(track)))
    if n == 0:
        raise MQError(STATUS.index("MQ_ERR_ARG"), lib().mq_last_error().decode(errors="replace"))
    ws = torch.empty(n, dtype=torch.uint8, device=cache.device)
    ws[:ATTN_WS_ZERO].zero_()
    return ws


def _pages_ld(name, pages, n_seqs, positions, page_size, int32):
    """Row stride of a page table that must hold `positions` of each sequence."""
    (rows, width), (ld, inner) = pages.shape, pages.stride()
    if pages.dtype != int32 or rows != n_seqs or (inner != 1 and width != 1):
        _refuse(f"{name} must be int32 [S][pages]")
    if positions > width * page_size:
        _refuse(f"{name}: {positions} positions are more than {width} pages hold")
    return ld if n_seqs > 1 else width


def attn_decode(cache: KVCache, q, pages, lens, max_len, scale=None, window=0, track=False,
                ws=None, o=None, stream=None):
    """Attention of one new token per sequence: q [S][n_heads][head_dim] (f32, f16 or bf16),
    pages int32 [S][max pages], lens int32 [S] (at most max_len).  scale defaults to
    head_dim ** -0.5.  ws: a workspace kept from attn_workspace (else one is made for the
    call).  Returns o, of q's shape and type."""
    torch = _torch or _torch_setup()
    if stream is not None and (ws is None or o is None):
        with torch.cuda.stream(stream):
            return attn_decode(cache, q, pages, lens, max_len, scale, window, track, ws, o)
    S, n_heads, d = q.shape
    io = _IO.get(q.dtype)
    if io is None or d != cache.head_dim or not q.is_contiguous():
        _refuse(f"q must be a contiguous tensor [S][n_heads][{cache.head_dim}] of f32, f16 or "
                f"bf16, not {q.dtype} {tuple(q.shape)}")
    pages_ld = _pages_ld("pages", pages, S, max_len, cache.page_size, torch.int32)
    if lens.dtype != torch.int32 or lens.shape != (S,) or not lens.is_contiguous():
        _refuse("lens must be contiguous int32 [S]")
    if track and cache.sums is None:
        _refuse("the cache keeps no weight sums")
    if ws is None:
        ws = attn_workspace(cache, S, n_heads, max_len, track)
    if o is None:
        o = _empty_cuda((S, n_heads, d), (n_heads * d, d, 1), q.dtype)
    elif o.dtype != q.dtype or o.shape != q.shape or not o.is_contiguous():
        _refuse("o must be contiguous, of q's shape and type")
    status = lib().mq_attn_decode(
        cache._ref, io, q.data_ptr(), o.data_ptr(), pages.data_ptr(), pages_ld, lens.data_ptr(), S,
        n_heads, max_len, d ** -0.5 if scale is None else scale, window, 1 if track else 0,
        ws.data_ptr(), ws.numel(),
        _raw_current_stream(cache._device_index) if stream is None else stream.cuda_stream)
    if status:
        _check(status)
    return o


def kv_evict(cache: KVCache, pages, lens, max_len, new_pages, keep, sink=0, recent=0, kept=None,
             new_lens=None, stream=None):
    """Copy the rows that stay (the first sink, the last recent and the heaviest of the rest, keep
    in all) to new_pages.  Returns (kept int32 [S][n_kv_heads][keep], new_lens int32 [S]); new_lens
    may be lens itself."""
    torch = _torch or _torch_setup()
    if stream is not None and (kept is None or new_lens is None):
        with torch.cuda.stream(stream):
            return kv_evict(cache, pages, lens, max_len, new_pages, keep, sink, recent, kept, new_lens)
    if lens.dtype != torch.int32 or lens.dim() != 1 or not lens.is_contiguous():
        _refuse("lens must be contiguous int32 [S]")
    S = lens.shape[0]
    pages_ld = _pages_ld("pages", pages, S, max_len, cache.page_size, torch.int32)
    new_ld = _pages_ld("new_pages", new_pages, S, keep, cache.page_size, torch.int32)
    if cache.sums is None:
        _refuse("the cache keeps no weight sums")
    if kept is None:
        heads = cache.n_kv_heads
        kept = _empty_cuda((S, heads, keep), (heads * keep, keep, 1), torch.int32)
    elif (kept.dtype != torch.int32 or kept.numel() != S * cache.n_kv_heads * keep
          or not kept.is_contiguous()):
        _refuse("kept must be contiguous int32 [S][n_kv_heads][keep]")
    if new_lens is None:
        new_lens = _empty_cuda((S,), (1,), torch.int32)
    elif (new_lens.dtype != torch.int32 or new_lens.shape != lens.shape
          or not new_lens.is_contiguous()):
        _refuse("new_lens must be contiguous int32 [S]")
    status = lib().mq_kv_evict(
        cache._ref, pages.data_ptr(), pages_ld, lens.data_ptr(), S, max_len, new_pages.data_ptr(),
        new_ld, keep, sink, recent, kept.data_ptr(), new_lens.data_ptr(),
        _raw_current_stream(cache._device_index) if stream is None else stream.cuda_stream)
    if status:
        _check(status)
    return kept, new_lens


def stream_status(stream=None):
    _check(lib().mq_stream_status(_stream(stream)))
