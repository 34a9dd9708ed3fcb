"""Refusals of outputs that overlap inputs in ways the kernels cannot serve; no device needed (they
are made before the pointers themselves are looked at)."""
import ctypes

import pytest

import gguf_block_quantized_q4_gb300 as mq
from gguf_block_quantized_q4_gb300 import build as mqbuild
from tests.test_kv_abi_cpu import cache, rope


@pytest.fixture(scope="module")
def L():
    mqbuild.build()
    return mq.lib()


@pytest.mark.parametrize("S,shift,refused", [(8, 0, False), (8, 4, True), (8, -4, True), (8, 28, True),
                                             (8, -28, True), (8, 32, False), (8, -32, False),
                                             (1, 4, False), (1, -4, False)])
def test_new_lengths_are_the_lengths_or_apart(L, S, shift, refused):
    """In place or apart goes on (to the next refusal, the missing device or a NULL pointer)."""
    base = 1 << 20
    c = cache()
    st = L.mq_kv_evict(ctypes.byref(c), None, 7, base, S, 100, None, 4, 64, 0, 0, None, base + shift, None)
    assert ("overlaps" in L.mq_last_error().decode()) == refused
    assert mq.STATUS[st] in (["MQ_ERR_ARG"] if refused else ["MQ_ERR_ARG", "MQ_ERR_STATE", "MQ_ERR_CUDA"])


@pytest.mark.parametrize("T,shift,refused", [(1, 0, False),            # in place: a thread its own elements
                                             (1, 16, True), (1, -16, True),
                                             (1, 36 * 128 * 2, False), (1, -28 * 128 * 2, False),
                                             (3, 0, True),             # a token's queries over another's row
                                             (3, 2 * 40 * 128 * 2, True), (3, -3 * 28 * 128 * 2 + 16, True),
                                             (3, (2 * 40 + 36) * 128 * 2, False), (3, -3 * 28 * 128 * 2, False)])
def test_rotated_queries_are_apart_from_the_rows(L, T, shift, refused):
    """Rows of 36 heads, 40 heads from one to the next, f16; queries of 28 heads."""
    base = 1 << 24
    c, r = cache(), rope()
    st = L.mq_rope_store(ctypes.byref(c), ctypes.byref(r), mq.F16, base, 40 * 128, None, None, None,
                         base + shift, T, 28, None)
    assert ("overlaps" in L.mq_last_error().decode()) == refused
    assert mq.STATUS[st] in (["MQ_ERR_ARG"] if refused else ["MQ_ERR_ARG", "MQ_ERR_STATE", "MQ_ERR_CUDA"])


@pytest.mark.parametrize("shift,refused", [(0, False), (16, True), (-16, True), (2 * 28 * 128 * 4 - 16, True),
                                           (2 * 28 * 128 * 4, False), (-2 * 28 * 128 * 4, False)])
def test_attention_outputs_are_the_queries_or_apart(L, shift, refused):
    """Two sequences, 28 heads of 128, f32."""
    base = 1 << 24
    c = cache()
    st = L.mq_attn_decode(ctypes.byref(c), 0, base, base + shift, None, 7, None, 2, 28, 100, 0.1, 0, 0, None, 0, None)
    assert ("overlaps" in L.mq_last_error().decode()) == refused
    assert mq.STATUS[st] in (["MQ_ERR_ARG"] if refused else ["MQ_ERR_ARG", "MQ_ERR_STATE", "MQ_ERR_CUDA"])
