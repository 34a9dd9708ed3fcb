"""Sampling without a device: the 64-bit definition pinned by worked rows, the call's refusals, the
binding's checks."""
import ctypes
import math

import numpy as np
import pytest

import gguf_block_quantized_q4_gb300 as mq
from gguf_block_quantized_q4_gb300 import build as mqbuild
from oracle.sampling import sample

L4 = np.log(np.array([4.0, 1.0, 2.0, 1.0]))  # shares 1/2, 1/8, 1/4, 1/8


@pytest.mark.parametrize("u,token", [(0.0, 0), (0.49, 0), (0.51, 1), (0.62, 1), (0.63, 2), (0.87, 2), (0.88, 3), (0.999, 3)])
def test_plain_draws(u, token):
    got = sample(L4, u)
    assert got[0] == token and abs(got[1] - math.log([0.5, 0.125, 0.25, 0.125][token])) < 1e-12


def test_limits():
    assert [sample(L4, u, top_k=1)[0] for u in (0.0, 0.99)] == [0, 0]
    # two stay: 0 and 2, by 2/3 and 1/3
    assert [sample(L4, u, top_k=2)[0] for u in (0.6, 0.7)] == [0, 2]
    # three stay: of the equal ones the first
    assert [sample(L4, u, top_k=3)[0] for u in (0.5, 0.6, 0.999)] == [0, 1, 2]
    assert sample(L4, 0.999, top_p=0.5)[0] == 0 and sample(L4, 0.999, top_p=0.51)[0] == 2
    assert sample(L4, 0.999, top_p=0.0)[0] == 0
    # 3/4 of the sum is reached by two
    assert [sample(L4, u, top_p=0.74)[0] for u in (0.6, 0.7)] == [0, 2]
    assert [sample(L4, u, min_p=0.3)[0] for u in (0.6, 0.7)] == [0, 2] and sample(L4, 0.99, min_p=2.0)[0] == 0
    # T = 1/2 squares the weights: 16, 1, 4, 1
    assert [sample(L4, u, temperature=0.5)[0] for u in (0.72, 0.73)] == [0, 1]
    assert sample(L4, 0.9, temperature=0.0)[:2] == (0, 0.0) and sample([1.0, 3.0, 3.0], 0.9, temperature=float("nan"))[0] == 1


def test_what_is_no_number():
    inf, nan = float("inf"), float("nan")
    assert sample([-inf, nan, -inf], 0.5)[:2] == (-1, -inf)
    assert sample([nan, 0.0, -inf], 0.99)[0] == 1
    assert [sample([0.0, inf, inf], u)[0] for u in (0.4, 0.6)] == [1, 2]
    assert [sample([0.0, 5.0, -inf, 1.0], u, temperature=inf)[0] for u in (0.3, 0.6, 0.7)] == [0, 1, 3]
    assert sample(L4, 1.5)[0] == 3 and sample(L4, nan)[0] == 0 and sample(L4, -1.0)[0] == 0


@pytest.fixture(scope="module")
def L():
    mqbuild.build()
    return mq.lib()


def call(L, io=0, ld=100, B=2, V=100, token=None, logprob=None, u=None, logits=None, top_k=None):
    p = ctypes.c_void_p
    st = L.mq_sample(io, p(logits), ld, B, V, p(u), None, p(top_k), None, None, p(token), p(logprob), None)
    return mq.STATUS[st], L.mq_last_error().decode()


@pytest.mark.parametrize("kw,status,word", [
    (dict(io=mq.Q8_0), "MQ_ERR_TYPE", "io type"), (dict(B=-1), "MQ_ERR_ARG", "B=-1"), (dict(B=65536), "MQ_ERR_ARG", "B="),
    (dict(V=0), "MQ_ERR_SHAPE", "V=0"), (dict(V=1 << 19, ld=1 << 19), "MQ_ERR_SHAPE", "V="), (dict(ld=99), "MQ_ERR_SHAPE", "ld=99"),
    (dict(ld=(1 << 31) + 1), "MQ_ERR_SHAPE", "ld="),
    (dict(logits=4096, token=4096 + 796), "MQ_ERR_ARG", "overlaps logits"), (dict(u=4096, token=4092), "MQ_ERR_ARG", "overlaps u"),
    (dict(top_k=4096, logprob=4100), "MQ_ERR_ARG", "overlaps top_k"), (dict(token=4096, logprob=4096), "MQ_ERR_ARG", "overlaps token")])
def test_refusals(L, kw, status, word):
    got = call(L, **kw)
    assert got[0] == status and word in got[1], got


def test_what_does_not_overlap_goes_on_to_the_next_check(L):
    got = call(L, logits=4096, token=4096 + 800, logprob=4096 + 808, u=4096 + 816)
    assert "overlaps" not in got[1], got


def test_the_binding_refuses_other_shapes():
    torch = pytest.importorskip("torch")
    x, u = torch.zeros((2, 10)), torch.zeros(2)
    for bad in (dict(u=torch.zeros(3)), dict(u=torch.zeros(2, dtype=torch.float64)), dict(u=None), dict(top_k=torch.zeros(2)),
                dict(temperature=torch.zeros((2, 1))), dict(min_p=torch.zeros(4)[::2]), dict(token=torch.zeros(2)),
                dict(logits=torch.zeros((10, 2)).T), dict(logits=torch.zeros((2, 10), dtype=torch.float64))):
        args = dict(logits=x, u=u) | bad
        with pytest.raises(ValueError):
            mq.sample(args.pop("logits"), args.pop("u"), **args)
