"""mq_sample's kernel run on the host, its threads going on in any order that its barriers allow: results are the
definition's, and the same to the last bit, whichever thread, warp or block is behind."""
import ctypes

import numpy as np
import pytest

from oracle.sampling import sample as exact
from tests import sample_threads as st


@pytest.fixture(scope="module")
def f(tmp_path_factory):
    return st.build(str(tmp_path_factory.mktemp("sample_host")))


def run(f, x, u, ranks_log, orders=st.ORDERS, **given):
    """All orders' results, which are one, and the definition's."""
    first = None
    for order in orders:
        token, logprob = st.sample(f, x, u, ranks_log, order, **given)
        if first is None:
            first = token, logprob
        assert token.tolist() == first[0].tolist() and logprob.tobytes() == first[1].tobytes(), (order, token, first)
    for b in range(len(x)):
        kw = {k: v[b] for k, v in given.items()}
        want, lp, margin = exact(x[b], float(u[b]), **kw)
        assert margin > 2.0 ** -24  # (of these rows)
        assert int(first[0][b]) == want and abs(float(first[1][b]) - lp) < 2.0 ** -20, (b, first, want, lp)


def rows(B, V, seed):
    g = np.random.default_rng(seed)
    return (g.standard_normal((B, V)) * 2).astype(np.float32), g.random(B).astype(np.float32)


@pytest.mark.parametrize("ranks_log", [0, 1, 2])
@pytest.mark.parametrize("V", [16384, 20001])
def test_temperature_alone(f, V, ranks_log):
    """A block that is ahead has its sum ready while others still choose the weights' unit."""
    x, u = rows(2, V, 0)
    run(f, x, u, ranks_log, temperature=[0.8, 1.3])


@pytest.mark.parametrize("ranks_log", [0, 1])
@pytest.mark.parametrize("k", [257, 289, 321, 500, 700])
def test_cuts_that_leave_more_than_are_counted(f, k, ranks_log):
    """The cut is read from the sorted list by all threads before the list's place is used again."""
    x, u = rows(1, 12001, k)
    run(f, x, u, ranks_log, top_k=[k])
    run(f, x, u, ranks_log, top_k=[k], top_p=[0.999])


def test_unit_of_the_weights(f):
    """What the unit is chosen by has every group's maximum: here their mean lies at 2^-7.93, and at
    2^-8.03 without the last one of each warp; the other tokens, at 2^-36, count in the smaller unit only."""
    V, ln2 = 16384, np.log(2.0)
    x = np.full((1, V), -36 * ln2, np.float32)
    x[0, 64::128] = -8.1 * ln2      # 128 groups, nine to a warp
    x[0, 64 + 128 * 8::128 * 9] = -7.1 * ln2
    x[0, 5] = 0
    u = np.array([0.3], np.float32)
    run(f, x, u, 0, temperature=[1.0])


@pytest.mark.parametrize("io_rows", [1, 2])
@pytest.mark.parametrize("ranks_log", [0, 1])
def test_results_do_not_depend_on_the_address(f, ranks_log, io_rows):
    """The same logits from any element of a 16-byte block on: groups of 128 are counted from the row's start.  Of every
    second group the first and the last token are heavy (2^-7.2), so that groups counted from a block's start would
    all have one, and their mean another unit, in which the tokens at 2^-36 do not count."""
    V, ln2 = 16384 + 70, np.log(2.0)
    x = np.full((io_rows, V), -36 * ln2, np.float32)
    x[:, 0::256] = x[:, 127::256] = -7.2 * ln2
    x[:, 7] = 0
    x[1:, 9000:9050] = np.nan
    u = np.array([0.3, 0.9][:io_rows], np.float32)
    want = st.sample(f, x, u, ranks_log, temperature=[1.0] * io_rows)
    for shift in range(4):
        for ld in (V + 2, V + 3):
            wide = np.full(io_rows * ld + 8, 50, np.float32)
            start = -(wide.ctypes.data // 4) % 4 + shift
            view = wide[start:start + io_rows * ld].reshape(io_rows, ld)[:, :V]
            view[:] = x
            token, logprob = st.sample(f, view, u, ranks_log, temperature=[1.0] * io_rows)
            assert token.tolist() == want[0].tolist() and logprob.tobytes() == want[1].tobytes(), (shift, ld)


def test_clusters_that_every_type_can_have(f):
    """The kernels of the three types have one table: what is resident at once of each of them."""
    per_kernel = [[100, 50, 24, 10, 5], [90, 60, 24, 11, -1], [120, 70, 30, 12, 6]]
    given, out = (ctypes.c_int * 15)(*sum(per_kernel, [])), (ctypes.c_int * 5)()
    init = f.library.sample_host_init
    init.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    assert init(given, out) == 0 and list(out) == [90, 50, 24, 10, 0]


@pytest.mark.parametrize("T", [2.0 ** -149, 1e-40, 2.0 ** -128])
def test_temperatures_below_the_smallest(f, T):
    """A temperature below 2^-127, whose inverse binary32 does not hold, is taken as that: weights and logprob alike."""
    x = np.array([[0.0, -1.0, -2.0, -0.5, -200.0] * 3], np.float32) * np.float32(2.0 ** -127)
    for u in (0.05, 0.3, 0.5, 0.8, 0.97):
        token, logprob = st.sample(f, x, [u], 0, temperature=[T])
        want, lp, margin = exact(x[0], float(np.float32(u)), temperature=2.0 ** -127)
        assert margin > 1e-3 and token[0] == want and abs(logprob[0] - lp) < 1e-6, (u, token, logprob, want, lp)
    token, logprob = st.sample(f, x * np.float32(2.0 ** 100), [0.9], 0, temperature=[T])
    assert token[0] == 10 and abs(logprob[0] - np.log(1 / 3)) < 1e-6


@pytest.mark.parametrize("V,size", [(1000, 1.0), (5000, 0.1), (16384, 2.0), (3, 5.0)])
def test_log_probabilities_are_rounded_once(f, V, size):
    """To binary32's nearest, but for the sum's own error (2^-26 of it) and what two parts of a quotient and a logarithm
    leave (2^-28 of each)."""
    g = np.random.default_rng(V)
    B = 24
    x = (g.standard_normal((B, V)) * size).astype(np.float32)
    u = g.random(B).astype(np.float32)
    for kw in ({"temperature": [0.9 + 0.1 * b for b in range(B)]}, {"top_k": [100] * B, "temperature": [1.7] * B}, {"min_p": [0.01] * B}):
        token, logprob = st.sample(f, x, u, 0, **kw)
        for b in range(B):
            want, lp, margin = exact(x[b], float(u[b]), **{k: v[b] for k, v in kw.items()})
            if margin < 2.0 ** -24:
                continue
            assert int(token[b]) == want
            step = 2.0 ** (np.floor(np.log2(abs(lp) + 1e-30)) - 24)
            assert abs(float(logprob[b]) - lp) <= step + 2.0 ** -26 + abs(lp) * 2.0 ** -27, (b, kw, logprob[b], lp)


def test_distances_beyond_binary32(f):
    """What the header says of logits that lie further apart than binary32 reaches, at any temperature."""
    x = np.array([[3e38, -3e38, 2.9e38, 0.0]], np.float32)
    for u, T, want in ((0.5, np.inf, 2), (0.99, np.inf, 3), (0.1, 1e38, 0), (0.99, 1e38, 3)):
        token, logprob = st.sample(f, x, [u], 0, temperature=[T])
        w = np.exp((x[0, [0, 2, 3]].astype(np.float64) - 3e38) / T)
        assert token[0] == want and abs(logprob[0] - np.log(w[[0, 2, 3].index(want)] / w.sum())) < 1e-6
