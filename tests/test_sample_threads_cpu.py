"""mq_sample's kernel run on the host, its threads going on in any order that its barriers allow: results are the
definition's, and the same to the last bit, whichever thread, warp or block is behind."""
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
