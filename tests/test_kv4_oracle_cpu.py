"""The 64-bit definitions of Q4_0 rows and of the heads' norms, pinned by worked values."""
import numpy as np

from oracle import kv


def test_a_block_by_hand():
    x = np.zeros(32, np.float32)
    x[0], x[1], x[2], x[16], x[31] = -4.0, 2.0, 0.25, 3.4, -0.75
    n, d = kv.quantise_rows4(x)
    # the largest is -4: d = 0.5, n = 8 + x / d with 0.25 / 0.5 = 0.5 and -1.5 rounded to even
    assert d.tolist() == [0.5]
    assert [int(n[i]) for i in (0, 1, 2, 3, 16, 31)] == [0, 12, 8, 8, 15, 6]
    b = kv.pack4(n)
    assert b.shape == (16,) and b[0] == (0 | 15 << 4) and b[15] == (8 | 6 << 4)
    assert np.array_equal(kv.unpack4(b), n)


def test_the_largest_of_two_alike_is_the_positive_one():
    for at in ((3, 20), (20, 3)):
        x = np.zeros(32, np.float32)
        x[at[0]], x[at[1]] = 1.0, -1.0
        n, d = kv.quantise_rows4(x)
        assert d[0] == -0.125 and n[at[0]] == 0 and n[at[1]] == 15  # (16 does not fit)


def test_ends():
    n, d = kv.quantise_rows4(np.zeros(64, np.float32))
    assert not d.any() and (n == 8).all()
    n, d = kv.quantise_rows4(np.full(32, 3e38, np.float32))
    assert d[0] == -65504 and (n == 0).all()


def test_values_are_within_half_a_step():
    x = np.random.default_rng(1).standard_normal((50, 64)).astype(np.float32)
    n, d = kv.quantise_rows4(x)
    step = np.repeat(np.abs(d.astype(np.float64)), 32, -1)
    err = np.abs((n - 8.0) * np.repeat(d.astype(np.float64), 32, -1) - x)
    # (the side opposite to the largest ends at 7, a step short)
    assert (err <= step * 1.01).all() and (err <= step * 0.501).mean() > 0.98


def test_norm_by_hand():
    x = np.array([[3.0, 4.0, 0.0, 0.0]], np.float32)
    assert abs(kv.head_scale(x, 0.0)[0] - 0.4) < 1e-15
    assert abs(kv.head_scale(x, 0.25)[0] - 1 / np.sqrt(6.5)) < 1e-15
