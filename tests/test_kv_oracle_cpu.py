"""The 64-bit definitions of the decode-attention operators against hand-worked values."""
import numpy as np

from oracle import kv


def test_attention_of_two_keys_by_hand():
    cache = {"k": np.zeros((2, 1, 2, 2)), "v": np.zeros((2, 1, 2, 2))}
    # page 1 holds positions 0, 1; page 0 position 2
    cache["k"][1, 0, 0], cache["k"][1, 0, 1], cache["k"][0, 0, 0] = (1, 0), (0, 2), (50, 50)
    cache["v"][1, 0, 0], cache["v"][1, 0, 1], cache["v"][0, 0, 0] = (4, 8), (8, 0), (1, 1)
    q = np.array([[[np.log(3.0), 0.0]]])
    pages = np.array([[1, 0]])
    # s = (ln 3, 0): w = (3/4, 1/4)
    o, mass, reach, weights = kv.attn_decode(cache, 2, q, pages, [2], 1.0)
    assert np.allclose(o[0, 0], [5.0, 6.0]) and np.allclose(mass, o)
    assert np.isclose(reach[0, 0], np.log(3.0)) and weights[0][0] == 0
    assert np.allclose(weights[0][1], [[0.75, 0.25]])
    # a window of one sees the last key alone; no keys give zeros
    o, _, _, weights = kv.attn_decode(cache, 2, q, pages, [2], 1.0, window=1)
    assert np.allclose(o[0, 0], [8.0, 0.0]) and weights[0][0] == 1
    assert not kv.attn_decode(cache, 2, q, pages, [0], 1.0)[0].any()


def test_rotation_by_a_right_angle():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    table = np.zeros((3, 2, 2))
    table[..., 0] = 1.0  # no turn
    table[2, 1] = (0.0, 1.0)  # a quarter turn of pair 1 at position 2
    pos = np.array([[0], [2]])
    # pair 1 on axis 1: halves (2, 4) -> (-4, 2); neighbours (3, 4) -> (-4, 3)
    assert kv.rope(x, table, pos, [0, 1], False)[0, 0].tolist() == [1, -4, 3, 2, 5, 6, 7, 8]
    assert kv.rope(x, table, pos, [0, 1], True)[0, 0].tolist() == [1, 2, -4, 3, 5, 6, 7, 8]
    assert kv.rope(x, table, pos, [0, 0], True)[0, 0].tolist() == list(range(1, 9))


def test_quantised_rows_by_hand():
    x = np.zeros((1, 64), np.float32)
    x[0, 0], x[0, 1], x[0, 2] = 127.0, -0.5, 1.5  # d = 1: ties go to the even quant
    x[0, 33] = -254.0
    q, d = kv.quantise_rows(x)
    assert d.tolist() == [[1.0, 2.0]]
    assert q[0, :3].tolist() == [127, 0, 2] and q[0, 33] == -127
    q, d = kv.quantise_rows(np.zeros((1, 32), np.float32))
    assert not q.any() and not d.any()


def test_eviction_order():
    w = [9.0, 1.0, 5.0, 5.0, 0.0, 5.0, 2.0, 0.0]
    assert kv.evict(w, 8, 8, 0, 0) == list(range(8))
    assert kv.evict(w, 8, 3, 0, 0) == [0, 2, 3]  # the equal sums from the lowest position
    assert kv.evict(w, 8, 4, 1, 1) == [0, 2, 3, 7]
    assert kv.evict(w, 8, 2, 1, 1) == [0, 7]
    w[4] = float("nan")
    assert kv.evict(w, 8, 2, 0, 0) == [0, 4]
