"""The number of position axes of a rotation: that of the caller's positions, not only of the axes
that its pairs use (a section may be empty)."""
import types

import pytest

torch = pytest.importorskip("torch")

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402


def table(half):
    return types.SimpleNamespace(dim=lambda: 3, shape=(10, half, 2), is_contiguous=lambda: True, is_cuda=True,
                                 dtype=torch.float32, data_ptr=lambda: 16)


def test_axes_without_pairs():
    assert mq.Rope(table(4), [0, 0, 1, 1]).n_axes == 2
    r = mq.Rope(table(4), [0, 0, 1, 1], n_axes=3)
    assert r.n_axes == 3 and r._c.n_axes == 3 and r.axis == [0, 0, 1, 1]
    assert mq.Rope(table(4), n_axes=4).n_axes == 4


@pytest.mark.parametrize("n_axes", [0, 1, 5])
def test_axes_out_of_range(n_axes):
    with pytest.raises(ValueError, match="axes"):
        mq.Rope(table(4), [0, 0, 1, 1], n_axes=n_axes)
