"""How the paged cache's calls make their outputs: straight from torch's allocator where its entry
is there and takes what it is given, else by torch.empty_strided."""
import types

import pytest

torch = pytest.importorskip("torch")

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402


def direct(shape, strides, dtype):
    return torch.zeros(shape, dtype=dtype)


def other_signature(shape, strides, *, dtype, device):
    raise AssertionError("not to be reached")


def other_result(shape, strides, dtype):
    return None


@pytest.mark.parametrize("entry,used", [(direct, True), (other_signature, False), (other_result, False),
                                        (None, False)])
def test_outputs_come_from_an_entry_that_works(monkeypatch, entry, used):
    monkeypatch.setattr(torch._C, "_dynamo", types.SimpleNamespace(
        guards=types.SimpleNamespace(**({} if entry is None else {"_empty_strided_cuda": entry}))))
    made = []

    def empty_strided(shape, strides, dtype, device):
        made.append(device)
        return torch.zeros(shape, dtype=dtype)
    monkeypatch.setattr(torch, "empty_strided", empty_strided)
    try:
        mq._torch_setup()
        out = mq._empty_cuda((2, 3), (3, 1), torch.float16)
    finally:
        monkeypatch.undo()
        mq._torch_setup()
    assert out.shape == (2, 3) and out.dtype == torch.float16
    assert made == ([] if used else ["cuda"])
