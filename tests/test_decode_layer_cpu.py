"""The example's layer refuses budgets that its calls could not keep, before it makes anything."""
import pytest

pytest.importorskip("torch")

from gguf_block_quantized_q4_gb300.examples import decode_layer  # noqa: E402


@pytest.mark.parametrize("kw,word", [(dict(limit=8, keep=8), "keep"), (dict(limit=8, keep=9), "keep"),
                                     (dict(limit=64, keep=0, sink=0, recent=0), "keep"),
                                     (dict(limit=64, keep=19), "sink"), (dict(limit=64, keep=32, sink=-1), "sink"),
                                     (dict(limit=64, keep=32, recent=29), "sink")])
def test_budgets(kw, word):
    """(an eviction has to make room, and keeps the first and the last)"""
    with pytest.raises(ValueError, match=word):
        decode_layer.DecodeLayer(None, None, 1, 2, 1, 64, **kw)
