"""The example's step refuses parts that do not fit one another, before it makes anything: a token that the head can
name and the embedding has no row for would be read past its end."""
import types

import pytest

torch = pytest.importorskip("torch")

from gguf_block_quantized_q4_gb300.examples import decode_step  # noqa: E402


def layer(n):
    return types.SimpleNamespace(held=[0] * n)


@pytest.mark.parametrize("rows,heads,layers,word", [(100, 101, [2], "101"), (100, 99, [2], "99"), (100, 100, [2, 3], "sequences"),
                                                    (100, 100, [], "layers")])
def test_parts(rows, heads, layers, word):
    with pytest.raises(ValueError, match=word):
        decode_step.DecodeStep(torch.zeros((rows, 32)), [layer(n) for n in layers], types.SimpleNamespace(N=heads, K=32))
