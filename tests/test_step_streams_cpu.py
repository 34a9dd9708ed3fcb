"""As test_kv_streams_cpu, for the norms' and the sampling calls: what they make belongs to the stream that
their kernels run on, what the caller gives is used."""
import types

import pytest

torch = pytest.importorskip("torch")

import gguf_block_quantized_q4_gb300 as mq
from tests.test_kv_streams_cpu import HERE, OTHER, Stream, record, store  # noqa: F401


def norm_store(**kw):
    return store(norm=types.SimpleNamespace(head_dim=64, _ref=0), **kw)


def sample(**kw):
    return mq.sample(torch.zeros((2, 50)), torch.zeros(2), top_p=torch.ones(2), **kw)


CALLS = {"mq_norm_rope_store": (norm_store, ["empty"], lambda: dict(q=torch.zeros((2, 2, 64)))),
         "mq_sample": (sample, ["empty", "empty"], lambda: dict(token=torch.zeros(2, dtype=torch.int32), logprob=torch.zeros(2)))}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("given", [False, True])
def test_one_stream_for_a_call_and_what_it_makes(record, name, given):  # noqa: F811
    call, makes, _ = CALLS[name]
    call(**(dict(stream=Stream()) if given else {}))
    assert [what for what, _ in record] == [*makes, name]
    assert {stream for _, stream in record} == {OTHER if given else HERE}


@pytest.mark.parametrize("name", CALLS)
def test_what_the_caller_gives_is_used(record, name):  # noqa: F811
    call, _, outputs = CALLS[name]
    call(**outputs(), stream=Stream())
    assert record == [(name, OTHER)]
    call(**outputs())
    assert record[1:] == [(name, HERE)]


def test_one_output_of_the_callers(record):  # noqa: F811
    """The other is made on the call's stream."""
    token = torch.zeros(2, dtype=torch.int32)
    got = sample(token=token, stream=Stream())
    assert got[0] is token and record == [("empty", OTHER), ("mq_sample", OTHER)]


def test_norms_for_other_heads_are_refused(record):  # noqa: F811
    with pytest.raises(ValueError, match="heads of 128"):
        store(norm=types.SimpleNamespace(head_dim=128, _ref=0))
    assert all(what != "mq_norm_rope_store" for what, _ in record)
