"""Which stream the paged cache's calls allocate, clear and launch on, with the library and the
device's streams replaced by records: what a call makes for itself (outputs, a workspace and its
cleared counters) must belong to the stream that the kernels run on, for nothing orders another
stream's work before them or keeps the memory until they have ended."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402

HERE, OTHER = 11, 22  # streams' handles


class Stream:
    cuda_stream = OTHER


@pytest.fixture
def record(monkeypatch):
    """Events (what, the current stream then) of a call; launches name their own stream too."""
    events, current = [], [HERE]

    @contextlib.contextmanager
    def use(stream):
        before, current[0] = current[0], stream.cuda_stream
        yield
        current[0] = before

    def empty(shape, strides, dtype):
        events.append(("empty", current[0]))
        return torch.empty_strided(shape, strides, dtype=dtype)

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                if name == "mq_attn_workspace_bytes":
                    events.append(("workspace", current[0]))
                    return 8192
                events.append((name, args[-1]))
                return 0
            return call

    mq._torch_setup()
    monkeypatch.setattr(mq, "_empty_cuda", empty)
    monkeypatch.setattr(mq, "_raw_current_stream", lambda device: current[0])
    monkeypatch.setattr(mq, "lib", lambda: Lib())
    monkeypatch.setattr(torch.cuda, "stream", use)
    return events


def cache():
    return types.SimpleNamespace(head_dim=64, n_kv_heads=1, page_size=16, sums=torch.zeros(1),
                                 device="cpu", _device_index=0, _ref=0)


def attn(**kw):
    return mq.attn_decode(cache(), torch.zeros((2, 2, 64)), torch.zeros((2, 3), dtype=torch.int32),
                          torch.zeros(2, dtype=torch.int32), 40, **kw)


def store(**kw):
    rope = types.SimpleNamespace(n_axes=1, _ref=0)
    return mq.rope_store(cache(), rope, torch.zeros((2, 4 * 64)), torch.zeros((1, 2), dtype=torch.int32),
                         torch.zeros(2, dtype=torch.int64), 2, **kw)


def evict(**kw):
    pages = torch.zeros((2, 3), dtype=torch.int32)
    return mq.kv_evict(cache(), pages, torch.zeros(2, dtype=torch.int32), 40, pages, 16, **kw)


CALLS = {"mq_attn_decode": (attn, ["workspace", "empty"]), "mq_rope_store": (store, ["empty"]),
         "mq_kv_evict": (evict, ["empty", "empty"])}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("given", [False, True])
def test_one_stream_for_a_call_and_what_it_makes(record, name, given):
    call, makes = CALLS[name]
    call(**(dict(stream=Stream()) if given else {}))
    assert [what for what, _ in record] == [*makes, name]
    assert {stream for _, stream in record} == {OTHER if given else HERE}


@pytest.mark.parametrize("name", CALLS)
def test_what_the_caller_gives_is_used(record, name):
    """Outputs and workspace of the caller's: nothing is made, and the launch is on its stream."""
    call, _ = CALLS[name]
    i32 = dict(dtype=torch.int32)
    given = {"mq_attn_decode": dict(ws=torch.zeros(8192, dtype=torch.uint8), o=torch.zeros((2, 2, 64))),
             "mq_rope_store": dict(q=torch.zeros((2, 2, 64))),
             "mq_kv_evict": dict(kept=torch.zeros((2, 1, 16), **i32), new_lens=torch.zeros(2, **i32))}[name]
    call(**given, stream=Stream())
    assert record == [(name, OTHER)]
    call(**given)
    assert record[1:] == [(name, HERE)]
