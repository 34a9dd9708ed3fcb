"""Which stream the products' calls allocate and launch on, with the library and the device's streams
replaced by records: outputs, activation buffers (whose barrier count must be zero before the
kernel) and copies of strided inputs belong to the stream that the kernel runs on."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402

HERE, OTHER = 11, 22  # streams' handles


@pytest.fixture
def record(monkeypatch):
    """(what, stream) of every allocation and launch."""
    events, current = [], [HERE]

    @contextlib.contextmanager
    def use(stream):
        before, current[0] = current[0], stream.cuda_stream
        yield
        current[0] = before

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                if name == "mq_act_bytes":
                    return 4096
                events.append((name, args[-1].value))
                return 0
            return call

    def recorded(make):
        def run(*args, **kw):
            events.append(("made", current[0]))
            return make(*args, **kw)
        return run

    monkeypatch.setattr(mq, "lib", lambda: Lib())
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=current[0]))
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    return events


W = types.SimpleNamespace(qtype=0, handle=0, N=64, K=256)
X = torch.ones((3, 256))
XQ = torch.ones(4096, dtype=torch.uint8)
CALLS = {
    "mq_matvec": (lambda **kw: mq.matvec(W, X, **kw), 1),
    "mq_ffn_gu_matvec": (lambda **kw: mq.ffn_gu_matvec(W, X, **kw), 1),
    "mq_ffn_gu_mmq": (lambda **kw: mq.ffn_gu_mmq(W, XQ, 3, **kw), 1),
    "mq_quantize_act": (lambda **kw: mq.quantize_act(X, **kw), 1),
    "mq_mmq": (lambda **kw: mq.mmq(W, XQ, 3, **kw), 1),
    "mq_mmq_fused": (lambda **kw: mq.mmq_fused(W, X, **kw), 2),
    "mq_mmq_fused_static": (lambda **kw: mq.mmq_fused_static(W, X, **kw), 1),
    "mq_mmq_blockdots": (lambda **kw: mq.mmq_blockdots(W, XQ, 3, **kw), 1),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("given", [False, True])
def test_one_stream_for_a_call_and_what_it_makes(record, name, given):
    call, makes = CALLS[name]
    call(**(dict(stream=types.SimpleNamespace(cuda_stream=OTHER)) if given else {}))
    assert [what for what, _ in record] == ["made"] * makes + [name]
    assert {stream for _, stream in record} == {OTHER if given else HERE}


@pytest.mark.parametrize("name,out", [("mq_matvec", dict(y=X)), ("mq_ffn_gu_matvec", dict(h=X)),
                                      ("mq_ffn_gu_mmq", dict(h=X)), ("mq_quantize_act", dict(xq=XQ)),
                                      ("mq_mmq", dict(y=X)), ("mq_mmq_fused", dict(xq=XQ, y=X)),
                                      ("mq_mmq_fused_static", dict(y=X)), ("mq_mmq_blockdots", dict(D=X))])
def test_what_the_caller_gives_is_used(record, name, out):
    CALLS[name][0](**out, stream=types.SimpleNamespace(cuda_stream=OTHER))
    assert record == [(name, OTHER)]


@pytest.mark.parametrize("call", [mq.matvec, mq.ffn_gu_matvec])
def test_a_strided_input_is_copied_on_the_stream(record, monkeypatch, call):
    """(the library reads rows that follow each other)"""
    seen = []

    class Strided:
        def reshape(self, *shape):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return X

        def is_contiguous(self):
            return False
        device = X.device
    call(W, Strided(), torch.ones((3, 64)), stream=types.SimpleNamespace(cuda_stream=OTHER))
    assert seen == [OTHER]
