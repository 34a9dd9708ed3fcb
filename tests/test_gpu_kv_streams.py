"""The paged cache's calls on a stream that is not the current one, which has work of its own:
results are those of calls on the current stream, bit for bit."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from tests.kv_cases import Paged  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def busy(a, n=30):
    """Some milliseconds of work on the current stream."""
    for _ in range(n):
        a = a @ a
    return a


def test_calls_beside_work_of_the_current_stream():
    """Outputs and workspace of the calls' own, made again and again beside that work and beside
    allocations of the current stream that take up what is released."""
    lens = [5000, 7, 1200, 0]
    p = Paged("f16", lens, 2, 64, 16, sums=True, seed=1, spare=40)
    g = torch.Generator().manual_seed(2)
    q = torch.randn((4, 8, 64), generator=g).cuda()
    qkv = torch.randn((9, 12 * 64), generator=g).cuda()
    rope = mq.Rope(mq.rope_table(50, [1.0] * 32))
    pos = torch.arange(9, dtype=torch.int32, device="cuda").view(1, 9)
    slot = torch.arange(9, device="cuda") + p.free[39] * 16
    new = torch.tensor(p.free[:32], dtype=torch.int32, device="cuda").view(4, 8)

    def calls(**kw):
        return (mq.attn_decode(p.cache, q, p.pages, p.lens, p.max_len, **kw),
                mq.rope_store(p.cache, rope, qkv, pos, slot, 8, **kw),
                *mq.kv_evict(p.cache, p.pages, p.lens, p.max_len, new, 128, 4, 16, **kw))
    ref = calls()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    a = torch.randn((4096, 4096), device="cuda", dtype=torch.bfloat16) / 64
    size = mq.attn_workspace(p.cache, 4, 8, p.max_len).numel()
    for _ in range(5):
        busy(a)
        out = []
        for _ in range(10):
            out.append(calls(stream=st))
            torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for got in out:
            assert all(torch.equal(x, y) for x, y in zip(got, ref))
    mq.stream_status()
