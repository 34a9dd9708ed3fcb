"""mq_attn_decode with its outputs written over the queries."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from tests.kv_cases import IO, Paged  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


@pytest.mark.parametrize("kind,io", [("f16", "f32"), ("bf16", "bf16"), ("q8_0", "f16")])
@pytest.mark.parametrize("lens,hq,hkv,dim", [([30000], 28, 4, 128), ([0, 900, 1, 5000, 33], 17, 1, 64),
                                             ([40 + 7 * i for i in range(50)], 20, 2, 256)])
def test_outputs_over_the_queries(kind, io, lens, hq, hkv, dim):
    """Units of one block and of several, joined in one and in two steps, several row groups."""
    p = Paged(kind, lens, hkv, dim, 16, seed=hq)
    q = torch.randn((len(lens), hq, dim), generator=torch.Generator().manual_seed(dim)).to(IO[io]).cuda()
    want = mq.attn_decode(p.cache, q, p.pages, p.lens, p.max_len)
    for _ in range(10):
        x = q.clone()
        assert mq.attn_decode(p.cache, x, p.pages, p.lens, p.max_len, o=x) is x
        assert torch.equal(x, want)
    mq.stream_status()
