"""mq_rope_store of a single token with its queries written over the start of its row."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from tests.kv_cases import IO, KINDS  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["f16", "q8_0"])
@pytest.mark.parametrize("hq,hkv,dim,rot", [(28, 4, 128, 128), (5, 1, 96, 40), (71, 1, 64, 64)])
@pytest.mark.parametrize("pairs", [False, True])
def test_one_token(io, kind, hq, hkv, dim, rot, pairs):
    g = torch.Generator(device="cuda").manual_seed(hq)
    width = (hq + 2 * hkv) * dim
    row = torch.randn((1, width), device="cuda", generator=g).to(IO[io])
    bias = torch.randn(width, device="cuda", generator=g)
    rope = mq.Rope(mq.rope_table(50, [1e4 ** (-2 * i / rot) for i in range(rot // 2)]), pairs=pairs)
    pos = torch.full((1, 1), 33, dtype=torch.int32, device="cuda")
    slot = torch.tensor([5], device="cuda")
    caches = [mq.kv_cache(KINDS[kind], 1, 16, hkv, dim) for _ in range(2)]
    want = mq.rope_store(caches[0], rope, row, pos, slot, hq, bias=bias)
    qkv = row.clone()
    q = qkv[:, :hq * dim].view(1, hq, dim)
    got = mq.rope_store(caches[1], rope, qkv, pos, slot, hq, bias=bias, q=q)
    mq.stream_status()
    assert got is q and torch.equal(got, want) and torch.equal(qkv[:, hq * dim:], row[:, hq * dim:])
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
