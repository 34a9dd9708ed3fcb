"""mq_attn_decode where sequences of one call share pages: several new tokens of one sequence, as
entries with the same pages and lengths of their own, and sequences with a common beginning."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quantized_q4_gb300 as mq  # noqa: E402
from gguf_block_quantized_q4_gb300 import build as mqbuild  # noqa: E402
from oracle import kv  # noqa: E402
from tests.kv_cases import Paged, attn_bound  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mqbuild.build()
    mq.init(0)
    yield


def check(p, rows, lens, hq, dim, window=0):
    """rows: the page table, by sequence of p or as lists of pages."""
    table = np.stack([p.pages_host[r] if isinstance(r, int) else r for r in rows])
    q = torch.randn((len(rows), hq, dim), generator=torch.Generator().manual_seed(hq))
    o = mq.attn_decode(p.cache, q.cuda(), torch.from_numpy(table).cuda(),
                       torch.tensor(lens, dtype=torch.int32, device="cuda"), p.max_len, window=window)
    mq.stream_status()
    ref, mass, reach, _ = kv.attn_decode(p.host, p.page_size, q.numpy(), table, lens, dim ** -0.5, window)
    assert (np.abs(o.cpu().numpy() - ref) <= attn_bound(dim, reach, mass, ref, "f32")).all()


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("hq,hkv,dim", [(8, 8, 128), (32, 8, 128), (14, 2, 64), (6, 1, 256)])
@pytest.mark.parametrize("window", [0, 50])
def test_several_tokens_of_each_sequence(kind, hq, hkv, dim, window):
    """Four tokens each, the last four lengths (for the short one: from none on)."""
    p = Paged(kind, [700, 3, 130], hkv, dim, 16, seed=hq)
    rows = [s for s in range(3) for _ in range(4)]
    check(p, rows, [n - 3 + i for n in p.lens_list for i in range(4)], hq, dim, window)


@pytest.mark.parametrize("kind", ["f16", "q8_0"])
def test_several_tokens_of_a_long_sequence(kind):
    """Units of the same rows in one block and in several; more tokens than a row group's rows."""
    p = Paged(kind, [30001], 2, 128, 64, seed=1)
    check(p, [0] * 9, list(range(30001 - 8, 30002)), 4, 128)
    check(p, [0] * 40, list(range(1, 30001, 751)), 4, 128)


def test_sequences_with_a_common_beginning():
    p = Paged("f16", [200, 200, 300], 2, 128, 16, seed=2)
    first = p.pages_host[2][:6]  # 96 positions of the third sequence, then each its own
    rows = [np.concatenate([first, p.pages_host[s][6:13], p.pages_host[s][:6]]) for s in (0, 1)]
    check(p, [*rows, 2], [200, 187, 300], 8, 128)
    check(p, [*rows, 2], [96, 97, 95], 8, 128, window=96)
