"""The cache attention at the ends of its sizes (GPU)."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def built():
    from audio_dit_gb300 import build
    build.build()


def test_rows_of_2_to_the_34_elements_that_see_nothing():
    """One row of 2^26 heads of 256: its vectors of 16 bytes are 2^31, one more than 32 bits hold."""
    import audio_dit_gb300 as A
    Hq, D = 1 << 26, 256
    q = torch.zeros(8 * Hq + D, dtype=torch.bfloat16, device="cuda").as_strided((1, Hq, D), (8 * Hq, 8, 1))
    out = torch.ones(1, Hq, D, dtype=torch.bfloat16, device="cuda")   # 34 GB
    lse = torch.zeros(1, Hq, device="cuda")
    cache = A.alloc_kv_cache(1, 1, D, 16)
    table, length = (torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((1, 1), (1,)))
    ws = A.alloc_cache_attn_workspace(1, 1, Hq, 1, D)
    A.h3fp4_cache_attn(q, cache, table, length, out, ws, lse=lse)
    A.h3fp4_check(ws)
    assert not any(bool(part.any()) for part in out.view(-1).split(1 << 30))
    assert bool((lse == -math.inf).all())
