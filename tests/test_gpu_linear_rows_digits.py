"""The linear of a few rows where single digits of x decide (GPU): elements far below the largest of their block and row."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import _digits_ref as D  # noqa: E402
import _token_ref as T  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from audio_dit_gb300 import build
    build.build()


# (one to four and five to eight rows of few and of many columns a CTA, and the three kernels' one and two passes)
@pytest.mark.parametrize("M,K", [(1, 512), (2, 1088), (3, 512), (4, 4096), (5, 512), (7, 1088), (8, 4096), (9, 512), (20, 1088),
                                 (33, 512), (64, 1024), (1, 65536 // 4)])
def test_elements_far_below_the_largest(M, K):
    import audio_dit_gb300 as A
    x, w = D.make(np.random.default_rng(1000 * M + K), M, K)
    w = torch.cat([w, w.new_zeros(-len(w) % 8, K)])
    N = len(w)
    wq = A.alloc_nvfp4(N, K)
    A.h3fp4_quantize_weight(w.cuda(), *wq, A.alloc_workspace(N, 0, K))
    out, ws = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), A.alloc_rows_workspace(M, N, K)
    A.h3fp4_linear_rows(x.cuda(), *wq, out, ws)
    A.h3fp4_check(ws)
    ref, tol = D.reference(x, T.decode_weight(*(t.cpu() for t in wq), K))
    err = (out.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), (int((~(err <= tol)).sum()), (~(err <= tol)).nonzero()[:3].tolist())
