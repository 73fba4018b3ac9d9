"""The linear of a few rows at the ends of fp32's range, in each of its forms (GPU)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import _token_ref as T  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from audio_dit_gb300 import build
    build.build()


def weight(rng, N, K, size):
    import audio_dit_gb300 as A
    w = torch.from_numpy((size * rng.standard_normal((N, K))).astype(np.float32)).to(torch.bfloat16)
    wq = A.alloc_nvfp4(N, K)
    A.h3fp4_quantize_weight(w.cuda(), *wq, A.alloc_workspace(N, 0, K))
    return wq, T.decode_weight(*(t.cpu() for t in wq), K)


def check(got, ref, tol, what):
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), (what, int((~(err <= tol)).sum()), (~(err <= tol)).nonzero()[:3].tolist())


# Rows and weights at opposite ends of the range: the outputs fit bf16, what is multiplied on the way there need not.
@pytest.mark.parametrize("rows,weights", [(1e35, 0.05), (1e37, 0.05), (1e37, 1e-30), (1e-36, 1e33), (1e-30, 1e36), (1e-36, 0.05)])
@pytest.mark.parametrize("M", [1, 2, 4, 5, 8, 20, 64])
def test_finite_rows_give_finite_outputs(M, rows, weights):
    import audio_dit_gb300 as A
    rng = np.random.default_rng(M)
    N, K = 256, 1024
    wq, w = weight(rng, N, K, weights)
    x = torch.from_numpy((rows * rng.standard_normal((M, K))).astype(np.float32)).to(torch.bfloat16)
    bias = torch.from_numpy((rows * weights * rng.standard_normal(N)).astype(np.float32)).to(torch.bfloat16)
    out, ws = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), A.alloc_rows_workspace(M, N, K)
    for b in (None, bias):
        A.h3fp4_linear_rows(x.cuda(), *wq, out, ws, bias=None if b is None else b.cuda())
        A.h3fp4_check(ws)
        ref, tol = T.linear_rows(x, w, b, None, None, False)
        assert float(ref.abs().max()) < 3e38
        check(out, ref, tol, (rows, weights, b is None))
