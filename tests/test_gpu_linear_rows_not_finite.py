"""Single rows of the linear of a few rows that are not finite, in each of its forms (GPU)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


@pytest.fixture(scope="module", autouse=True)
def built():
    from audio_dit_gb300 import build
    build.build()


@pytest.mark.parametrize("M,N,K,swiglu", [(2, 256, 4096, False), (4, 512, 8192, True), (4, 128, 1024, False), (8, 256, 4096, False),
                                          (3, 40960, 512, False), (20, 256, 4096, False), (64, 512, 1024, True)])
def test_one_row_that_is_not_finite(M, N, K, swiglu):
    """It is NaN, wherever the element stands, and the others have the bits that they have without it."""
    import audio_dit_gb300 as A
    torch.manual_seed(M)
    x, w = torch.randn(M, K, device="cuda").bfloat16(), (torch.randn(N, K, device="cuda") * 0.05).bfloat16()
    wq = A.alloc_nvfp4(N, K)
    A.h3fp4_quantize_weight(w, *wq, A.alloc_workspace(N, 0, K))
    ws = A.alloc_rows_workspace(M, N, K)
    good, bad = (torch.empty(M, N // 2 if swiglu else N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.h3fp4_linear_rows(x, *wq, good, ws, swiglu=swiglu)
    assert bool(good.isfinite().all())
    for m, k, v in ((0, 0, "nan"), (M - 1, K - 1, "inf"), (M // 2, K // 2 + 5, "-inf")):
        y = x.clone()
        y[m, k] = float(v)
        A.h3fp4_linear_rows(y, *wq, bad, ws, swiglu=swiglu)
        rest = [i for i in range(M) if i != m]
        assert rest and bool(bad[m].isnan().all()), (m, k)
        assert torch.equal(bad[rest].view(torch.int16), good[rest].view(torch.int16)), (m, k)
    A.h3fp4_check(ws)
