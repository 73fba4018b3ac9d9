"""The linear of a few rows over NVFP4 weights (GPU) against a plain 64-bit form."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import _token_ref as T  # noqa: E402
from _gpu_helpers import Guarded  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from audio_dit_gb300 import build
    build.build()


def bits(t):
    return t.contiguous().view(torch.int16)


def cuda(t):
    return None if t is None else t.cuda()


def weight(rng, N, K):
    """Quantised on the GPU by the package: device (codes, sf, gscale) and the float64 values."""
    import audio_dit_gb300 as A
    w = torch.from_numpy((0.05 * rng.standard_normal((N, K))).astype(np.float32)).to(torch.bfloat16)
    wq, ws = A.alloc_nvfp4(N, K), A.alloc_workspace(N, 0, K)
    A.h3fp4_quantize_weight(w.cuda(), *wq, ws)
    return wq, T.decode_weight(*(t.cpu() for t in wq), K)


def bf(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).to(torch.bfloat16)


def activations(rng, M, K):
    """Rows with a few large channels, blocks of zeros and elements of very different sizes."""
    x = bf(rng, M, K) * torch.from_numpy(np.where(rng.random(K) < 0.02, 20.0, 1.0).astype(np.float32)).bfloat16()
    x[:, 16:32] = 0
    x[:, 33] *= 2.0 ** -12
    x[:, 40:44] *= 2.0 ** -20
    return x


def check(got, x, w, bias, gate, resid, swiglu, what):
    ref, tol = T.linear_rows(x, w, bias, gate, resid, swiglu)
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), (what, int((~(err <= tol)).sum()), (~(err <= tol)).nonzero()[:3].tolist(),
                                      float((err / tol).max()))


CASES = [  # M, N, K, bias, gate ("rows", "one" or None), swiglu
    (1, 8, 64, False, None, False),
    (1, 128, 256, True, None, False),
    (1, 9216, 3072, True, None, False),
    (1, 512, 4096, True, None, True),
    (2, 136, 320, False, "one", False),
    (3, 1000, 1088, True, "rows", False),
    (7, 256, 192, False, None, True),
    (8, 264, 512, True, None, False),
    (9, 128, 16384, False, None, False),
    (16, 4096, 1024, True, "rows", False),
    (17, 200, 704, True, "one", False),
    (31, 768, 2048, True, None, True),
    (32, 520, 640, False, "rows", False),
    (33, 384, 960, True, None, False),
    (48, 256, 128, False, None, True),
    (61, 6152, 448, True, "rows", False),
    (64, 1024, 1024, True, "rows", False),
    (64, 3072, 12288, True, "one", False),
    (5, 40000, 64, True, None, False),
    (4, 1024, 8192, True, "rows", False),                             # eight CTAs a tile, four stages each
    (8, 9216, 4096, False, None, False),                              # more stages than the ring has
    (6, 512, 14336, True, None, True),                                # gate and up tiles of four CTAs each
    (8, 128, 65536, False, "one", False),
    (2, 24, 1856, True, None, False),
    (3, 20480, 3072, True, "rows", False),                            # more tiles than a wave: the other form
    (1, 57344, 512, True, None, True),
    (16, 6144, 4096, True, "rows", False),
    (13, 1024, 14336, False, None, True),
    (9, 3000, 1984, True, "one", False),
    (12, 256, 65536, False, None, False),
    (1, 4096, 14336, True, None, False),                              # few rows, rings that are filled again and again
    (2, 4096, 14336, False, "rows", False),
    (3, 128, 65536, True, None, False),
    (1, 128, 65536, False, None, False),
    (2, 256, 65536, True, None, True),
    (1, 24576, 2560, False, "rows", False),                           # few rows, several tiles a CTA
    (2, 24576, 2112, True, None, True),
    (3, 40960, 1088, True, "one", False),
    (4, 49000, 64, True, None, False),
    (4, 28672, 1984, True, None, True),
    (64, 128, 256, True, "rows", False),                              # the most rows, one tile
    (40, 40000, 192, False, "one", False),                            # several tiles a CTA, two passes
    (21, 24320, 320, True, None, True),
    (32, 3080, 4160, True, "rows", False),
]


@pytest.mark.parametrize("M,N,K,with_bias,gated,swiglu", CASES)
def test_against_64_bits(M, N, K, with_bias, gated, swiglu):
    import audio_dit_gb300 as A
    rng = np.random.default_rng(M * 100000 + N + K)
    wq, w = weight(rng, N, K)
    x = activations(rng, M, K)
    bias = bf(rng, N) if with_bias else None
    gate = torch.from_numpy(rng.standard_normal((M, N) if gated == "rows" else (N,)).astype(np.float32)) if gated else None
    resid = bf(rng, M, N) if gated else None
    out = Guarded((M, N // 2 if swiglu else N), torch.bfloat16)
    n = A.h3fp4_linear_rows_workspace_bytes(M, N, K)
    ws = Guarded((n,), torch.uint8, zero=True)
    kw = dict(bias=cuda(bias), gate=cuda(gate), swiglu=swiglu)
    A.h3fp4_linear_rows(x.cuda(), *wq, out.t, ws.t, resid=cuda(resid), **kw)
    A.h3fp4_check(ws.t)
    out.check("out"), ws.check("ws")
    check(out.t, x, w, bias, gate, resid, swiglu, "out")
    # the same bits again, over a workspace that an earlier call left
    again = torch.empty_like(out.t) if resid is None else resid.cuda().clone()
    A.h3fp4_linear_rows(x.cuda(), *wq, again, ws.t, resid=None if resid is None else again, **kw)
    assert torch.equal(bits(again), bits(out.t))
    # a row's outputs do not depend on its neighbours
    one = torch.empty(1, out.t.shape[1], dtype=torch.bfloat16, device="cuda")
    g1 = gate if gate is None or gate.dim() == 1 else gate[M - 1:]
    A.h3fp4_linear_rows(x[M - 1:].cuda(), *wq, one, ws.t, bias=cuda(bias), gate=cuda(g1),
                        resid=None if resid is None else resid[M - 1:].cuda(), swiglu=swiglu)
    check(one, x[M - 1:], w, bias, g1, None if resid is None else resid[M - 1:], swiglu, "one row")
    A.h3fp4_check(ws.t)


def test_ranges_and_zero_rows():
    import audio_dit_gb300 as A
    rng = np.random.default_rng(3)
    M, N, K = 20, 256, 512
    wq, w = weight(rng, N, K)
    x = bf(rng, M, K) * torch.logspace(-30, 30, M).to(torch.bfloat16)[:, None]
    x[4] = 0
    x[5, 1:] = 0
    x[6] *= torch.from_numpy(np.exp2(rng.integers(-60, 0, (K // 16, 1))) * np.ones((1, 16))).flatten().bfloat16()
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ws = A.alloc_rows_workspace(M, N, K)
    A.h3fp4_linear_rows(x.cuda(), *wq, out, ws)
    A.h3fp4_check(ws)
    check(out, x, w, None, None, None, False, "ranges")
    assert not bool(out[4].any())


@pytest.mark.parametrize("M,N,K,swiglu", [(3, 256, 1024, False), (7, 512, 512, True), (20, 384, 2112, False), (40, 256, 320, True)])
def test_rows_that_are_not_finite(M, N, K, swiglu):
    """They are NaN, and the others have the bits that they have without them."""
    import audio_dit_gb300 as A
    torch.manual_seed(M)
    x, w = torch.randn(M, K, device="cuda").bfloat16(), (torch.randn(N, K, device="cuda") * 0.05).bfloat16()
    wq = A.alloc_nvfp4(N, K)
    A.h3fp4_quantize_weight(w, *wq, A.alloc_workspace(256, N, K))
    ws = A.alloc_rows_workspace(M, N, K)
    good, bad = (torch.empty(M, N // 2 if swiglu else N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.h3fp4_linear_rows(x, *wq, good, ws, swiglu=swiglu)
    x[0, K - 1], x[M - 1, 5], x[M // 2, 0] = float("nan"), float("inf"), float("-inf")
    A.h3fp4_linear_rows(x, *wq, bad, ws, swiglu=swiglu)
    A.h3fp4_check(ws)
    rest = [m for m in range(M) if m not in (0, M // 2, M - 1)]
    assert bool(bad[[0, M // 2, M - 1]].isnan().all()) and bool(good.isfinite().all())
    assert torch.equal(bad[rest].view(torch.int16), good[rest].view(torch.int16))


def test_captured():
    import audio_dit_gb300 as A
    rng = np.random.default_rng(4)
    M, N, K = 3, 1024, 1024
    wq, w = weight(rng, N, K)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    out, ws = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), A.alloc_rows_workspace(M, N, K)
    A.h3fp4_linear_rows(x, *wq, out, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.h3fp4_linear_rows(x, *wq, out, ws)
    for i in range(3):
        new = activations(rng, M, K)
        x.copy_(new)
        g.replay()
        check(out, new, w, None, None, None, False, i)
    A.h3fp4_check(ws)


def test_near_the_linear():
    """As the linear of quantised activations, but for that quantisation."""
    import audio_dit_gb300 as A
    rng = np.random.default_rng(5)
    M, N, K = 24, 512, 1024
    wq, _ = weight(rng, N, K)
    x, b = bf(rng, M, K).cuda(), bf(rng, N).cuda()
    one, two = (torch.empty(M, N // 2, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.h3fp4_linear_rows(x, *wq, one, A.alloc_rows_workspace(M, N, K), bias=b, swiglu=True)
    A.h3fp4_linear(x, *wq, two, A.alloc_workspace(M, N, K), bias=b, swiglu=True)
    assert float((one.float() - two.float()).norm() / one.float().norm()) < 0.25


def test_waits_that_run_out():
    import audio_dit_gb300 as A
    ws = A.alloc_rows_workspace(64, 128, 1024)
    A.h3fp4_selftest_linear_rows_timeout(ws, 1000000)
    with pytest.raises(A.H3FP4Error) as e:
        A.h3fp4_check(ws)
    assert e.value.status == 5
    A.h3fp4_check(ws)                                                 # read and cleared
