"""Per-head norm (GPU): comparisons that a NaN fails, and the rows that are NaN by the formula."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import numpy as np  # noqa: E402

import _heads_ref as R  # noqa: E402
from _norm_check import within  # noqa: E402
from test_gpu_norm_rope import CASES, angles, built, cuda  # noqa: E402,F401


@pytest.mark.parametrize("M,Hq,Hk,D,rot,pairs,off,weights", CASES)
def test_no_place_is_nan_or_far_off(M, Hq, Hk, D, rot, pairs, off, weights):
    import audio_dit_gb300 as A
    rng = np.random.default_rng(M * 999 + D + rot)
    nseg = 1 if off is None else len(off) - 1
    x = [R.rand_bf16(rng, M, h, D, scale=3.0) for h in (Hq, Hk)]
    w = [torch.from_numpy(rng.uniform(-2, 2, (nseg, D)).astype(np.float32)) if weights else None for _ in x]
    cos, sin = angles(rng, M, rot // 2)
    y = [torch.full_like(t, float("nan"), device="cuda") for t in x]
    A.h3fp4_qk_norm_rope(x[0].cuda(), x[1].cuda(), *y, q_weight=cuda(w[0]), k_weight=cuda(w[1]), cos=cuda(cos),
                         sin=cuda(sin), interleaved=pairs, seg_off=off, eps=1e-5)
    for got, t, weight in zip(y, x, w):
        ref = R.norm_rope(t, weight, cos, sin, pairs, off or [0, M], 1e-5)
        assert within(got.cpu(), ref, R.norm_rope_bound(ref, rot // 2, pairs))


def test_magnitudes_and_far_rows():
    import audio_dit_gb300 as A
    rng = np.random.default_rng(6)
    x = R.rand_bf16(rng, 64, 4, 128) * torch.logspace(-15, 15, 64).to(torch.bfloat16)[:, None, None]
    out = torch.full_like(x, float("nan"), device="cuda")
    A.h3fp4_qk_norm_rope(x.cuda(), None, out, None, eps=1e-12)
    ref = R.norm_rope(x, None, None, None, False, [0, 64], 1e-12)
    assert within(out.cpu(), ref, R.norm_rope_bound(ref, 0, False))
    step = 1 << 27                                                  # element offsets up to 5.2e9
    far = torch.empty(40 * step, dtype=torch.bfloat16, device="cuda").as_strided((40, 2, 64), (step, 64, 1))
    x = R.rand_bf16(rng, 40, 2, 64)
    far.copy_(x)
    A.h3fp4_qk_norm_rope(far, None, far, None, eps=1e-6)
    ref = R.norm_rope(x, None, None, None, False, [0, 40], 1e-6)
    assert within(far.cpu(), ref, R.norm_rope_bound(ref, 0, False))


@pytest.mark.parametrize("D,rot", [(128, 64), (80, 80), (8, 0)])
def test_zero_rows_without_eps_are_nan_and_nothing_else(D, rot):
    """0 * rsqrt(0) is NaN, as the formula has it: in the heads that are zero, and in no other."""
    import audio_dit_gb300 as A
    rng = np.random.default_rng(D)
    x = R.rand_bf16(rng, 37, 5, D)
    x[3] = 0
    x[7, 2] = 0
    cos, sin = angles(rng, 37, rot // 2)
    out = torch.zeros_like(x, device="cuda")
    A.h3fp4_qk_norm_rope(x.cuda(), None, out, None, cos=cuda(cos), sin=cuda(sin), eps=0.0)
    ref = R.norm_rope(x, None, cos, sin, False, [0, 37], 0.0)
    zero = (x == 0).all(-1)
    assert torch.equal(torch.isnan(out.cpu()).all(-1), zero) and torch.equal(torch.isnan(out.cpu()).any(-1), zero)
    assert within(out.cpu()[~zero], ref[~zero], R.norm_rope_bound(ref, rot // 2, False)[~zero])
