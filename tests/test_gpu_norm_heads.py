"""Per-head norm (GPU) with head counts far from a warp's, against a plain 64-bit form."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import numpy as np  # noqa: E402

import _heads_ref as R  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from audio_dit_gb300 import build
    build.build()


@pytest.mark.parametrize("M,Hq,Hk,D,rot", [(1, 300_007, 5, 8, 0), (3, 6001, 2999, 16, 16), (2, 4999, 1, 136, 32),
                                           (5, 97, 95, 72, 64)])
def test_many_heads(M, Hq, Hk, D, rot):
    import audio_dit_gb300 as A
    rng = np.random.default_rng(Hq)
    q, k = R.rand_bf16(rng, M, Hq, D), R.rand_bf16(rng, M, Hk, D)
    w = torch.from_numpy(rng.uniform(-2, 2, (1, D)).astype(np.float32))
    a = torch.from_numpy(rng.uniform(-300.0, 300.0, (M, rot // 2)).astype(np.float32))
    cos, sin = (torch.cos(a), torch.sin(a)) if rot else (None, None)
    qo, ko = (torch.full_like(t, float("nan"), device="cuda") for t in (q, k))
    A.h3fp4_qk_norm_rope(q.cuda(), k.cuda(), qo, ko, q_weight=w.cuda(), cos=cos.cuda() if rot else None,
                         sin=sin.cuda() if rot else None)
    for got, x, weight in ((qo, q, w), (ko, k, None)):
        ref = R.norm_rope(x, weight, cos, sin, False, [0, M], 1e-6)
        off = (got.cpu().double() - ref).abs()
        assert bool((off <= R.norm_rope_bound(ref, rot // 2, False)).all())
