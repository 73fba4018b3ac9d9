"""Attention (GPU) with scores at the ends of fp32's range: past it a row is NaN, and never taken for one without a key."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import _heads_ref as R  # noqa: E402
from test_gpu_attn import Case, built  # noqa: E402,F401

SIZES = [([0, 3], [0, 200], 0, 2, 2, 64), ([0, 300], [0, 900], 0, 24, 24, 128), ([0, 1], [0, 20000], 0, 8, 2, 128),
         ([0, *range(1, 41)], [5 * i for i in range(41)], 9000, 4, 4, 64)]


@pytest.mark.parametrize("q_off,kv_off,ctx,Hq,Hkv,D", SIZES)
def test_scores_past_the_range(q_off, kv_off, ctx, Hq, Hkv, D):
    """q.k = 2^127 is finite, times 2 log2(e) it is not; the other rows are right."""
    c = Case(5, Hq, Hkv, D, q_off, kv_off, ctx=ctx, scale=2.0)
    c.q[..., 0] = 0
    far = c.M - 1
    c.q[far] = 0
    c.q[far, :, 0] = 2.0 ** 63
    for k in (c.k, c.kc):
        if k is not None:
            k[..., 0] = 2.0 ** 64
    out, lse = c.run()
    assert bool(torch.isnan(out[far]).all()) and not bool(torch.isneginf(lse[far]).any())
    ref = R.attention(c.q, c.k, c.v, q_off, kv_off, c.scale, None, c.kc, c.vc)
    tol, tol_lse = R.attention_bounds(*ref, D)
    assert bool(((out.double() - ref[0]).abs() <= tol)[:far].all())
    assert bool(((lse.double() - ref[1]).abs() <= tol_lse)[:far].all())


@pytest.mark.parametrize("q_off,kv_off,ctx,Hq,Hkv,D", SIZES)
def test_largest_scores_within_the_range(q_off, kv_off, ctx, Hq, Hkv, D):
    """One key scores 2^126 and has all the weight."""
    c = Case(6, Hq, Hkv, D, q_off, kv_off, ctx=ctx, scale=1.0)
    far = c.M - 1
    c.q[far] = 0
    c.q[far, :, 0] = 2.0 ** 63
    for k in (c.k, c.kc):
        if k is not None:
            k[..., 0] = 0
    c.k[kv_off[-1] - 1, :, 0] = 2.0 ** 63
    out, lse = c.run()
    want = c.v[kv_off[-1] - 1].repeat_interleave(Hq // Hkv, 0)
    assert torch.equal(out[far].view(torch.int16), want.view(torch.int16))
    assert bool(((lse[far].double() - 2.0 ** 126).abs() <= 2.0 ** (126 - 22)).all())
