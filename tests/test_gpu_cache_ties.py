"""Block scales of the 4-bit cache where the product with the rounded sixth and the quotient part (GPU)."""
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


def test_scales_of_a_largest_over_2688():
    """Global scales amax / 2688, as calibration gives them, of the mantissas of amax that put block maxima on ties of E4M3."""
    import audio_dit_gb300 as A
    tops = torch.tensor([m * 2.0 ** (e - 7) for e in range(-6, 2) for m in range(128, 256)])
    k = torch.stack([tops * f for f in (1.0, -0.75, 0.5, 0.25) * 4], -1).bfloat16()[:, None].expand(-1, 4, -1).contiguous()
    s = torch.tensor([1.09375, 1.203125, 1.53125, 1.75]) / torch.tensor(2688.0)
    top = k.float().abs().amax(-1)
    code = lambda x: (x / s).clamp(max=448.0).to(torch.float8_e4m3fn).float()  # noqa: E731
    assert bool((code(top * torch.tensor(1.0 / 6.0)) != code(torch.div(top, torch.tensor(6.0)))).any(0).all())
    n = len(k)
    cache = A.alloc_kv_cache(n // 16, 4, 16, 16)
    table = torch.arange(n // 16, dtype=torch.int32, device="cuda")[None]
    length, off = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    g = dict(k_gscale=s.cuda(), v_gscale=s.flip(0).cuda())
    A.h3fp4_cache_append(k.cuda(), k.cuda(), cache, table, length, off, **g)
    ko, vo = (torch.empty(n, 4, 16, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.h3fp4_cache_read(ko, vo, cache, table, length, off, **g)
    for got, scale in ((ko, s), (vo, s.flip(0))):
        assert torch.equal(got.cpu().view(torch.int16), T.held(k, scale)[1].contiguous().view(torch.int16))
