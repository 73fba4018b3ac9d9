"""Attention (GPU) whose units last longer than the wait limit that is set: no wait runs out, since the limit grows with
a unit's length."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

LIMIT_NS = 100_000


@pytest.fixture(autouse=True)
def limit():
    from audio_dit_gb300 import build
    build.build()
    import audio_dit_gb300 as A
    yield lambda ns: A.h3fp4_set_wait_limit_ns(ns)
    A.h3fp4_set_wait_limit_ns(2_000_000_000)


def both(limit, *args, **kw):
    import audio_dit_gb300 as A
    got = []
    for ns in (2_000_000_000, LIMIT_NS):
        limit(ns)
        out = torch.full_like(args[0], float("nan"))
        A.h3fp4_cross_attn(*args[:3], out, args[3], **kw)
        A.h3fp4_check(args[3])
        got.append(out)
    assert torch.equal(got[0].view(torch.int16), got[1].view(torch.int16))
    return got[0]


def test_long_units(limit):
    """152 whole units of 512 tiles, about 0.6 ms each."""
    import audio_dit_gb300 as A
    g = torch.Generator(device="cuda").manual_seed(1)
    M, T = 152 * 256, 65536
    q, k, v = (torch.randn(n, 1, 8, generator=g, device="cuda").bfloat16() for n in (M, T, T))
    out = both(limit, q, k, v, A.alloc_attn_workspace(M, T, 1, 1, 8))
    some = slice(0, M, 4999)
    ref = torch.softmax(q[some, 0].double() @ k[:, 0].double().T * 8 ** -0.5, -1) @ v[:, 0].double()
    assert float((out[some, 0].double() - ref).norm() / ref.norm()) < 0.01


def test_long_masked_end(limit):
    """A mask that keeps the first key of two million: looking for it takes milliseconds."""
    import audio_dit_gb300 as A
    T = 1 << 21
    q, k, v = (torch.ones(n, 1, 8, dtype=torch.bfloat16, device="cuda") for n in (1, T, T))
    v[1:] = float("nan")
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    mask[0] = True
    out = both(limit, q, k, v, A.alloc_attn_workspace(1, T, 1, 1, 8), key_mask=mask)
    assert bool((out == 1.0).all())
