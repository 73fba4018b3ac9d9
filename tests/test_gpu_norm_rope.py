"""Per-head norm with rotation (GPU) against a plain 64-bit form."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import _heads_ref as R  # noqa: E402
from _gpu_helpers import Guarded  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from audio_dit_gb300 import build
    build.build()


def angles(rng, M, half):
    if not half:
        return None, None
    a = torch.from_numpy(rng.uniform(-300.0, 300.0, (M, half)).astype(np.float32))
    return torch.cos(a), torch.sin(a)


def cuda(t):
    return None if t is None else t.cuda()


def check(got, x, w, cos, sin, pairs, off, eps, what):
    ref = R.norm_rope(x, w, cos, sin, pairs, off, eps)
    bad = (got.cpu().double() - ref).abs() > R.norm_rope_bound(ref, 0 if cos is None else cos.shape[1], pairs)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:3].tolist())


CASES = [  # M, Hq, Hk, D, rot, pairs, offsets, weights
    (1, 24, 24, 128, 128, False, None, True),
    (5, 24, 8, 128, 128, True, [0, 5], True),
    (257, 24, 24, 128, 64, False, [0, 200, 257], True),
    (300, 20, 5, 80, 48, True, [0, 0, 299, 300], True),
    (300, 7, 1, 80, 80, False, [0, 100, 100, 300], True),
    (33, 3, 3, 8, 0, False, None, True),
    (33, 5, 2, 16, 16, False, None, True),
    (33, 5, 2, 16, 16, True, None, False),
    (40, 2, 1, 24, 16, False, None, True),
    (40, 2, 1, 24, 16, True, None, True),
    (65, 4, 2, 256, 256, False, [0, 1, 2, 3, 4, 5, 6, 7, 65], True),
    (65, 4, 2, 256, 176, True, None, False),
    (19, 9, 3, 232, 112, False, None, True),
    (19, 1, 1, 40, 32, False, None, True),
    (1030, 16, 4, 64, 64, False, [0, 1029, 1030], True),
]


@pytest.mark.parametrize("M,Hq,Hk,D,rot,pairs,off,weights", CASES)
def test_against_64_bits(M, Hq, Hk, D, rot, pairs, off, weights):
    import audio_dit_gb300 as A
    rng = np.random.default_rng(M * 1000 + D + rot)
    # strided views of one interleaved buffer in, guarded contiguous outputs
    qkv = R.rand_bf16(rng, M, Hq + 2 * Hk, D, scale=3.0)
    nseg = 1 if off is None else len(off) - 1
    w = [torch.from_numpy(rng.uniform(-2, 2, (nseg, D)).astype(np.float32)) if weights else None for _ in range(2)]
    cos, sin = angles(rng, M, rot // 2)
    dev = qkv.cuda()
    qo, ko = Guarded((M, Hq, D), torch.bfloat16), Guarded((M, Hk, D), torch.bfloat16)
    kw = dict(q_weight=cuda(w[0]), k_weight=cuda(w[1]), cos=cuda(cos), sin=cuda(sin), interleaved=pairs, seg_off=off,
              eps=1e-5)
    A.h3fp4_qk_norm_rope(dev[:, :Hq], dev[:, Hq:Hq + Hk], qo.t, ko.t, **kw)
    qo.check("q"), ko.check("k")
    table = off or [0, M]
    check(qo.t, qkv[:, :Hq], w[0], cos, sin, pairs, table, 1e-5, "q")
    check(ko.t, qkv[:, Hq:Hq + Hk], w[1], cos, sin, pairs, table, 1e-5, "k")
    # in place on the views: the same bits, and the values beside them untouched
    A.h3fp4_qk_norm_rope(dev[:, :Hq], dev[:, Hq:Hq + Hk], dev[:, :Hq], dev[:, Hq:Hq + Hk], **kw)
    assert torch.equal(dev[:, :Hq].contiguous().view(torch.int16), qo.t.view(torch.int16))
    assert torch.equal(dev[:, Hq:Hq + Hk].contiguous().view(torch.int16), ko.t.view(torch.int16))
    assert torch.equal(dev[:, Hq + Hk:].cpu().view(torch.int16), qkv[:, Hq + Hk:].view(torch.int16))
    # the queries alone
    one = torch.empty_like(qo.t)
    A.h3fp4_qk_norm_rope(qkv.cuda()[:, :Hq], None, one, None, **{**kw, "k_weight": None})
    assert torch.equal(one.view(torch.int16), qo.t.view(torch.int16))


def test_head_major_layout_and_zero_rows():
    import audio_dit_gb300 as A
    rng = np.random.default_rng(5)
    M, H, D = 37, 6, 64
    x = R.rand_bf16(rng, M, H, D)
    x[3] = 0
    x[4, 2] = 0
    xt = x.transpose(0, 1).contiguous().cuda().transpose(0, 1)     # stored [H][M][D]
    out = torch.full((H, M, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    A.h3fp4_qk_norm_rope(xt, None, out, None, eps=1e-6)
    check(out, x, None, None, None, False, [0, M], 1e-6, "head-major")
    assert not bool(out[3].any())
    none = torch.empty(0, H, D, dtype=torch.bfloat16, device="cuda")
    A.h3fp4_qk_norm_rope(none, None, none, None)                    # no rows: nothing to do


def test_wide_range_of_magnitudes():
    import audio_dit_gb300 as A
    rng = np.random.default_rng(6)
    x = R.rand_bf16(rng, 64, 4, 128) * torch.logspace(-15, 15, 64).to(torch.bfloat16)[:, None, None]
    out = torch.empty_like(x, device="cuda")
    A.h3fp4_qk_norm_rope(x.cuda(), None, out, None, eps=1e-12)
    check(out, x, None, None, None, False, [0, 64], 1e-12, "magnitudes")


def test_offsets_past_32_bits():
    import audio_dit_gb300 as A
    rng = np.random.default_rng(7)
    M, step = 40, 1 << 27                                           # element offsets up to 5.2e9
    big = torch.empty(M * step, dtype=torch.bfloat16, device="cuda")
    view = big.as_strided((M, 2, 64), (step, 64, 1))
    x = R.rand_bf16(rng, M, 2, 64)
    view.copy_(x)
    A.h3fp4_qk_norm_rope(view, None, view, None, eps=1e-6)
    check(view, x, None, None, None, False, [0, M], 1e-6, "far rows")


def test_side_stream_and_graph():
    import audio_dit_gb300 as A
    rng = np.random.default_rng(8)
    x = R.rand_bf16(rng, 500, 8, 128).cuda()
    cos, sin = (t.cuda() for t in angles(rng, 500, 64))
    want = torch.empty_like(x)
    A.h3fp4_qk_norm_rope(x, None, want, None, cos=cos, sin=sin)
    got = torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    A.h3fp4_qk_norm_rope(x, None, got, None, cos=cos, sin=sin, stream=side)
    side.synchronize()
    assert torch.equal(want.view(torch.int16), got.view(torch.int16))
    got.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.h3fp4_qk_norm_rope(x, None, got, None, cos=cos, sin=sin)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(want.view(torch.int16), got.view(torch.int16))
