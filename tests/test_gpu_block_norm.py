"""The norms around a block (GPU) against a plain 64-bit form."""
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


def cuda(t):
    return None if t is None else t.cuda()


def bits(t):
    return t.contiguous().view(torch.int16)


def check(got, ref, tol, what):
    bad = ~((got.cpu().double() - ref).abs() <= tol)                # (a NaN is bad)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:3].tolist())


def inputs(M, K, off, y, post, parts, seed):
    rng = np.random.default_rng(seed)
    n = len(off) - 1
    bf = lambda: torch.from_numpy(rng.standard_normal((M, K), dtype=np.float32)).to(torch.bfloat16)  # noqa: E731
    vec = lambda on, m: torch.from_numpy((m + 0.5 * rng.standard_normal((n, K))).astype(np.float32)) if on else None  # noqa: E731
    return dict(x=bf() * 3 + 1, y=bf() if y else None, y_weight=vec(post and "y_weight" in parts, 1),
                gate=vec(y and "gate" in parts, 0), weight=vec("weight" in parts, 1), shift=vec("shift" in parts, 0),
                scale=vec("scale" in parts, 0))


ALL = ("y_weight", "gate", "weight", "shift", "scale")
CASES = [  # M, K, offsets, y, post, layer, vectors
    (1, 8, None, False, False, False, ()),
    (1, 3072, None, True, True, False, ALL),
    (3, 16, [0, 1, 1, 3], True, False, True, ALL),
    (131, 256, [0, 130, 131], True, True, True, ALL),
    (70, 264, None, True, False, False, ("gate",)),
    (70, 520, [0, 70], False, False, True, ("shift", "scale")),
    (33, 1024, None, True, True, False, ("y_weight", "weight")),
    (33, 1032, None, True, True, False, ("gate", "shift")),
    (9, 2056, [0, 4, 9], True, True, True, ALL),
    (300, 3072, [0, 200, 300], True, False, True, ("gate", "shift", "scale")),
    (5, 3080, None, False, False, False, ("weight",)),
    (5, 4104, None, True, True, True, ALL),
    (3, 8192, None, True, False, True, ("scale",)),
    (3, 8200, None, True, True, False, ALL),
    (2, 16392, [0, 0, 1, 2], True, True, True, ALL),
    (2, 32768, None, True, True, True, ALL),
    (2000, 64, [0, 1, 2, 3, 4, 5, 6, 7, 2000], True, True, False, ALL),
    (1501, 72, [0, 1500, 1501], True, False, True, ALL),
    (1027, 128, None, False, False, False, ("scale",)),
    # many rows: the vectors kept, or read for each row
    (1024, 520, [0, 1, 700, 701, 1024], True, True, True, ALL),
    (1100, 1024, None, False, False, True, ("shift", "scale")),
    (1500, 3072, [0, 3, 900, 1500], True, True, False, ALL),
    (1025, 4096, [0, 1024, 1025], True, False, True, ("gate", "shift", "scale")),
    (1300, 5192, [0, 600, 600, 1300], True, True, True, ALL),
    (1024, 8192, None, True, True, False, ("y_weight", "weight")),
    (1030, 8200, [0, 1029, 1030], True, True, True, ALL),
    (1024, 16384, [0, 1023, 1024], True, True, True, ALL),
    (1024, 16392, None, True, False, False, ("gate", "weight")),
    (300, 8200, [0, 299, 300], True, True, True, ALL),
    (97, 72, [0, 5, 97], True, True, False, ALL),
    (1001, 136, None, True, False, True, ("gate", "scale")),
    (70001, 264, [0, 33, 70001], True, True, False, ALL),
    (33, 8200, None, False, False, False, ("weight",)),
]


@pytest.mark.parametrize("M,K,off,y,post,layer,parts", CASES)
def test_against_64_bits(M, K, off, y, post, layer, parts):
    import audio_dit_gb300 as A
    at = off or [0, M]
    i = inputs(M, K, at, y, post, parts, M + K)
    kw = dict(x_scale=0.75, eps=1e-5)
    ref, x_ref, tol, x_tol = T.block_norm(*(i[n] for n in ("x", "y", "y_weight", "gate")), 0.75, i["weight"], i["shift"],
                                          i["scale"], at, 1e-5, post, layer)
    d = {n: cuda(v) for n, v in i.items()}
    x = d.pop("x")
    out, x_out, amax = Guarded((M, K), torch.bfloat16), Guarded((M, K), torch.bfloat16), Guarded((1,), torch.float32)
    kw.update(d, seg_off=off, post_norm=post, layer_norm=layer)
    A.h3fp4_block_norm(x, out.t, x_out=x_out.t if y else None, out_amax=amax.t, **kw)
    for b in (out, x_out, amax):
        b.check()
    check(out.t, ref, tol, "out")
    assert float(amax.t) == float(out.t.float().abs().max())
    if y:
        check(x_out.t, x_ref, x_tol, "x_out")
        # the residual alone, and in place: the same bits
        if not (layer or i["weight"] is not None or i["shift"] is not None or i["scale"] is not None):
            alone = torch.empty_like(x)
            A.h3fp4_block_norm(x, x_out=alone, **{**kw})
            assert torch.equal(bits(alone), bits(x_out.t))
        x2, y2 = x.clone(), d["y"].clone()
        A.h3fp4_block_norm(x2, y2, x_out=x2, **{**kw, "y": y2})
        assert torch.equal(bits(x2), bits(x_out.t)) and torch.equal(bits(y2), bits(out.t))
    else:
        x2 = x.clone()
        A.h3fp4_block_norm(x2, x2, **kw)
        assert torch.equal(bits(x2), bits(out.t))


def test_offsets_past_32_bits():
    import audio_dit_gb300 as A
    M, K = 66000, 32768                                             # 2.16e9 elements
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(3)
    some = torch.from_numpy(rng.standard_normal((2, K), dtype=np.float32)).to(torch.bfloat16)
    x[0], x[-1] = some[0].cuda(), some[1].cuda()
    amax = torch.full((1,), -1.0, device="cuda")
    A.h3fp4_block_norm(x, x, eps=1e-5, out_amax=amax)
    ref, _, tol, _ = T.block_norm(some, None, None, None, 1.0, None, None, None, [0, 2], 1e-5, False, False)
    check(torch.stack([x[0], x[-1]]), ref, tol, "first and last row")
    assert not bool(x[1:-1:997].any()) and float(amax) == float(x[[0, -1]].float().abs().max())


def test_no_rows_large_means_and_nan():
    import audio_dit_gb300 as A
    none = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    amax = torch.full((1,), 5.0, device="cuda")
    A.h3fp4_block_norm(none, none, out_amax=amax)
    assert float(amax) == 0.0
    # layer norm of values far from zero: the variance is about the mean
    rng = np.random.default_rng(4)
    x = (torch.from_numpy(rng.standard_normal((40, 512), dtype=np.float32)) + 200).to(torch.bfloat16)
    out = torch.empty_like(x, device="cuda")
    A.h3fp4_block_norm(x.cuda(), out, layer_norm=True, eps=0.0)
    ref, _, tol, _ = T.block_norm(x, None, None, None, 1.0, None, None, None, [0, 40], 0.0, False, True)
    check(out, ref, tol, "large mean")
    # zeros: zero, or (eps = 0) NaN as the formula gives; the other rows are not touched by it, max|out| is
    x[3] = 0
    for eps in (1e-6, 0.0):
        A.h3fp4_block_norm(x.cuda(), out, eps=eps, out_amax=amax)
        assert bool((out[3] == 0).all()) if eps else bool(out[3].isnan().all())
        assert bool(out[[0, 1, 2, 4]].isfinite().all()) and bool(amax.isnan()) == (eps == 0)


def test_largest_of_rows_in_place():
    """Rows that do not fill a block, in place: r = y - x here, and y - r is x, whose norm has a far larger element."""
    import audio_dit_gb300 as A
    for M, K in ((1, 64), (3, 64), (17, 64), (5, 128), (9, 256), (2, 512)):
        x0 = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
        x0[:, 3] = 1
        y, out, amax = torch.ones_like(x0), torch.empty_like(x0), torch.empty(1, device="cuda")
        for _ in range(50):
            x = x0.clone()
            A.h3fp4_block_norm(x, out, y=y, x_out=x, x_scale=-1.0, out_amax=amax)
            assert float(amax) == float(out.float().abs().max()) < 2


def test_feeds_the_linear():
    """Norm with max|out|, its scale, and the linear in one pass: the same bits as the two-pass quantisation."""
    import audio_dit_gb300 as A
    M, N, K = 300, 256, 512
    i = inputs(M, K, [0, 100, 300], True, True, ALL, 11)
    d = {n: cuda(v) for n, v in i.items()}
    x = d.pop("x")
    wq, ws = A.alloc_nvfp4(N, K), A.alloc_workspace(M, N, K)
    A.h3fp4_quantize_weight((torch.randn(N, K, device="cuda") * 0.02).bfloat16(), *wq, ws)
    h, amax, gs = torch.empty_like(x), torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    A.h3fp4_block_norm(x, h, x_out=x, seg_off=[0, 100, 300], post_norm=True, layer_norm=True, out_amax=amax, **d)
    A.h3fp4_gscale_from_amax(amax, gs)
    one, two = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.h3fp4_linear(h, *wq, one, ws, a_gscale=gs, gscale_given=True)
    A.h3fp4_linear(h, *wq, two, ws)
    A.h3fp4_check(ws)
    assert torch.equal(bits(one), bits(two))
