"""Attention to encoder states and shared contexts (GPU) against a plain 64-bit form."""
import math

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


def cuda(t):
    return None if t is None else t.cuda()


class Case:
    """Host tensors of one problem and the call on them."""

    def __init__(self, seed, Hq, Hkv, D, q_off, kv_off, ctx=0, scale=None, spread=1.0):
        rng = np.random.default_rng(seed)
        self.rng, self.Hq, self.Hkv, self.D, self.q_off, self.kv_off = rng, Hq, Hkv, D, q_off, kv_off
        self.M, self.T, self.C = q_off[-1], kv_off[-1], ctx
        self.q = R.rand_bf16(rng, self.M, Hq, D, scale=spread)
        self.k, self.v = R.rand_bf16(rng, self.T, Hkv, D, scale=spread), R.rand_bf16(rng, self.T, Hkv, D)
        self.kc = R.rand_bf16(rng, ctx, Hkv, D, scale=spread) if ctx else None
        self.vc = R.rand_bf16(rng, ctx, Hkv, D) if ctx else None
        self.key_mask = self.ctx_mask = None
        self.scale = D ** -0.5 if scale is None else scale

    def run(self, stream=None, guard=True):
        import audio_dit_gb300 as A
        out, lse = Guarded((self.M, self.Hq, self.D), torch.bfloat16), Guarded((self.M, self.Hq), torch.float32)
        n = A.h3fp4_attn_workspace_bytes(self.M, self.T, self.Hq, self.Hkv, self.D, self.q_off, self.kv_off, self.C)
        ws = Guarded((n,), torch.uint8, zero=True)
        torch.cuda.synchronize()
        kw = dict(q_off=self.q_off, kv_off=self.kv_off, key_mask=cuda(self.key_mask), scale=self.scale, lse=lse.t,
                  stream=stream)
        # K and V as views of one projection's output, side by side
        kv = torch.cat([self.k, self.v], 1).cuda()
        k, v = kv[:, :self.Hkv], kv[:, self.Hkv:]
        if self.C:
            A.h3fp4_shared_attn(self.q.cuda(), k, v, self.kc.cuda(), self.vc.cuda(), out.t, ws.t,
                                ctx_mask=cuda(self.ctx_mask), **kw)
        else:
            A.h3fp4_cross_attn(self.q.cuda(), k, v, out.t, ws.t, **kw)
        A.h3fp4_check(ws.t, stream=stream)
        for g, what in ((out, "out"), (lse, "lse"), (ws, "ws")):
            g.check(what)
        return out.t.cpu(), lse.t.cpu()

    def check(self, out=None, lse=None):
        if out is None:
            out, lse = self.run()
        ref = R.attention(self.q, self.k, self.v, self.q_off, self.kv_off, self.scale, self.key_mask, self.kc, self.vc,
                          self.ctx_mask)
        tol, tol_lse = R.attention_bounds(*ref, self.D)
        off = (out.double() - ref[0]).abs()
        bad = ~(off <= tol)
        assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:3].tolist(), float((off / tol).max()))
        empty = torch.isinf(ref[1])
        assert torch.equal(torch.isneginf(lse), empty)
        bad = ~((lse.double() - ref[1]).abs() <= tol_lse) & ~empty
        assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:3].tolist())
        return out, lse


# query and key lengths around every tile edge, as segments of one call
EDGES = [(1, 1), (2, 16), (127, 17), (128, 127), (129, 128), (255, 129), (256, 255), (257, 256), (300, 257), (3, 0),
         (0, 50), (1, 1000), (64, 383), (513, 1)]


@pytest.mark.parametrize("D", [128, 64, 8, 72, 96, 120])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (6, 2)])
def test_lengths_around_tiles(D, Hq, Hkv):
    q_off = [0] + list(np.cumsum([a for a, _ in EDGES]))
    kv_off = [0] + list(np.cumsum([b for _, b in EDGES]))
    Case(D + Hq, Hq, Hkv, D, [int(x) for x in q_off], [int(x) for x in kv_off]).check()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (7, 1), (24, 1), (130, 1), (10, 5), (28, 4), (48, 3)])
@pytest.mark.parametrize("M", [1, 5, 140])
def test_head_groups(Hq, Hkv, M):
    Case(Hq * 10 + M, Hq, Hkv, 64, [0, M], [0, 333]).check()
    Case(Hq * 10 + M, Hq, Hkv, 128, [0, M // 2, M], [0, 100, 190], ctx=150).check()


@pytest.mark.parametrize("M,T,ctx", [(1, 5000, 0), (3, 4097, 0), (200, 6000, 0), (1, 1, 4000), (40, 40, 3001),
                                     (300, 2000, 2500)])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 128), (8, 2, 64)])
def test_long_keys(M, T, ctx, Hq, Hkv, D):
    Case(M + T + ctx, Hq, Hkv, D, [0, M], [0, T], ctx=ctx).check()


@pytest.mark.parametrize("rows,n,ctx,own", [(1, 48, 700, 20), (1, 200, 300, 3), (2, 60, 1000, 0), (130, 5, 333, 140),
                                            (300, 3, 128, 300), (7, 256, 129, 5)])
def test_shared_context(rows, n, ctx, own):
    rng = np.random.default_rng(rows * n)
    c = Case(rows + n, 4, 2, 64, R.lengths(rng, rows * n, n), R.lengths(rng, own * n, n), ctx=ctx)
    c.check()
    c.ctx_mask = torch.from_numpy(rng.random(ctx) < 0.5)
    c.check()


def test_context_alone_and_no_context_agree_with_cross():
    c = Case(77, 4, 4, 128, [0, 150, 290], [0, 0, 0], ctx=300)
    out, lse = c.check()
    whole = Case(77, 4, 4, 128, [0, 290], [0, 300])
    whole.q, whole.k, whole.v = c.q, c.kc, c.vc
    o2, l2 = whole.check()
    assert torch.allclose(lse, l2, atol=1e-4)


MASKS = ["holes", "none left", "padded", "first tile gone", "last key only", "one segment gone"]


@pytest.mark.parametrize("kind", MASKS)
@pytest.mark.parametrize("D,Hq,Hkv,ctx", [(128, 2, 2, 0), (64, 6, 2, 0), (96, 2, 1, 200)])
def test_masks_with_poisoned_places(kind, D, Hq, Hkv, ctx):
    """What lies at a key that is left out, in another segment or behind the last key must not matter."""
    c = Case(MASKS.index(kind) + D, Hq, Hkv, D, [0, 1, 150, 450], [0, 300, 610, 911], ctx=ctx)
    T = c.T
    if kind == "holes":
        m = c.rng.random(T) < 0.5
    elif kind == "none left":
        m = np.zeros(T, bool)
    elif kind == "padded":
        m = np.concatenate([np.arange(300) < 130, np.arange(310) < 1, np.arange(301) < 257])
    elif kind == "first tile gone":
        m = np.concatenate([np.arange(300) >= 128, np.arange(310) >= 300, np.arange(301) >= 256])
    elif kind == "last key only":
        m = np.concatenate([np.arange(300) == 299, np.arange(310) == 309, np.arange(301) == 300])
    else:
        m = np.arange(T) >= 300
    c.key_mask = torch.from_numpy(m)
    if ctx:
        c.ctx_mask = torch.from_numpy(m[:ctx].copy())
    want = c.check()
    gone = ~c.key_mask
    bits = torch.tensor([float("nan"), float("inf"), float("-inf"), 3.3e38, -3.3e38]).to(torch.bfloat16)
    for t in (c.k, c.v):
        t[gone] = bits[torch.from_numpy(c.rng.integers(0, 5, (int(gone.sum()), Hkv, D)))]
    if ctx:
        c.vc[~c.ctx_mask] = float("nan")
        c.kc[~c.ctx_mask] = float("inf")
    got = c.run()
    assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16))
    assert torch.equal(got[1], want[1])


def test_neighbouring_segments_do_not_leak():
    c = Case(9, 2, 2, 128, [0, 100, 230, 231], [0, 77, 210, 300])
    want = c.check()
    c.k[77:210] = float("nan")
    c.v[77:210] = float("nan")
    c.q[100:230] = float("inf")
    out, lse = c.run()
    for r in (slice(0, 100), slice(230, 231)):
        assert torch.equal(out[r].view(torch.int16), want[0][r].view(torch.int16))
        assert torch.equal(lse[r], want[1][r])


@pytest.mark.parametrize("spread", [4.0, 16.0])
def test_peaked_scores(spread):
    """Scores of hundreds: the maximum moves from tile to tile and most weights vanish."""
    c = Case(31, 2, 2, 128, [0, 200], [0, 1500], spread=spread)
    c.k[700:] *= 3
    c.check()
    c = Case(32, 4, 1, 64, [0, 5], [0, 3000], ctx=1000, spread=spread)
    c.check()


def test_scale_is_used():
    for scale in (1e-3, 1.0, 0.37):
        Case(41, 2, 2, 64, [0, 70], [0, 300], scale=scale).check()


def test_scores_of_minus_infinity_leave_a_row_empty():
    c = Case(51, 1, 1, 64, [0, 130], [0, 200])
    c.q[:] = c.q.abs() + 0.1
    c.k[:] = float("-inf")
    out, lse = c.run()
    assert not bool(out.any()) and bool(torch.isneginf(lse).all())


def test_nan_of_a_kept_key_reaches_its_rows():
    c = Case(52, 1, 1, 64, [0, 100, 200], [0, 130, 260])
    c.v[5] = float("nan")
    out, lse = c.run()
    assert bool(torch.isnan(out[:100]).all()) and bool(torch.isfinite(out[100:]).all())
    c.v[5] = 1.0
    c.k[5] = float("nan")
    out, lse = c.run()
    assert bool(torch.isnan(out[:100]).all()) and bool(torch.isnan(lse[:100]).all())
    assert bool(torch.isfinite(out[100:]).all()) and bool(torch.isfinite(lse[100:]).all())


def test_strided_layouts():
    """Q from the interleaved projection output, K and V head-major, the output interleaved with other data."""
    import audio_dit_gb300 as A
    c = Case(61, 6, 2, 64, [0, 90, 201], [0, 300, 431])
    qkv = torch.full((c.M, 10, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    qkv[:, 2:8] = c.q.cuda()
    k = c.k.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    v = c.v.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    hold = torch.full((c.M, 9, 96), 5.0, dtype=torch.bfloat16, device="cuda")
    out = hold[:, 1:7, 16:80]
    ws = A.alloc_attn_workspace(c.M, c.T, 6, 2, 64, c.q_off, c.kv_off)
    lse = torch.empty(c.M, 6, device="cuda")
    A.h3fp4_cross_attn(qkv[:, 2:8], k, v, out, ws, q_off=c.q_off, kv_off=c.kv_off, lse=lse)
    A.h3fp4_check(ws)
    c.check(out.cpu(), lse.cpu())
    hold[:, 1:7, 16:80] = 5.0
    assert bool((hold == 5.0).all())
    # head-major output
    o2 = torch.empty(6, c.M, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    A.h3fp4_cross_attn(qkv[:, 2:8], k, v, o2, ws, q_off=c.q_off, kv_off=c.kv_off)
    A.h3fp4_check(ws)
    c.check(o2.cpu(), lse.cpu())


def test_offsets_past_32_bits():
    import audio_dit_gb300 as A
    c = Case(71, 2, 1, 64, [0, 40], [0, 200])
    step = 1 << 25                                                  # element offsets up to 6.7e9
    big = torch.empty(200 * step + 128, dtype=torch.bfloat16, device="cuda")
    k, v = big.as_strided((200, 1, 64), (step, 64, 1)), big.as_strided((200, 1, 64), (step, 64, 1), 64)
    k.copy_(c.k), v.copy_(c.v)
    out = big.as_strided((40, 2, 64), (step, 128, 1), step // 2)
    q = big.as_strided((40, 2, 64), (step, 128, 1), step // 4)
    q.copy_(c.q)
    lse = torch.empty(40, 2, device="cuda")
    ws = A.alloc_attn_workspace(40, 200, 2, 1, 64)
    A.h3fp4_cross_attn(q, k, v, out, ws, lse=lse)
    A.h3fp4_check(ws)
    c.check(out.cpu(), lse.cpu())


def test_same_bits_on_other_streams_and_again():
    c = Case(81, 4, 2, 128, [0, 100, 333], [0, 900, 1500], ctx=1200)
    want = c.run()
    again = c.run()
    side = c.run(stream=torch.cuda.Stream())
    for o, l in (again, side):
        assert torch.equal(o.view(torch.int16), want[0].view(torch.int16)) and torch.equal(l, want[1])


def test_graph_replay_with_new_inputs():
    import audio_dit_gb300 as A
    c = Case(91, 4, 4, 64, [0, 130], [0, 2500])
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    out, lse = torch.zeros(130, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(130, 4, device="cuda")
    ws = A.alloc_attn_workspace(130, 2500, 4, 4, 64)
    A.h3fp4_cross_attn(q, k, v, out, ws, lse=lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.h3fp4_cross_attn(q, k, v, out, ws, lse=lse)
    d = Case(92, 4, 4, 64, [0, 130], [0, 2500])
    q.copy_(d.q), k.copy_(d.k), v.copy_(d.v)
    for _ in range(3):
        g.replay()
    A.h3fp4_check(ws)
    d.check(out.cpu(), lse.cpu())


def test_workspace_serves_calls_of_other_sizes():
    """One workspace (the largest that is needed) for a series of calls in one stream."""
    import audio_dit_gb300 as A
    cases = [Case(100 + i, 2, 2, 64, [0, m], [0, t], ctx=x) for i, (m, t, x) in enumerate(
        [(1, 3000, 0), (200, 700, 0), (64, 5, 2000), (1, 3000, 0), (300, 300, 300)])]
    n = max(A.h3fp4_attn_workspace_bytes(c.M, c.T, 2, 2, 64, ctx=c.C) for c in cases)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    got = []
    for c in cases:
        out, lse = torch.empty(c.M, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(c.M, 2, device="cuda")
        if c.C:
            A.h3fp4_shared_attn(c.q.cuda(), c.k.cuda(), c.v.cuda(), c.kc.cuda(), c.vc.cuda(), out, ws, lse=lse)
        else:
            A.h3fp4_cross_attn(c.q.cuda(), c.k.cuda(), c.v.cuda(), out, ws, lse=lse)
        got.append((out, lse))
    A.h3fp4_check(ws)
    for c, (out, lse) in zip(cases, got):
        c.check(out.cpu(), lse.cpu())


def test_no_rows_and_no_keys():
    import audio_dit_gb300 as A
    ws = A.alloc_attn_workspace(0, 0, 2, 2, 64)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    A.h3fp4_cross_attn(none, none, none, none, ws)
    q = torch.randn(5, 2, 64, device="cuda").to(torch.bfloat16)
    out, lse = torch.full_like(q, 3.0), torch.zeros(5, 2, device="cuda")
    ws = A.alloc_attn_workspace(5, 0, 2, 2, 64)
    A.h3fp4_cross_attn(q, none, none, out, ws, lse=lse)
    A.h3fp4_check(ws)
    assert not bool(out.any()) and bool(torch.isneginf(lse).all())
    A.h3fp4_shared_attn(q, none, none, none, none, out.fill_(3.0), ws, lse=lse.zero_())
    A.h3fp4_check(ws)
    assert not bool(out.any()) and bool((lse == -math.inf).all())


def test_cold_caches_and_repeats():
    """Copies that take long and land out of order: the same bits as with everything in L2, many times over."""
    import audio_dit_gb300 as A
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for c in (Case(111, 32, 8, 128, [0, 1], [0, 9000]), Case(112, 4, 4, 64, [0, 40, 700], [0, 3000, 5000], ctx=2000),
              Case(113, 2, 2, 128, [0, 300, 600, 1300], [0, 100, 230, 231], ctx=128)):
        q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
        kc, vc = (c.kc.cuda(), c.vc.cuda()) if c.C else (k[:0], v[:0])
        out, lse = torch.empty_like(q), torch.empty(c.M, c.Hq, device="cuda")
        ws = A.alloc_attn_workspace(c.M, c.T, c.Hq, c.Hkv, c.D, c.q_off, c.kv_off, ctx=c.C)
        first = None
        for i in range(30):
            if i % 3:
                flush.zero_()
            A.h3fp4_shared_attn(q, k, v, kc, vc, out.zero_(), ws, q_off=c.q_off, kv_off=c.kv_off, lse=lse)
            A.h3fp4_check(ws)
            if first is None:
                first = out.clone(), lse.clone()
                c.check(out.cpu(), lse.cpu())
            assert torch.equal(out.view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse, first[1]), i


def test_many_units_without_keys_between_masked_ones():
    """Runs of units that only get zeros, between units whose every tile has keys that are left out."""
    c = Case(121, 24, 8, 96, [0, 900, 2500, 2600, 4000, 4001, 5200], [0, 300, 300, 700, 700, 1011, 1400])
    c.key_mask = torch.from_numpy(c.rng.random(1400) < 0.7)
    c.check()
    c = Case(122, 4, 2, 64, list(range(0, 201)), [i // 7 * 150 for i in range(201)], ctx=0)
    c.key_mask = torch.from_numpy(c.rng.random(c.T) < 0.7)
    c.check()


def test_padding_behind_the_last_kept_key():
    """Whole tiles of padding, in the context and behind each segment's keys, beside segments without a kept key."""
    c = Case(131, 4, 2, 64, [0, 100, 101, 400, 900, 901], [0, 700, 900, 900, 1500, 2200], ctx=1000)
    keep = np.zeros(2200, bool)
    for a, n in ((0, 130), (700, 0), (900, 1), (1500, 513)):
        keep[a:a + n] = True
    keep[640:642] = False
    c.key_mask = torch.from_numpy(keep)
    c.check()
    for n in (0, 1, 128, 300, 1000):
        c.ctx_mask = torch.from_numpy(np.arange(1000) < n)
        c.check()
    c.key_mask = None
    c.check()
    # a long axis that is cut, kept at its beginning, in the middle and at its end
    d = Case(132, 8, 2, 128, [0, 3], [0, 9000])
    for a, b in ((0, 100), (4000, 4500), (8990, 9000)):
        d.key_mask = torch.from_numpy((np.arange(9000) >= a) & (np.arange(9000) < b))
        d.check()


def test_timeout_is_reported_and_the_next_call_is_right():
    import time

    import audio_dit_gb300 as A
    ws = torch.zeros(2048, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    t = time.perf_counter()
    A.h3fp4_selftest_attn_timeout(ws, 2_000_000)                    # 2 ms, and no load is issued
    with pytest.raises(A.H3FP4Error) as e:
        A.h3fp4_check(ws)
    assert e.value.status == 5 and time.perf_counter() - t < 1.0
    A.h3fp4_check(ws)                                               # cleared
    Case(141, 2, 2, 128, [0, 300], [0, 300]).check()


def test_whole_waves_and_what_is_left_over():
    """More units of a segment than SMs: dealt out whole, the rest cut."""
    Case(151, 2, 2, 64, [0, 40001], [0, 40]).check()
    Case(152, 2, 1, 64, [0, 20001, 21000], [0, 1300, 1500], ctx=200).check()


def test_units_of_a_head_side_by_side():
    """Keys of more than half the L2 and few rows."""
    Case(161, 2, 2, 128, [0, 601], [0, 70000]).check()
