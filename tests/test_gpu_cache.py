"""The paged 4-bit cache and the attention that reads it (GPU) against plain 64-bit forms."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import _heads_ref as R  # noqa: E402
import _token_ref as T  # noqa: E402
from _cache_helpers import Paged  # noqa: E402
from _gpu_helpers import Guarded  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    from audio_dit_gb300 import build
    build.build()


def bits(t):
    return t.contiguous().view(torch.int16)


# ------------------------------------------------------------------------------------------------ rows in and out

STORE = [  # lengths before, new rows, heads, D, page
    ([0], [1], 1, 16, 16),
    ([0, 5, 17], [16, 1, 30], 2, 64, 16),
    ([15, 0, 100, 3], [1, 1, 1, 1], 8, 128, 64),
    ([7, 40], [100, 0], 3, 128, 48),
    ([0, 33, 2], [70, 5, 1], 2, 256, 32),
    ([9, 1], [33, 64], 3, 80, 16),
    ([1] * 40, [1] * 40, 1, 192, 128),
    ([0], [1100], 2, 48, 1024),
]


@pytest.mark.parametrize("before,rows,heads,D,page", STORE)
def test_rows_in_and_out(before, rows, heads, D, page):
    import audio_dit_gb300 as A
    rng = np.random.default_rng(sum(rows) * 1000 + D)
    c = Paged(rng, before, heads, D, page)
    old = c.fill(rng)
    total = [a + b for a, b in zip(before, rows)]
    p = Paged(rng, total, heads, D, page)                            # the same with room for the new rows
    p.k_gscale, p.v_gscale = c.k_gscale, c.v_gscale
    if sum(before):
        A.h3fp4_cache_append(*(torch.cat(t).cuda() for t in old), p.cache, *p.args(before, total=before), **p.scales())
    # the new rows are strided views of one projection's output; scales of all magnitudes, zeros among them
    M = sum(rows)
    kv = R.rand_bf16(rng, M, 2 * heads + 1, D) * torch.from_numpy(np.exp2(rng.integers(-30, 8, (M, 1, 1)))).bfloat16()
    kv[0, 0] = 0
    dev = kv.cuda()
    k, v = dev[:, :heads], dev[:, heads + 1:]
    A.h3fp4_cache_append(k, v, p.cache, *p.args(rows), **p.scales())
    ones = all(n == 1 for n in rows)
    if ones:                                                         # without row_off: the same places
        again = p.cache.clone()
        A.h3fp4_cache_append(k, v, again, *p.args(None), **p.scales())
        assert torch.equal(again, p.cache)
    ko, vo = (Guarded((sum(total), heads, D), torch.bfloat16) for _ in range(2))
    A.h3fp4_cache_read(ko.t, vo.t, p.cache, *p.args(total), **p.scales())
    ko.check("k"), vo.check("v")
    for got, was, new, s in ((ko.t, old[0], kv[:, :heads], p.k_gscale), (vo.t, old[1], kv[:, heads + 1:], p.v_gscale)):
        want, at = [], 0
        for i, n in enumerate(rows):
            want += [T.held(was[i], s)[1], T.held(new[at:at + n], s)[1]]
            at += n
        assert torch.equal(bits(got.cpu()), bits(torch.cat(want)))
    # the new rows alone, into strided views
    back = torch.zeros(M, 2 * heads, D, dtype=torch.bfloat16, device="cuda")
    A.h3fp4_cache_read(back[:, heads:], back[:, :heads], p.cache, *p.args(rows), **p.scales())
    last = torch.cat([torch.arange(t - n, t) + o for t, n, o in zip(total, rows, np.cumsum([0] + total[:-1]))]).cuda()
    assert torch.equal(bits(back[:, heads:]), bits(ko.t[last])) and torch.equal(bits(back[:, :heads]), bits(vo.t[last]))


def test_scales_at_ties():
    """Block maxima of every bf16 mantissa under global scales that put some of them on ties of E4M3."""
    import audio_dit_gb300 as A
    tops = torch.tensor([m * 2.0 ** (e - 7) for e in range(-6, 1) for m in range(128, 256)])
    rows = torch.stack([tops * f for f in (1.0, -0.75, 0.5, 0.25) * 4], -1).bfloat16()
    k = rows[:, None].expand(-1, 2, -1).contiguous()
    s = torch.tensor([1.75, 1.5]) * torch.tensor(1.0 / 2688.0) * 1.25
    want = T.held(k, s)[1]
    old = k.float().abs().amax(-1) / 6.0 / s
    new = k.float().abs().amax(-1) * torch.tensor(1.0 / 6.0) / s
    assert int((old.to(torch.float8_e4m3fn).float() != new.to(torch.float8_e4m3fn).float()).sum()) > 0
    n = len(rows)
    cache = A.alloc_kv_cache(n // 16, 2, 16, 16)
    table = torch.arange(n // 16, dtype=torch.int32, device="cuda")[None]
    length, off = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    g = dict(k_gscale=s.cuda(), v_gscale=s.flip(0).cuda())
    A.h3fp4_cache_append(k.cuda(), k.cuda(), cache, table, length, off, **g)
    ko, vo = (torch.empty(n, 2, 16, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.h3fp4_cache_read(ko, vo, cache, table, length, off, **g)
    assert torch.equal(bits(ko.cpu()), bits(want))
    assert torch.equal(bits(vo.cpu()), bits(T.held(k, s.flip(0))[1]))


def test_rows_without_a_place():
    import audio_dit_gb300 as A
    rng = np.random.default_rng(1)
    c = Paged(rng, [40, 33], 2, 64, 16, wide=0)
    c.cache.fill_(0xA5)
    c.table[0, 1], c.table[1, 0] = -1, c.n_pages                      # no pages of the pool
    k, v = R.rand_bf16(rng, 80, 2, 64).cuda(), R.rand_bf16(rng, 80, 2, 64).cuda()
    # rows behind the last sequence, positions below zero (more rows than tokens) and past the table
    t, n, off = c.args([50, 20], total=[40, 60])
    A.h3fp4_cache_append(k, v, c.cache, t, n, off, **c.scales())
    # positions 0..39 of sequence 0 come from rows 10..49 (16..31 have no page); 40..59 of sequence 1 from rows
    # 50..69, of which the table has room for 40..47
    ko, vo = (torch.full((80, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.h3fp4_cache_read(ko, vo, c.cache, t, n, off, **c.scales())
    got = torch.tensor([r for r in range(80) if (10 <= r < 26 or 42 <= r < 50 or 50 <= r < 58)])
    rest = torch.tensor([r for r in range(80) if r not in set(got.tolist())])
    assert torch.equal(bits(ko.cpu()[got]), bits(T.held(k.cpu()[got], c.k_gscale)[1]))
    assert torch.equal(bits(vo.cpu()[got]), bits(T.held(v.cpu()[got], c.v_gscale)[1]))
    assert bool((ko[rest.cuda()] == 7).all()) and bool((vo[rest.cuda()] == 7).all())
    used = set(c.table[0, [0, 2]].tolist()) | {int(c.table[1, 2])}
    other = torch.tensor([i for i in range(c.n_pages) if i not in used]).cuda()
    assert bool((c.cache[other] == 0xA5).all())
    # tables of nonsense neither read nor write outside
    out = Guarded((80, 2, 64), torch.bfloat16)
    pool = Guarded(tuple(c.cache.shape), torch.uint8)
    for _ in range(20):
        bad = [torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, s).astype(np.int32)).cuda() for s in ((2, 3), (2,), (3,))]
        for args in (bad, [bad[0] % 9 - 2, bad[1] % 200 - 50, bad[2] % 200 - 60], [t, bad[1], bad[2] % 90]):
            A.h3fp4_cache_append(k, v, pool.t, *args, **c.scales())
            A.h3fp4_cache_read(out.t, ko, pool.t, *args, **c.scales())
    out.check(), pool.check()


# ------------------------------------------------------------------------------------------------ attention

def run_attention(c, q, rows, causal, scale=None, lse=True, out=None, total=None):
    import audio_dit_gb300 as A
    M, Hq, D = q.shape
    ws = A.alloc_cache_attn_workspace(M, len(c.total), Hq, c.heads, D)
    out = Guarded((M, Hq, D), torch.bfloat16) if out is None else out
    l = Guarded((M, Hq), torch.float32) if lse else None
    t, n, off = c.args(rows, total)
    A.h3fp4_cache_attn(q, c.cache, t, n, out.t, ws, row_off=off, causal=causal, scale=scale, lse=l.t if lse else None,
                       **c.scales())
    A.h3fp4_check(ws)
    out.check("out")
    if lse:
        l.check("lse")
    return out.t, l.t if lse else None


def check_attention(got, lse, q, c, kv, rows, causal, scale, what, there=None, total=None):
    k, v = ([T.held(x, s)[0] for x in t] for t, s in zip(kv, (c.k_gscale, c.v_gscale)))
    off = [0] + [int(x) for x in np.cumsum(rows)]
    ref, l_ref, size, reach, keys = T.cache_attention(q, k, v, off, c.total if total is None else total, causal, scale,
                                                      there)
    top = max((float(x.abs().max()) for x in v if x.numel()), default=0.0)
    tol, l_tol = T.cache_attention_bounds(ref, l_ref, size, reach, keys, top, q.shape[2])
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), (what, int((~(err <= tol)).sum()), (~(err <= tol)).nonzero()[:3].tolist())
    if lse is not None:
        none = keys == 0
        assert bool((lse.cpu()[none] == -math.inf).all()) and bool((got.cpu()[none] == 0).all())
        d = (lse.cpu().double() - l_ref).abs()[~none]
        assert bool((d <= l_tol[~none]).all()), (what, "lse", float(d.max()))


ATTN = [  # lengths, rows, heads of q and kv, D, page, causal
    ([1], [1], 1, 1, 64, 16, True),
    ([1], [1], 4, 2, 128, 64, True),
    ([15], [1], 8, 1, 128, 16, True),
    ([16, 17, 63, 64, 65], [1, 1, 1, 1, 1], 8, 2, 64, 16, True),
    ([300], [1], 32, 8, 128, 64, False),
    ([300, 1000, 77], [5, 1, 9], 28, 4, 128, 32, True),
    ([300, 1000, 77], [5, 0, 9], 28, 4, 64, 48, False),
    ([50], [50], 6, 2, 128, 16, True),                                # a whole prompt
    ([129, 1], [100, 1], 5, 5, 64, 16, True),
    ([200, 90], [3, 4], 16, 1, 256, 64, True),
    ([700], [2], 4, 4, 256, 16, False),
    ([333, 5], [2, 5], 20, 5, 80, 32, True),
    ([100, 99], [1, 2], 3, 3, 16, 16, True),
    ([257, 0, 31], [2, 0, 1], 24, 8, 96, 64, True),
    ([130], [3], 16, 2, 208, 16, True),
    ([5000], [1], 8, 1, 128, 128, True),                              # one unit over many CTAs
    ([4097, 3], [4, 3], 64, 2, 64, 64, True),
    ([20] * 300, [1] * 300, 2, 1, 64, 16, True),
    ([9000, 1, 2000], [1, 1, 17], 16, 2, 128, 64, True),
    ([128 * 76], [1], 32, 8, 128, 64, True),                          # as many tiles as CTAs, and some more and less
    ([128 * 76 + 1], [1], 32, 8, 128, 64, True),
    ([128 * 607], [1], 4, 1, 128, 64, False),
    ([128 * 1217 - 5], [1], 4, 1, 64, 64, True),
    ([18 + i % 40 for i in range(1024)], [1] * 1024, 4, 2, 256, 16, True),   # the most sequences
    ([40] * 1024, [2] * 1024, 16, 4, 64, 16, True),
    ([1 + i * 37 % 128 for i in range(700)], [1] * 700, 16, 4, 128, 32, True),  # many short units, which warps take alone
    ([1 + i * 53 % 600 for i in range(300)], [1] * 300, 8, 8, 64, 16, False),
    ([130] * 500 + [5] * 300 + [0] * 20 + [257] * 200, [1] * 1020, 4, 1, 128, 64, True),
    ([64] * 400, [2] * 400, 8, 2, 256, 16, True),
]


@pytest.mark.parametrize("total,rows,Hq,heads,D,page,causal", ATTN)
def test_attention_against_64_bits(total, rows, Hq, heads, D, page, causal):
    rng = np.random.default_rng(sum(total) * 100 + Hq + D)
    c = Paged(rng, total, heads, D, page)
    kv = c.fill(rng)
    q = R.rand_bf16(rng, sum(rows), Hq, D, scale=2.0)
    got, lse = run_attention(c, q.cuda(), rows, causal)
    check_attention(got, lse, q, c, kv, rows, causal, D ** -0.5, "contiguous")
    first = bits(got).clone()
    again, _ = run_attention(c, q.cuda(), rows, causal, lse=False)
    assert torch.equal(bits(again), first)                            # the same bits, with or without lse
    if all(n == 1 for n in rows):
        again, _ = run_attention(c, q.cuda(), None, causal)
        assert torch.equal(bits(again), first)


def test_attention_on_views_and_rows_that_are_none_s():
    import audio_dit_gb300 as A
    rng = np.random.default_rng(7)
    c = Paged(rng, [130, 47], 2, 128, 16)
    kv = c.fill(rng)
    M, Hq, D = 9, 8, 128
    qkv = R.rand_bf16(rng, M, Hq + 4, D)
    t, n, off = c.args([2, 3])                                        # rows 5 to 8 belong to nobody
    ws = A.alloc_cache_attn_workspace(M, 2, Hq, 2, D)
    out = torch.full((Hq, M, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)      # stored [head][row]
    lse = torch.full((M, Hq), 5.0, device="cuda")
    A.h3fp4_cache_attn(qkv.cuda()[:, 2:2 + Hq], c.cache, t, n, out, ws, row_off=off, scale=0.3, lse=lse, **c.scales())
    A.h3fp4_check(ws)
    check_attention(out[:5], lse[:5], qkv[:5, 2:2 + Hq], c, kv, [2, 3], True, 0.3, "views")
    assert bool((out[5:] == 7).all()) and bool((lse[5:] == 5).all())


def test_attention_where_nothing_is():
    rng = np.random.default_rng(8)
    # sequences without a token, with more rows than tokens, with pages that are not there, longer than their table
    total, rows = [0, 3, 100, 64, 40], [2, 5, 2, 1, 1]
    c = Paged(rng, total, 2, 64, 16, wide=0)
    kv = c.fill(rng)
    c.table[2, 1], c.table[2, 3], c.table[4, :] = -1, 1 << 30, -1
    there = [torch.ones(n, dtype=torch.bool) for n in total]
    there[2][16:32] = there[2][48:64] = False
    there[4][:] = False
    q = R.rand_bf16(rng, sum(rows), 4, 64, scale=2.0)
    for causal in (True, False):
        got, lse = run_attention(c, q.cuda(), rows, causal)
        check_attention(got, lse, q, c, kv, rows, causal, 0.125, "holes", there)
    got, lse = run_attention(c, q.cuda(), rows, True, total=[-5, 3, 100, 64, 40])
    check_attention(got, lse, q, c, kv, rows, True, 0.125, "negative length", there, total=[-5, 3, 100, 64, 40])


def test_lengths_past_the_table():
    rng = np.random.default_rng(15)
    c = Paged(rng, [64, 30], 2, 64, 16, wide=0)                       # room for 64 tokens each
    kv = c.fill(rng)
    q = R.rand_bf16(rng, 5, 4, 64, scale=2.0)
    # rows at positions 61 to 65 of a sequence of 66: the tokens from 64 on are not there
    got, lse = run_attention(c, q.cuda(), [5, 0], True, total=[66, 30])
    check_attention(got, lse, q, c, kv, [5, 0], True, 0.125, "past the table", total=[66, 30])
    got, lse = run_attention(c, q.cuda(), [5, 0], False, total=[2 ** 31 - 1, 30])
    check_attention(got, lse, q, c, kv, [5, 0], False, 0.125, "all of the table", total=[64, 30])


def test_attention_with_tables_of_nonsense():
    import audio_dit_gb300 as A
    rng = np.random.default_rng(9)
    c = Paged(rng, [64, 64, 64], 2, 64, 16)
    c.fill(rng)
    M = 20
    q = R.rand_bf16(rng, M, 4, 64).cuda()
    out, lse = Guarded((M, 4, 64), torch.bfloat16), Guarded((M, 4), torch.float32)
    n = A.h3fp4_cache_attn_workspace_bytes(64)
    ws = Guarded((n,), torch.uint8, zero=True)
    for i in range(30):
        t, ln, off = (torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, s).astype(np.int32)).cuda()
                      for s in ((3, 5), (3,), (4,)))
        for args in ((t, ln % 300, off % 40 - 10), (t % 9, ln, off), (t % 20 - 4, ln % 400 - 100, off % 60 - 20)):
            A.h3fp4_cache_attn(q, c.cache, *args[:2], out.t, ws.t, row_off=args[2], causal=bool(i & 1), lse=lse.t)
    A.h3fp4_check(ws.t)
    out.check(), lse.check(), ws.check()


def test_wide_ranges_of_scores():
    import audio_dit_gb300 as A
    rng = np.random.default_rng(10)
    c = Paged(rng, [400], 1, 128, 64)
    kv = c.fill(rng)
    # queries of all magnitudes, elements of one head 2^30 apart, steep and flat softmaxes
    q = R.rand_bf16(rng, 1, 64, 128) * torch.logspace(-30, 4, 64).to(torch.bfloat16)[None, :, None]
    q[0, 5, ::2] *= 2.0 ** -30
    q[0, 6] = 0
    got, lse = run_attention(c, q.cuda(), [1], True, scale=0.7)
    check_attention(got, lse, q, c, kv, [1], True, 0.7, "magnitudes")
    # scores that leave fp32's range are NaN, in their columns alone
    q[0, 7] = 1e37
    q[0, 8] = -1e37
    k = torch.full((400, 1, 128), 0.05, dtype=torch.bfloat16, device="cuda")
    A.h3fp4_cache_append(k, k, c.cache, *c.args([400]), **c.scales())
    got, lse = run_attention(c, q.cuda(), [1], True, scale=50.0)
    bad = got.isnan().all(-1)[0].cpu()
    assert bad.nonzero()[:, 0].tolist() == [7, 8] and bool(lse[0, 7:9].isnan().all())
    assert bool(got[0][~bad].isfinite().all())


def test_growing_maxima():
    """Keys that keep raising the largest score, and ones that lower it, over pages and CTAs."""
    import audio_dit_gb300 as A
    rng = np.random.default_rng(11)
    for direction in (1, -1):
        c = Paged(rng, [3000], 1, 64, 16)
        k = torch.zeros(3000, 1, 64)
        k[:, 0, 0] = torch.linspace(-20, 20, 3000) * direction
        k, v = k.bfloat16(), R.rand_bf16(rng, 3000, 1, 64)
        c.k_gscale[:] = 0.01
        A.h3fp4_cache_append(k.cuda(), v.cuda(), c.cache, *c.args([3000]), **c.scales())
        q = torch.zeros(1, 2, 64)
        q[0, :, 0] = torch.tensor([3.0, -3.0])
        q = q.bfloat16()
        got, lse = run_attention(c, q.cuda(), [1], True, scale=1.0)
        check_attention(got, lse, q, c, [[k], [v]], [1], True, 1.0, direction)


def test_one_captured_call_serves_growing_sequences():
    import audio_dit_gb300 as A
    rng = np.random.default_rng(12)
    heads, Hq, D, steps = 2, 8, 128, 70
    c = Paged(rng, [100, 3, 500], heads, D, 16)
    kv = c.fill(rng)
    total = [n + steps for n in c.total]
    p = Paged(rng, total, heads, D, 16)
    p.k_gscale, p.v_gscale = c.k_gscale, c.v_gscale
    A.h3fp4_cache_append(*(torch.cat(t).cuda() for t in kv), p.cache, *p.args(c.total, total=c.total), **p.scales())
    t, n, _ = p.args(None, total=c.total)
    new = R.rand_bf16(rng, steps, 3, Hq + 2 * heads, D)
    row = torch.zeros(3, Hq + 2 * heads, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(3, Hq, D, dtype=torch.bfloat16, device="cuda")
    ws = A.alloc_cache_attn_workspace(3, 3, Hq, heads, D)

    scales = p.scales()

    def step():
        A.h3fp4_cache_append(row[:, Hq:Hq + heads], row[:, Hq + heads:], p.cache, t, n, **scales)
        A.h3fp4_cache_attn(row[:, :Hq], p.cache, t, n, out, ws, **scales)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        keep = p.cache.clone()
        step()                                                        # one-time setup, over what the first token brings
        p.cache.copy_(keep)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(steps):
        row.copy_(new[i].cuda())
        n += 1
        g.replay()
        kv = [[torch.cat([old, new[i, s, a:b][None]]) for s, old in enumerate(have)]
              for have, a, b in ((kv[0], Hq, Hq + heads), (kv[1], Hq + heads, Hq + 2 * heads))]
        if i in (0, 11, 12, 13, steps - 1):
            now = [m + i + 1 for m in c.total]
            check_attention(out, None, new[i, :, :Hq], p, kv, [1, 1, 1], True, D ** -0.5, i, total=now)
    A.h3fp4_check(ws)


def test_offsets_past_32_bits():
    import audio_dit_gb300 as A
    rng = np.random.default_rng(13)
    heads, D, page = 8, 128, 1024
    c = Paged(rng, [40], heads, D, page, spare=0)
    n_pages = 2400                                                    # 2.8e9 bytes
    assert n_pages * A.h3fp4_cache_page_bytes(heads, D, page) > 2 ** 31
    c.cache = torch.empty(n_pages, heads, page, 144, dtype=torch.uint8, device="cuda")
    c.n_pages = n_pages
    c.table[0, 0] = n_pages - 1
    kv = c.fill(rng)
    q = R.rand_bf16(rng, 1, 16, D)
    got, lse = run_attention(c, q.cuda(), [1], True)
    check_attention(got, lse, q, c, kv, [1], True, D ** -0.5, "last page")


def test_waits_that_run_out():
    import audio_dit_gb300 as A
    ws = A.alloc_cache_attn_workspace(1, 1, 1, 1, 64)
    A.h3fp4_selftest_cache_attn_timeout(ws, 1000000)
    with pytest.raises(A.H3FP4Error) as e:
        A.h3fp4_check(ws)
    assert e.value.status == 5
    A.h3fp4_check(ws)                                                 # read and cleared


def test_cached_context_for_attention_on_rows():
    """A cached sequence read back feeds the attention on bf16 rows: the two agree to what rounding K and V to bf16 does."""
    import audio_dit_gb300 as A
    rng = np.random.default_rng(14)
    c = Paged(rng, [300], 2, 64, 32)
    c.fill(rng)
    q = R.rand_bf16(rng, 4, 8, 64).cuda()
    k, v = (torch.empty(300, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.h3fp4_cache_read(k, v, c.cache, *c.args([300]), **c.scales())
    out = torch.empty_like(q)
    ws = A.alloc_attn_workspace(4, 300, 8, 2, 64)
    A.h3fp4_cross_attn(q, k, v, out, ws)
    A.h3fp4_check(ws)
    got, _ = run_attention(c, q, [4], False)
    assert float((got.float() - out.float()).norm() / out.float().norm()) < 2.0 ** -6
