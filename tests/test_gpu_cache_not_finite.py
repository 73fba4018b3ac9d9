"""Keys and values that are not finite, in the 4-bit cache and in the attention that reads it (GPU)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import _heads_ref as R  # noqa: E402
import _token_ref as T  # noqa: E402
from _cache_helpers import Paged  # noqa: E402

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    from audio_dit_gb300 import build
    build.build()


def bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("D", [16, 64, 80, 128, 256])
def test_what_is_held(D):
    """A block with a NaN comes back as NaN, an infinity as the largest of its scale; nothing else changes."""
    import audio_dit_gb300 as A
    rng = np.random.default_rng(D)
    c = Paged(rng, [37, 5], 3, D, 16)
    k, v = (R.rand_bf16(rng, 42, 3, D) for _ in range(2))
    for t in (k, v):
        t[3, 1, 0] = t[8, 2, D - 1] = t[9, 2, D - 1] = t[36, 0, 5] = t[41, 1, 7] = NAN
        t[20, 0] = NAN
        t[4, 1, 3], t[5, 0, D - 2] = float("inf"), -float("inf")
    A.h3fp4_cache_append(k.cuda(), v.cuda(), c.cache, *c.args([37, 5]), **c.scales())
    ko, vo = (torch.zeros(42, 3, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.h3fp4_cache_read(ko, vo, c.cache, *c.args([37, 5]), **c.scales())
    for got, x, s in ((ko.cpu(), k, c.k_gscale), (vo.cpu(), v, c.v_gscale)):
        bad = x.isnan().unflatten(-1, (-1, 16)).any(-1).repeat_interleave(16, -1)
        assert torch.equal(got.isnan(), bad) and bool(got[~bad].isfinite().all())
        assert torch.equal(bits(got)[~bad], bits(T.held(x, s)[1])[~bad])


# lengths, rows, heads of q and kv, D, page: units of 8 and of 16 columns; sequences' last rows of one warp, of several
# CTAs, and of short units that a warp takes alone
@pytest.mark.parametrize("n,rows,Hq,heads,D,page", [
    (40, 1, 2, 1, 64, 16), (40, 5, 2, 1, 64, 16), (300, 4, 2, 1, 128, 16), (300, 7, 6, 2, 128, 64), (70, 3, 4, 2, 256, 16),
    (1500, 9, 8, 2, 256, 64), (5000, 6, 16, 4, 64, 64), (129, 30, 4, 4, 80, 32), (9000, 4, 8, 4, 128, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_them_alone(n, rows, Hq, heads, D, page, causal):
    import audio_dit_gb300 as A
    rng = np.random.default_rng(n + D)
    seqs = 3
    c = Paged(rng, [n] * seqs, heads, D, page)
    k, v = (t.view(seqs, n, heads, D) for t in (R.rand_bf16(rng, seqs * n, heads, D) for _ in range(2)))
    q = R.rand_bf16(rng, seqs * rows, Hq, D).cuda()
    ws = A.alloc_cache_attn_workspace(seqs * rows, seqs, Hq, heads, D)

    def attend(k, v):
        A.h3fp4_cache_append(k.view(-1, heads, D).cuda(), v.view(-1, heads, D).cuda(), c.cache, *c.args([n] * seqs), **c.scales())
        t, ln, off = c.args([rows] * seqs)
        out, lse = torch.empty(seqs * rows, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(seqs * rows, Hq, device="cuda")
        A.h3fp4_cache_attn(q, c.cache, t, ln, out, ws, row_off=off, causal=causal, lse=lse, **c.scales())
        A.h3fp4_check(ws)
        return out.view(seqs, rows, Hq, D).cpu(), lse.view(seqs, rows, Hq).cpu()

    good, good_lse = attend(k, v)
    group = Hq // heads
    for at in sorted({0, n // 2, n - rows, n - (rows + 1) // 2, n - 1}):
        sees = torch.arange(rows) + n - rows >= at if causal else torch.ones(rows, dtype=torch.bool)
        h = at % heads
        heads_of = slice(h * group, (h + 1) * group)
        for d in (0, D - 1):
            # a key: the whole row and its sum, of its own head's queries
            x = k.clone()
            x[1, at, h, d] = NAN
            out, lse = attend(x, v)
            bad = torch.zeros(seqs, rows, Hq, dtype=torch.bool)
            bad[1, sees, heads_of] = True
            assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all()), ("k", at, d)
            assert torch.equal(bits(out)[~bad], bits(good)[~bad]) and torch.equal(lse[~bad], good_lse[~bad]), ("k", at, d)
            # a value: its block of 16
            x = v.clone()
            x[1, at, h, d] = NAN
            out, lse = attend(k, x)
            bad = torch.zeros(seqs, rows, Hq, D, dtype=torch.bool)
            block = bad[1, :, heads_of, d // 16 * 16:d // 16 * 16 + 16]
            block |= sees[:, None, None]
            assert torch.equal(out.isnan(), bad), ("v", at, d)
            assert torch.equal(bits(out)[~bad], bits(good)[~bad]) and torch.equal(lse, good_lse), ("v", at, d)
