"""Attention (GPU) over long key axes, checked so that one key lost or counted twice shows: whole, cut, side by side, with
the context apart, masked, and in both kinds of units."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import numpy as np  # noqa: E402

import _attn_counts as N  # noqa: E402
import _heads_ref as R  # noqa: E402
from test_gpu_attn import Case, built  # noqa: E402,F401

TOKENS = [0, *range(1, 41)]
CASES = {  # Hq, Hkv, D, offsets of rows, of keys, context
    "one token, cut": (8, 2, 128, [0, 1], [0, 32001], 0),
    "few rows, cut": (6, 6, 64, [0, 200], [0, 12345], 0),
    "pair units, cut": (8, 8, 128, [0, 900], [0, 9001], 0),
    "side by side": (2, 2, 128, [0, 601], [0, 70000], 0),
    "whole waves": (2, 2, 64, [0, 40001], [0, 700], 0),
    "whole units": (24, 24, 128, [0, 900], [0, 1300], 0),
    "context apart": (8, 2, 128, TOKENS, [7 * i for i in TOKENS], 16001),
    "context apart, wide": (4, 4, 64, [20 * i for i in range(21)], [300 * i for i in range(21)], 9999),
    "context and own": (4, 2, 128, [0, 700, 1500], [0, 5000, 5300], 3001),
    "ragged": (12, 4, 96, [0, 100, 101, 900, 2500], [0, 3000, 3000, 3129, 8000], 0),
}


def masks(c, kind, rng):
    for name, n in (("key_mask", c.T), ("ctx_mask", c.C)):
        if kind == "all" or n == 0:
            continue
        on = rng.random(n) < 0.7 if kind == "holes" else np.arange(n) < (n * 2) // 3
        setattr(c, name, torch.from_numpy(on))


@pytest.mark.parametrize("kind", ["all", "holes", "padded"])
@pytest.mark.parametrize("name", CASES)
def test_every_key_counts_once(name, kind):
    Hq, Hkv, D, q_off, kv_off, ctx = CASES[name]
    c = Case(1, Hq, Hkv, D, q_off, kv_off, ctx=ctx)
    masks(c, kind, np.random.default_rng(2))
    c.q[:] = 0
    most = ctx + max(b - a for a, b in zip(kv_off, kv_off[1:]))
    every = N.period(most, D)
    for shift in range(0, every, D):
        share, total = N.counts(q_off, kv_off, ctx, D, every, shift, c.key_mask, c.ctx_mask)
        for a, b in zip(kv_off, kv_off[1:]):
            c.v[a:b] = N.marked(ctx, b - a, Hkv, D, every, shift)
        if ctx:
            c.vc = N.marked(0, ctx, Hkv, D, every, shift)
        out, lse = c.run()
        assert N.counted(out, lse, q_off, share, total) is None, shift


@pytest.mark.parametrize("kind", ["all", "holes"])
@pytest.mark.parametrize("name", [n for n in CASES if n != "whole waves"])
def test_rows_are_as_near_as_two_roundings(name, kind):
    Hq, Hkv, D, q_off, kv_off, ctx = CASES[name]
    c = Case(3, Hq, Hkv, D, q_off, kv_off, ctx=ctx)
    masks(c, kind, np.random.default_rng(4))
    out, lse = c.run()
    ref, log = R.attention(c.q, c.k, c.v, q_off, kv_off, c.scale, c.key_mask, c.kc, c.vc, c.ctx_mask)[:2]
    assert N.far_off(out, ref) is None
    some = torch.isfinite(log)
    # scores of a few units in fp32 sums of D products, and the logarithm's own error
    assert bool(((lse.double() - log).abs()[some] <= 2.0 ** -16).all())
