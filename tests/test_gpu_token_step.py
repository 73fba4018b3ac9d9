"""A block's step for one token per sequence, as the example runs it: every call against a plain 64-bit form of what it
was given, eagerly and replayed from a graph."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import _heads_ref as R  # noqa: E402
import _token_ref as T  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    from audio_dit_gb300 import build
    build.build()


def example():
    spec = importlib.util.spec_from_file_location("token_step", os.path.join(ROOT, "examples", "token_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def within(got, ref, tol, what):
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), (what, int((~(err <= tol)).sum()), float((err / tol).max()))


def cached(b):
    """Float64 keys and values of every sequence, read back from the cache (exact but for bf16)."""
    import audio_dit_gb300 as A
    n = b.length.tolist()
    off = torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32).cuda()
    k, v = (torch.empty(sum(n), b.kv_heads, b.dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.h3fp4_cache_read(k, v, b.cache, b.table, b.length, off, k_gscale=b.k_gscale, v_gscale=b.v_gscale)
    return k, v, n


def checked_step(b):
    """The step call by call (the example's), each against its plain form."""
    import audio_dit_gb300 as A
    S, K = b.seqs, b.width
    w = {n: T.decode_weight(*(t.cpu() for t in q), 2 * q[0].shape[1]) for n, q in b.w.items()}
    cpu = lambda t: t.detach().cpu().clone()  # noqa: E731
    x0, len0 = cpu(b.x), b.length.clone()
    calls = []

    def spy(name):
        real = getattr(A, name)

        def call(*a, **kw):
            real(*a, **kw)
            torch.cuda.synchronize()
            calls.append((name, {n: cpu(t) for n, t in dict(x=b.x, h=b.h, y=b.y, qkv=b.qkv, attn=b.attn, up=b.up).items()}))
        return real, call

    names = ("h3fp4_block_norm", "h3fp4_linear_rows", "h3fp4_qk_norm_rope", "h3fp4_cache_append", "h3fp4_cache_attn")
    kept = {n: spy(n) for n in names}
    try:
        for n, (_, call) in kept.items():
            setattr(A, n, call)
        b.step()
    finally:
        for n, (real, _) in kept.items():
            setattr(A, n, real)
    st = [s for _, s in calls]
    assert [n for n, _ in calls] == [names[i] for i in (0, 1, 2, 3, 4, 1, 0, 1, 1)]
    one = [0, S]
    row = lambda t: t.cpu()  # noqa: E731
    out, _, tol, _ = T.block_norm(x0, None, None, None, 1.0, row(b.norm1), None, None, one, 1e-6, False, False)
    within(st[0]["h"], out, tol, "norm before the attention")
    out, tol = T.linear_rows(st[0]["h"], w["qkv"], row(b.bias["qkv"]), None, None, False)
    within(st[1]["qkv"].view(S, -1), out, tol, "qkv")
    q, k, v = b.views(st[1]["qkv"])
    pos = len0.cpu().long()
    cos, sin = b.all_cos.cpu()[pos], b.all_sin.cpu()[pos]
    q2, k2, v2 = b.views(st[2]["qkv"])
    for got, src, wt in ((q2, q, b.q_weight), (k2, k, b.k_weight)):
        ref = R.norm_rope(src, row(wt), cos, sin, False, one, 1e-6)
        within(got, ref, R.norm_rope_bound(ref, b.dim // 2, False), "norm and rotation")
    assert torch.equal(v2, v) and torch.equal(b.length, len0 + 1)
    # the new token is held as it should be, and all tokens are attended to
    kc, vc, n = cached(b)
    last = torch.tensor(n).cumsum(0) - 1
    for got, src, s in ((kc, k2, b.k_gscale), (vc, v2, b.v_gscale)):
        assert torch.equal(got.cpu()[last], T.held(src, s.cpu())[1])
    ks, vs = ([t.cpu().double() for t in x.split(n)] for x in (kc, vc))
    ref, l_ref, size, reach, keys = T.cache_attention(q2, ks, vs, list(range(S + 1)), n, True, b.dim ** -0.5)
    tol, _ = T.cache_attention_bounds(ref, l_ref, size, reach, keys, float(vc.abs().max()), b.dim)
    # (the values were read back in bf16: half a step of each, 2^-9, in the scores and in the sum)
    tol = tol + (2.0 ** -9 + 2 * 2.0 ** -9 * reach)[..., None] * size * 1.01
    within(st[4]["attn"].view(S, b.heads, b.dim), ref, tol, "attention")
    out, tol = T.linear_rows(st[4]["attn"], w["out"], row(b.bias["out"]), None, None, False)
    within(st[5]["y"], out, tol, "output projection")
    out, x_out, tol, x_tol = T.block_norm(x0, st[5]["y"], row(b.post), row(b.gate1), 1.0, row(b.norm2), None, None, one,
                                          1e-6, True, False)
    within(st[6]["x"], x_out, x_tol, "residual")
    within(st[6]["h"], out, tol, "norm before the MLP")
    out, tol = T.linear_rows(st[6]["h"], w["up"], row(b.bias["up"]), None, None, True)
    within(st[7]["up"], out, tol, "SwiGLU")
    out, tol = T.linear_rows(st[7]["up"], w["down"], row(b.bias["down"]), row(b.gate2), st[6]["x"], False)
    within(st[8]["x"], out, tol, "down projection")


def test_step_by_step():
    m = example()
    torch.manual_seed(1)
    lengths = [100, 1, 257]
    b = m.TokenBlock(3, 320, heads=8, kv_heads=2, dim=64, hidden=768, page=16, seed=3)
    b.prompt(torch.randn(sum(lengths), b.width, device="cuda").bfloat16(), lengths)
    for _ in range(3):
        checked_step(b)
    b.check()


def test_replayed_steps_have_the_same_bits():
    m = example()
    lengths = [63, 200]
    runs = []
    for graph in (False, True):
        torch.manual_seed(2)
        b = m.TokenBlock(2, 300, heads=8, kv_heads=4, dim=128, hidden=512, page=32, seed=4)
        b.prompt(torch.randn(sum(lengths), b.width, device="cuda").bfloat16(), lengths)
        x, n = b.x.clone(), b.length.clone()
        if graph:
            g = m.GraphBuckets(b.step)
            g.capture(0)
            b.x.copy_(x), b.length.copy_(n)                      # what the warm-up changed
        for _ in range(40):
            g.run(0) if graph else b.step()
        b.check()
        runs.append((b.x.clone(), b.length.clone()))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    assert bool(runs[0][0].isfinite().all())


def test_two_streams_with_workspaces_of_their_own():
    m = example()
    blocks = []
    for seed in (5, 6):
        torch.manual_seed(seed)
        b = m.TokenBlock(2, 200, heads=4, kv_heads=4, dim=64, hidden=256, page=16, seed=seed)
        b.prompt(torch.randn(90, b.width, device="cuda").bfloat16(), [40, 50])
        blocks.append((b, b.x.clone(), b.length.clone()))
    alone = []
    for b, _, _ in blocks:
        for _ in range(20):
            b.step()
        torch.cuda.synchronize()
        alone.append(b.x.clone())
    for b, x, n in blocks:
        b.x.copy_(x), b.length.copy_(n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(20):
        for (b, _, _), s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.step()
    torch.cuda.synchronize()
    for (b, _, _), want in zip(blocks, alone):
        assert torch.equal(b.x, want)
        b.check()


def test_example_runs(capsys):
    example().main()
    assert "us" in capsys.readouterr().out
