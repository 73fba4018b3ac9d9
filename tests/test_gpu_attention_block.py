"""The attention half of a block (examples/attention_block.py), each step against a plain 64-bit form of the step on
the values it read, and replayed from a CUDA graph."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import _heads_ref as R  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def block():
    from audio_dit_gb300 import build
    build.build()
    from attention_block import AttentionBlock
    return AttentionBlock(rows=[130, 201], prompt=150, other=77, heads=4, dim=64)


def test_steps_against_plain_forms(block):
    import audio_dit_gb300 as A
    # the projection alone, for the values that the norm reads
    A.h3fp4_linear(block.x, *block.w["qkv"], block.qkv, block.ws, shift=block.shift, scale=block.scale,
                   bias=block.bias["qkv"], seg_off=block.one)
    raw = [t.cpu().clone() for t in block.views()]
    block.step()
    block.check()
    q, k, v = (t.cpu() for t in block.views())
    assert torch.equal(v.view(torch.int16), raw[2].view(torch.int16))       # V is left alone
    cos, sin = block.cos.cpu(), block.sin.cpu()
    for got, x, w in ((q, raw[0], block.q_weight), (k, raw[1], block.k_weight)):
        ref = R.norm_rope(x, w.cpu(), cos, sin, False, [0, block.M], 1e-6)
        assert bool(((got.double() - ref).abs() <= R.norm_rope_bound(ref, cos.shape[1], False)).all())
    scale = block.dim ** -0.5
    ref = R.attention(q, k, v, block.off, block.off, scale, None, block.k_ctx.cpu(), block.v_ctx.cpu(),
                      block.ctx_mask.cpu())
    tol, _ = R.attention_bounds(*ref, block.dim)
    got = block.attn.cpu().view(block.M, block.heads, block.dim)
    assert bool(((got.double() - ref[0]).abs() <= tol).all())
    ref = R.attention(q, block.k_other.cpu(), block.v_other.cpu(), [0, block.M], [0, 77], scale)
    tol, _ = R.attention_bounds(*ref, block.dim)
    got = block.cross.cpu().view(block.M, block.heads, block.dim)
    assert bool(((got.double() - ref[0]).abs() <= tol).all())


def test_graph_replay_gives_the_same_bits(block):
    from audio_dit_gb300.graphs import GraphBuckets
    block.step()
    want = [t.clone() for t in (block.qkv, block.attn, block.y, block.cross)]
    graphs = GraphBuckets(lambda key: block.step())
    graphs.capture("block")
    for t in (block.qkv, block.attn, block.y, block.cross):
        t.zero_()
    graphs.run("block")
    block.check()
    for t, w in zip((block.qkv, block.attn, block.y, block.cross), want):
        assert torch.equal(t.view(torch.int16), w.view(torch.int16))
