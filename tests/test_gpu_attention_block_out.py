"""The attention half of a block (examples/attention_block.py): its output projection with gate and residual against the
oracle's linear on the attention's own outputs."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from _gpu_helpers import check_outputs, host_u16  # noqa: E402
from test_gpu_attention_block import block  # noqa: E402,F401


def test_output_projection(orc, block):  # noqa: F811
    block.step()
    block.check()
    K = block.width
    codes, sf, gscale = block.w["out"]
    w = (codes.cpu().numpy(), sf.cpu().numpy(), float(gscale.cpu()[0]))
    a = orc.quantize(host_u16(block.attn))
    ref, bound = orc.linear_full(a, w, block.M, K, K, bias=host_u16(block.bias["out"]), gate=block.gate.cpu().numpy(),
                                 resid=host_u16(block.x), seg_off=block.one)
    check_outputs(host_u16(block.y), ref, bound, "output projection")
