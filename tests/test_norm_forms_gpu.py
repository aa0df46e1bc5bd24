"""The norm's gradient at the numbers of rows where a workgroup takes several of them
with more pieces a lane (129 to 512) and next to them, and the norm's 8-bit rows where
a lane has two pieces of them (more than 256 rows), against the formulas: tolerances as
in test_norm_gpu.py."""
import pytest
import torch

import test_norm_gpu as base
from test_norm_gpu import F64, KINDS, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the GPU tests must run on an MI355X")
    base.moe.lib()


@pytest.mark.parametrize("H", [8, 520, 1024, 5120, 8192, 16384])
@pytest.mark.parametrize("T", [128, 129, 301, 509, 512, 513])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_norm_backward_forms(T, H, stream):
    base.say(f"norm_backward T={T} H={H} stream={stream}")
    g = gen(T * 131 + H)
    h = (randn(g, T, H) * torch.exp(randn(g, T, 1))).to(KINDS[stream])
    inv = (1.0 / torch.sqrt(h.to(F64).square().mean(dim=1) + 1e-6)).float()
    w = (1 + 0.2 * randn(g, H)).to(KINDS["f32" if T % 2 else "bf16"])
    d, t = randn(g, T, H).to(torch.bfloat16), randn(g, T, H).to(KINDS[stream])
    base.check_grad(d, h, inv, w, t, base.norm_backward(d, h, inv, w, t))


@pytest.mark.parametrize("H", [8, 504, 1032, 5120, 7168, 16384, 32768])
@pytest.mark.parametrize("T", [256, 257])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_norm_to_int8_forms(T, H, stream):
    base.say(f"norm to int8 T={T} H={H} stream={stream}")
    g = gen(T * 137 + H)
    x = (randn(g, T, H) * torch.exp(randn(g, T, 1))).to(torch.bfloat16)
    res = (3 * randn(g, T, H)).to(KINDS[stream])
    w = (1 + 0.2 * randn(g, H)).to(KINDS["f32" if T % 2 else "bf16"])
    base.check_norm(x, w, 1e-6, res, "int8", base.norm(x, w, 1e-6, res, "int8"))
