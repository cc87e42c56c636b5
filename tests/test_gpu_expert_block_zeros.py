"""The block of examples/expert_block.py on tensors of zeros: a largest
magnitude of 0 gives no scale of its own, and every gradient stays finite."""
import pytest
import torch

import scaled_fp8_linear_gb300 as F
from tests.test_gpu_expert_block import _example

pytestmark = pytest.mark.gpu


def _block():
    block = _example().ExpertBlock(256, 128, 4, 2, alpha=0.9)
    g = torch.Generator(device="cuda").manual_seed(2)
    return block, torch.randn(48, 256, generator=g, device="cuda").to(torch.bfloat16)


def test_zero_gradients():
    block, x = _block()
    _, _, s = block.forward(x)
    zero = torch.zeros_like(x)
    for name, t in block.backward(zero, zero, s).items():
        assert not t.any(), name          # NaN counts as nonzero
    assert F.fp8_device_status() == 0


def test_zero_input():
    block, x = _block()
    x_out, z, s = block.forward(torch.zeros_like(x))
    assert not x_out.any() and not z.any()
    for name, t in block.backward(x, x, s).items():
        assert torch.isfinite(t).all(), name
