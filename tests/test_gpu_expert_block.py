"""The block of examples/expert_block.py against the same block in 64 bits.

E4M3 rounds to within 2^-4 of a value and E5M2 to within 2^-3, so a product's
operands are each off by at most 2^-4 (2^-3) of themselves and, the roundings
being independent, a sum over K terms by about that fraction of the norm of
its terms.  Two products in a row forward, and four with E5M2 gradients
backward: the bounds below are the relative 2-norm errors 2 x 2^-4 x sqrt(2)
for forward outputs and 0.25 for gradients, with the router's choices taken
from the run itself."""
import importlib.util
import os

import pytest
import torch

import scaled_fp8_linear_gb300 as F

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("expert_block", os.path.join(ROOT, "examples", "expert_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rms(v, w):
    return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-5) * w


@pytest.mark.parametrize("tokens,experts,slots", [(256, 4, 2), (33, 8, 3), (1, 8, 2)])
def test_block(tokens, experts, slots):
    width, hidden = 512, 256
    block = _example().ExpertBlock(width, hidden, experts, slots, alpha=0.9)
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda s: (torch.randn(tokens, width, generator=g, device="cuda") * s).to(torch.bfloat16)
    x, d_out, d_z = r(1.0), r(1e-2), r(1e-2)
    x_out, z, s = block.forward(x)
    grads = block.backward(d_out, d_z, s)
    assert F.fp8_device_status() == 0

    f64 = lambda t: t.detach().double().requires_grad_(True)
    p = {n: f64(getattr(block, n)) for n in ("w_pre", "w_post", "w_next", "gate", "w_in", "w_out")}
    p["x"], p["w"] = f64(x), f64(s["w"])
    y = _rms(p["x"], p["w_pre"])
    b = torch.zeros_like(y)
    for j in range(slots):
        for e in range(experts):
            t = (s["ids"][:, j] == e).nonzero()[:, 0]
            if t.numel():
                v = y[t] @ p["w_in"][e].t()
                h = torch.nn.functional.silu(v[:, :hidden]) * v[:, hidden:]
                b = b.index_add(0, t, (h @ p["w_out"][e].t()) * p["w"][t, j, None])
    xo = 0.9 * p["x"] + p["gate"] * _rms(b, p["w_post"])
    zo = _rms(xo, p["w_next"])
    off = lambda got, want: ((got.double() - want).norm() / want.norm()).item()
    assert off(x_out, xo) < 2 ** -2.5 and off(z, zo) < 2 ** -2.5
    ((xo * d_out.double()).sum() + (zo * d_z.double()).sum()).backward()
    for name, t in p.items():
        assert off(grads[name].view(t.shape), t.grad) < 0.25, name
