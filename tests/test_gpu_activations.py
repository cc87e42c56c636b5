"""The activations over their whole range, forward and backward, against 64
bits with relative bounds.

With z exact, act(z) and act'(z) are products and sums of a few fp32 terms.  A
term's relative error is that of its exponent: an argument of at most 50 (z in
[-8, 8]) that saw four roundings of 2^-24, so 200 x 2^-24, and a few units in
the last place of the functions: below 2^-15 of the term.  The derivative is
held to 2^-15 of the sum of its terms' magnitudes.  The bf16 rounding comes on
top (tests/block_ref.py)."""
import math

import pytest
import torch

import scaled_fp8_linear_gb300 as F
from tests import block_ref as R

pytestmark = pytest.mark.gpu
DEV, F64, BF = "cuda", torch.float64, torch.bfloat16
ACTS = [F.ACT_NONE, F.ACT_RELU, F.ACT_SILU, F.ACT_GELU, F.ACT_GELU_TANH]
U = 2.0 ** -15


def _gates(z, act):
    """The factor s of act(z) = z s, its derivative by z, without cancellation."""
    if act == F.ACT_RELU:
        return (z > 0).to(F64), torch.zeros_like(z)
    if act == F.ACT_SILU:
        return torch.sigmoid(z), torch.sigmoid(z) * torch.sigmoid(-z)
    if act == F.ACT_GELU:
        return 0.5 * torch.erfc(-z / math.sqrt(2)), torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == F.ACT_GELU_TANH:
        u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        du = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
        return torch.sigmoid(u), torch.sigmoid(u) * torch.sigmoid(-u) * du
    return torch.ones_like(z), torch.zeros_like(z)


def _backward(z, act):
    """fp8_act_bwd with dD and the up product 1: act'(z) and act(z)."""
    n = (z.numel() + 15) // 16 * 16
    zz = torch.ones(1, 2 * n, dtype=BF)
    zz[0, :n] = torch.cat([z, z.new_zeros(n - z.numel())])
    dz = F.fp8_act_bwd(torch.ones(1, n, dtype=BF, device=DEV), zz.to(DEV), act, gated=True).dz[0]
    return dz[:z.numel()], dz[n:n + z.numel()]


def _forward(z, act):
    """D of a product whose z is the row factors themselves (fp32)."""
    one_hot = torch.zeros(max(z.numel(), 16), 16, dtype=torch.uint8, device=DEV)
    one_hot[:, 0] = 0x38                     # 1.0 in E4M3
    one = torch.ones(16, device=DEV)
    return F.fp8_gemm_act(one_hot[:z.numel()], F.E4M3, one_hot[:16], F.E4M3, z.to(DEV), one, ga=F.GRAN_ROW,
                          gb=F.GRAN_ROW, act=act).d[:, 0]


@pytest.mark.parametrize("act", ACTS)
def test_whole_range(act):
    z = torch.linspace(-8, 8, 1025).to(BF)
    s, ds = _gates(z.to(F64), act)
    a, g = z.to(F64) * s, s + z.to(F64) * ds
    got_g, got_a = _backward(z, act)
    R.check(got_a, a, a.abs(), "act, backward", U * a.abs())
    m = s + (z.to(F64) * ds).abs()
    R.check(got_g, g, m, "derivative", U * m)
    z = torch.linspace(-8, 8, 1025)
    a = z.to(F64) * _gates(z.to(F64), act)[0]
    R.check(_forward(z, act), a, a.abs(), "act, forward", U * a.abs())


@pytest.mark.parametrize("act", ACTS)
def test_largest_values(act):
    """Up to the largest bf16 and fp32 values, finite and right; from 1e5 on
    every activation is z (or 0, on its negative side) and its derivative 1
    (or 0), exactly."""
    z = torch.tensor([40.0, 1e5, 1e10, 2e19, 1e20, 1e30, 3e38]).to(BF)
    for sign in (1.0, -1.0):
        on = float(sign > 0 or act == F.ACT_NONE)
        s, ds = _gates(sign * z.to(F64), act)
        g, a = _backward(sign * z, act)
        d = _forward((sign * z).float(), act)
        m = s + (z.to(F64) * ds).abs()
        R.check(g, s + sign * z.to(F64) * ds, m, "derivative", U * m)
        R.check(a, sign * z.to(F64) * s, z.to(F64) * s, "act, backward", U * z.to(F64) * s)
        R.check(d, sign * z.to(F64) * s, z.to(F64) * s, "act, forward", U * z.to(F64) * s)
        assert torch.equal(g.cpu()[1:], torch.full_like(z[1:], on)), (act, sign)
        assert torch.equal(a.cpu()[1:], on * sign * z[1:]), (act, sign)
        assert torch.equal(d.cpu()[1:], on * sign * z[1:]), (act, sign)
