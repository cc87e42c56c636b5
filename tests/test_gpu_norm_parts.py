"""The norms with every combination of parts, at widths that reach each of
their kernels: rows in 16-byte pieces over a warp (256, 512) and over a CTA
(4096, 768 with idle threads, 16384), and other widths of each kind; against
64 bits (tests/block_ref.py has the bounds)."""
import pytest
import torch

import scaled_fp8_linear_gb300 as F
from tests import block_ref as R
from tests.test_gpu_norm import _64, _d, _g, _inputs

pytestmark = pytest.mark.gpu
F64, BF = torch.float64, torch.bfloat16

WIDTHS = [256, 512, 768, 4096, 16384, 100, 500, 999, 4095, 9001]
PARTS = [(False, 0), (False, 1), (False, 3), (True, 0), (True, 3)]


@pytest.fixture(scope="module", autouse=True)
def _status():
    yield
    assert F.fp8_device_status() == 0


def _parts(T, C, kind, stream, post, G, seed):
    x, h, gate, w1, b1, w2, b2 = _inputs(T, C, kind, stream, G, seed=seed)
    if not post:
        w1 = b1 = None
    return x, h, gate, w1, b1, w2, b2


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
@pytest.mark.parametrize("stream", [BF, torch.float32])
@pytest.mark.parametrize("post,G", PARTS)
@pytest.mark.parametrize("C", WIDTHS)
def test_forward(C, post, G, stream, kind):
    T = 39
    x, h, gate, w1, b1, w2, b2 = _parts(T, C, kind, stream, post, G, 1)
    o = F.fp8_norm_fwd(_d(x), _d(h), kind=kind, alpha=0.75, gate=_d(gate), post_norm=post, w_post=_d(w1),
                       b_post=_d(b1), w_pre=_d(w2), b_pre=_d(b2), want_stats=True)
    xo, xm, y, ym, st = R.norm_fwd(_64(x), _64(h), _64(gate), kind, 1e-5, 0.75, post, _64(w1), _64(b1), _64(w2), _64(b2))
    R.check(o.x_out, xo, xm, "x_out")
    R.check(o.y, y, ym, "y")
    R.check(o.stats[2], st[2], xm.mean(1) + st[2].abs(), "mean")
    R.check(o.stats[3], st[3], st[3] * (1 + 2 * (xm * st[3][:, None]).square().mean(1)), "rstd")


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
@pytest.mark.parametrize("stream", [BF, torch.float32])
@pytest.mark.parametrize("post,G", PARTS)
@pytest.mark.parametrize("C", WIDTHS)
def test_backward(C, post, G, stream, kind):
    """All parts, and the same without dx' (the kernels that test their parts
    as they run)."""
    T = 39 if C > 600 else 2499           # more rows than one batch a CTA
    x, h, gate, w1, b1, w2, b2 = _parts(T, C, kind, stream, post, G, 2)
    g = _g(9)
    dy, dxo = torch.randn(T, C, generator=g).to(BF), torch.randn(T, C, generator=g).to(stream)
    args = dict(kind=kind, alpha=1.25, gate=_d(gate), post_norm=post, w_post=_d(w1), b_post=_d(b1), w_pre=_d(w2),
                b_pre=_d(b2))
    f = F.fp8_norm_fwd(_d(x), _d(h), want_stats=True, **args)
    st, xo = _64(f.stats.cpu()), _64(f.x_out.cpu())
    for over in (dxo, None):
        o = F.fp8_norm_bwd(_d(dy), f.x_out, f.stats, dx_out=_d(over), h=_d(h), **args)
        ref = R.norm_bwd(_64(dy), xo, _64(over), _64(h), _64(gate), st, kind, 1.25, post, _64(w1), _64(b1), _64(w2))
        for name, got in o._asdict().items():
            if got is not None:
                R.check(got, *ref[name], name)


@pytest.mark.parametrize("C", [256, 4096, 999, 16384])
def test_backward_without_the_block(C):
    """No h: the gradient of a norm alone, and dx over dx'."""
    T = 300
    x, _, _, _, _, w2, _ = _parts(T, C, F.NORM_RMS, BF, False, 0, 3)
    g = _g(5)
    dy, dxo = torch.randn(T, C, generator=g).to(BF), torch.randn(T, C, generator=g).to(BF)
    f = F.fp8_norm_fwd(_d(x), w_pre=_d(w2), want_stats=True)
    ref = R.norm_bwd(_64(dy), _64(f.x_out.cpu()), _64(dxo), None, None, _64(f.stats.cpu()), 0, 1.0, False, None, None,
                     _64(w2))
    dx = _d(dxo)
    o = F.fp8_norm_bwd(_d(dy), f.x_out, f.stats, dx_out=dx, w_pre=_d(w2), dx=dx)
    R.check(dx, *ref["dx"], "dx")
    R.check(o.dw_pre, *ref["dw_pre"], "dw_pre")
    assert o.dh is None
