"""The norms around a block, against 64 bits (tests/block_ref.py has the bounds)."""
import pytest
import torch

import scaled_fp8_linear_gb300 as F
from tests import block_ref as R

pytestmark = pytest.mark.gpu
DEV, F64, BF = "cuda", torch.float64, torch.bfloat16


def _g(seed):
    return torch.Generator().manual_seed(seed)


def _inputs(T, C, kind, stream, gate_rows, seed=0, spread=1.0):
    g = _g(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    x = (r(T, C) * spread).to(stream)
    h = (r(T, C) * (0.1 + torch.rand(T, 1, generator=g))).to(BF)
    gate = r(gate_rows, C).to(BF) if gate_rows else None
    w1, w2 = 1 + 0.2 * r(C), 1 + 0.2 * r(C)
    b1, b2 = (0.3 * r(C), 0.3 * r(C)) if kind == F.NORM_LAYER else (None, None)
    return x, h, gate, w1, b1, w2, b2


def _d(t):
    return None if t is None else t.to(DEV)


def _64(t):
    return None if t is None else t.to(F64)


SHAPES = [(1, 1, 0), (3, 7, 1), (2, 8, 2), (5, 64, 0), (9, 250, 3), (33, 256, 1), (7, 504, 7),
          (6, 1000, 2), (8, 1024, 1), (5, 1032, 5), (12, 3000, 4), (300, 4096, 1), (4, 8192, 2),
          (3, 8200, 1), (2, 16384, 1), (2, 16383, 0)]


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
@pytest.mark.parametrize("stream", [BF, torch.float32])
@pytest.mark.parametrize("T,C,G", SHAPES)
def test_forward(T, C, G, stream, kind):
    x, h, gate, w1, b1, w2, b2 = _inputs(T, C, kind, stream, G)
    eps, alpha = 1e-5, 0.75
    o = F.fp8_norm_fwd(_d(x), _d(h), kind=kind, eps=eps, alpha=alpha, gate=_d(gate), post_norm=True,
                       w_post=_d(w1), b_post=_d(b1), w_pre=_d(w2), b_pre=_d(b2), want_stats=True)
    xo, xm, y, ym, st = R.norm_fwd(_64(x), _64(h), _64(gate), kind, eps, alpha, True, _64(w1),
                                   _64(b1), _64(w2), _64(b2))
    R.check(o.x_out, xo, xm, "x_out")
    R.check(o.y, y, ym, "y")
    # a statistic moves with its row's magnitudes (eps bounds rstd for C = 1)
    R.check(o.stats[2], st[2], xm.mean(1) + st[2].abs(), "mean")
    scale = (xm * st[3][:, None]).square().mean(1)
    R.check(o.stats[3], st[3], st[3] * (1 + 2 * scale), "rstd")


@pytest.mark.parametrize("gran,pow2,fmt", [(F.GRAN_TENSOR, False, F.E4M3), (F.GRAN_ROW, False, F.E4M3),
                                           (F.GRAN_ROW, True, F.E5M2)])
@pytest.mark.parametrize("T,C", [(1, 16), (5, 999), (17, 1024), (9, 4096), (3, 8192)])
def test_codes(T, C, gran, pow2, fmt):
    x, h, _, _, _, w2, _ = _inputs(T, C, F.NORM_RMS, BF, 0, seed=3)
    if T > 2:
        x[1], h[1] = 0, 0          # a row of zeros: scale 1
    scale = torch.tensor([37.5]) if gran == F.GRAN_TENSOR else None
    o = F.fp8_norm_fwd(_d(x), _d(h), w_pre=_d(w2), q_fmt=fmt, q_gran=gran, q_scale=_d(scale),
                       pow2=pow2, want_amax=gran == F.GRAN_TENSOR)
    _, _, y, ym, _ = R.norm_fwd(_64(x), _64(h), None, F.NORM_RMS, 1e-5, 1.0, False, None, None,
                                _64(w2), None)
    R.check(o.y, y, ym, "y")
    if gran == F.GRAN_TENSOR:
        s = torch.full((T, 1), 37.5, dtype=F64)
        R.check(o.amax, y.abs().amax().view(1), ym.amax().view(1), "amax")
    else:
        inv = o.q_scale_inv.to(F64).cpu()
        top = 448.0 if fmt == F.E4M3 else 57344.0
        a = y.abs().amax(1)
        want = torch.where(a > 0, a / top, torch.ones_like(a))
        if pow2:
            assert torch.equal(torch.frexp(inv)[0], torch.full_like(inv, 0.5))
            assert ((inv >= want * (1 - 1e-5)) & (inv < 2 * want * (1 + 1e-5))).all()
        else:
            assert ((inv - want).abs() <= R.U_F32 * (ym.amax(1) / top + want)).all()
        s = (1 / inv)[:, None]
    R.check_codes(o.q, fmt, y * s, R.U_F32 * ym * s * 2, "codes")


def test_forms():
    """Without h, without x, without the pre norm's weights, in place, and a
    constant row (variance 0: eps decides)."""
    x, h, gate, w1, _, w2, _ = _inputs(6, 512, F.NORM_RMS, BF, 2, seed=5)
    o = F.fp8_norm_fwd(_d(x), alpha=1.0, want_x_out=False)
    _, _, y, ym, _ = R.norm_fwd(_64(x), None, None, 0, 1e-5, 1.0, False, None, None, None, None)
    assert o.x_out is None
    R.check(o.y, y, ym, "y of x alone")
    o = F.fp8_norm_fwd(None, _d(h), gate=_d(gate), w_pre=_d(w2))
    xo, xm, y, ym, _ = R.norm_fwd(None, _64(h), _64(gate), 0, 1e-5, 1.0, False, None, None, _64(w2), None)
    R.check(o.x_out, xo, xm, "x_out of h alone")
    R.check(o.y, y, ym, "y of h alone")
    xs = _d(x)
    o = F.fp8_norm_fwd(xs, _d(h), x_out=xs, want_y=False)
    R.check(xs, _64(x) + _64(h), _64(x).abs() + _64(h).abs(), "in place")
    c = torch.full((3, 640), 2.5)
    o = F.fp8_norm_fwd(_d(c), kind=F.NORM_LAYER, eps=1e-6)
    assert torch.equal(o.y.cpu(), torch.zeros(3, 640, dtype=BF))


def test_nan_and_inf_stay_in_their_rows():
    x, h, *_ = _inputs(5, 2048, F.NORM_RMS, BF, 0, seed=6)
    x[1, 7], x[3, 100] = float("nan"), float("inf")
    o = F.fp8_norm_fwd(_d(x), _d(h), q_fmt=F.E4M3, q_scale=torch.ones(1, device=DEV), want_amax=True)
    assert not torch.isfinite(o.y[1]).any() and torch.isfinite(o.y[[0, 2, 4]]).all()
    assert torch.isnan(o.amax).all()


def test_no_rows():
    x = torch.empty(0, 256, dtype=BF, device=DEV)
    w = torch.ones(256, device=DEV)
    o = F.fp8_norm_fwd(x, x, want_stats=True)
    assert o.y.shape == (0, 256)
    b = F.fp8_norm_bwd(x, x, o.stats, h=x, w_pre=w, gate=torch.ones(2, 256, dtype=BF, device=DEV))
    assert not b.dw_pre.any() and not b.dgate.any()


@pytest.mark.parametrize("kind", [F.NORM_RMS, F.NORM_LAYER])
@pytest.mark.parametrize("stream", [BF, torch.float32])
@pytest.mark.parametrize("T,C,G", SHAPES + [(700, 128, 1), (641, 512, 641), (400, 2048, 4), (512, 640, 128),
                                            (200, 3, 100), (67, 1, 67), (1000, 13, 4), (333, 333, 3), (90, 4001, 30),
                                            (640, 4096, 640), (320, 8192, 160), (320, 4097, 320)])
def test_backward(T, C, G, stream, kind):
    x, h, gate, w1, b1, w2, b2 = _inputs(T, C, kind, stream, G, seed=1)
    g = _g(9)
    dy = torch.randn(T, C, generator=g).to(BF)
    dxo = torch.randn(T, C, generator=g).to(stream)
    args = dict(kind=kind, alpha=1.25, gate=_d(gate), post_norm=True, w_post=_d(w1), b_post=_d(b1),
                w_pre=_d(w2), b_pre=_d(b2))
    f = F.fp8_norm_fwd(_d(x), _d(h), want_stats=True, **args)
    o = F.fp8_norm_bwd(_d(dy), f.x_out, f.stats, dx_out=_d(dxo), h=_d(h), **args)
    ref = R.norm_bwd(_64(dy), _64(f.x_out.cpu()), _64(dxo), _64(h), _64(gate), _64(f.stats.cpu()),
                     kind, 1.25, True, _64(w1), _64(b1), _64(w2))
    for name, got in o._asdict().items():
        if got is not None:
            R.check(got, *ref[name], name)
    again = F.fp8_norm_bwd(_d(dy), f.x_out, f.stats, dx_out=_d(dxo), h=_d(h), **args)
    for name, got in o._asdict().items():
        assert got is None or torch.equal(got, getattr(again, name)), f"{name}: other bits"


def test_backward_parts():
    """Only dy, only dx_out, no post norm, accumulation into given sums."""
    T, C = 37, 768
    x, h, gate, w1, _, w2, _ = _inputs(T, C, F.NORM_RMS, BF, 1, seed=2)
    g = _g(4)
    dy, dxo = torch.randn(T, C, generator=g).to(BF), torch.randn(T, C, generator=g).to(BF)
    f = F.fp8_norm_fwd(_d(x), _d(h), gate=_d(gate), w_pre=_d(w2), want_stats=True)
    st, xo = _64(f.stats.cpu()), _64(f.x_out.cpu())
    old = torch.randn(C, generator=g)
    dw, dg = _d(old), _d(old).view(1, C).clone()
    o = F.fp8_norm_bwd(_d(dy), f.x_out, f.stats, h=_d(h), gate=_d(gate), w_pre=_d(w2), dw_pre=dw,
                       dgate=dg, accumulate=True)
    ref = R.norm_bwd(_64(dy), xo, None, _64(h), _64(gate), st, 0, 1.0, False, None, None, _64(w2))
    for name in ("dx", "dh"):
        R.check(getattr(o, name), *ref[name], name)
    R.check(dw, ref["dw_pre"][0] + old, ref["dw_pre"][1] + old.abs(), "dw_pre added")
    R.check(dg, ref["dgate"][0] + old, ref["dgate"][1] + old.abs(), "dgate added")
    o = F.fp8_norm_bwd(None, f.x_out, f.stats, dx_out=_d(dxo), h=_d(h), gate=_d(gate))
    ref = R.norm_bwd(None, xo, _64(dxo), _64(h), _64(gate), st, 0, 1.0, False, None, None, None)
    for name in ("dx", "dh", "dgate"):
        R.check(getattr(o, name), *ref[name], name)
    assert o.dw_pre is None
    dx = _d(dxo)
    o = F.fp8_norm_bwd(_d(dy), f.x_out, f.stats, dx_out=dx, w_pre=_d(w2), dx=dx)
    ref = R.norm_bwd(_64(dy), xo, _64(dxo), None, None, st, 0, 1.0, False, None, None, _64(w2))
    R.check(dx, *ref["dx"], "dx in place")


def test_another_stream_and_a_graph():
    x, h, _, _, _, w2, _ = _inputs(64, 1024, F.NORM_RMS, BF, 0, seed=8)
    x, h, w2 = _d(x), _d(h), _d(w2)
    want = F.fp8_norm_fwd(x, h, w_pre=w2).y
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(h)
    F.fp8_norm_fwd(x, h, w_pre=w2, y=y, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)
    graph, y2, xo = torch.cuda.CUDAGraph(), torch.empty_like(h), torch.empty_like(x)
    with torch.cuda.graph(graph):
        F.fp8_norm_fwd(x, h, w_pre=w2, y=y2, x_out=xo)
    x.mul_(2)
    graph.replay()
    assert torch.equal(y2, F.fp8_norm_fwd(x, h, w_pre=w2).y)


def test_binding_refusals_of_tensors():
    """Strided, misaligned and host tensors, and other types, before a launch."""
    x = torch.randn(64, 64, device=DEV).to(BF)
    with pytest.raises(ValueError, match="contiguous"):
        F.fp8_norm_fwd(x.t())
    with pytest.raises(ValueError, match="CUDA"):
        F.fp8_norm_fwd(x, x.cpu())
    with pytest.raises(TypeError):
        F.fp8_norm_fwd(x, w_pre=torch.ones(64, device=DEV, dtype=BF))
    with pytest.raises(ValueError, match="shape"):
        F.fp8_norm_fwd(x, w_pre=torch.ones(65, device=DEV))
    with pytest.raises(F.Fp8Error) as e:
        F.fp8_norm_fwd(x.view(-1)[4:4 + 63 * 64].view(63, 64))
    assert e.value.status == -3
    ids = torch.zeros(4, 2, device=DEV, dtype=torch.int64)
    with pytest.raises(TypeError):
        F.fp8_moe_plan(ids, 4)
    with pytest.raises(TypeError):
        F.fp8_gemm_act(x, 0, x, 0, torch.ones(1, device=DEV), torch.ones(1, device=DEV))


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows equal the same rows alone."""
    T, C = (1 << 18) + 5, 8192
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(T, C, dtype=BF, device=DEV)
    x.normal_(generator=g)
    w = 1 + 0.1 * torch.randn(C, device=DEV)
    f = F.fp8_norm_fwd(x, x, w_pre=w, want_stats=True)
    tail = x[-7:].contiguous()
    ft = F.fp8_norm_fwd(tail, tail, w_pre=w, want_stats=True)
    assert torch.equal(f.y[-7:], ft.y) and torch.equal(f.x_out[-7:], ft.x_out)
    assert torch.equal(f.stats[:, -7:], ft.stats)
    b = F.fp8_norm_bwd(f.y, f.x_out, f.stats, dx_out=x, h=x, w_pre=w)
    bt = F.fp8_norm_bwd(ft.y, ft.x_out, ft.stats, dx_out=tail, h=tail, w_pre=w)
    assert torch.equal(b.dx[-7:], bt.dx) and torch.equal(b.dh[-7:], bt.dh)
