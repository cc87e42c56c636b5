"""Activations in blocks of 128 with 8-bit checkpoints, their gradient, and the
transposing re-cast.

What is a cast of given numbers (the checkpoint, the transpose) is compared bit
for bit with the rule in FP32.  A computed value v is known to within 2^-17 of
its terms' magnitudes (tests/block_ref.py: fewer than 64 roundings of 2^-24 and
the functions' own error, at most 2^-18), so a factor is within 2^-16 of its
reference and a code within half a step of v times the scale that its factor
says."""
import pytest
import torch

import scaled_fp8_linear_gb300 as F
from tests import block_ref as R
from tests import expert_ref as E

pytestmark = pytest.mark.gpu
DEV, F64, BF = "cuda", torch.float64, torch.bfloat16
ACTS = [F.ACT_NONE, F.ACT_RELU, F.ACT_SILU, F.ACT_GELU, F.ACT_GELU_TANH]
SHAPES = [(1, 128), (3, 256), (16, 128), (129, 384), (700, 640)]


@pytest.fixture(scope="module", autouse=True)
def _status():
    yield
    assert F.fp8_device_status() == 0


def _check_block(q, inv, fmt, v, mag, pow2, what):
    """Codes q and factors inv of v [rows, cols] known to within 2^-17 mag."""
    q, inv = q.cpu(), inv.cpu().to(F64)
    b, bm = v.unflatten(1, (-1, 128)), mag.unflatten(1, (-1, 128))
    top, tol = b.abs().amax(2), (bm.abs() * R.U_F32).amax(2)
    ref = torch.where(top > 0, top / E.TOP[fmt], torch.ones_like(top))
    if pow2:
        lo = 2.0 ** torch.ceil(torch.log2((top - tol).clamp_min(2.0 ** -126) / E.TOP[fmt]) - 2.0 ** -30)
        hi = 2.0 ** torch.ceil(torch.log2((top + tol).clamp_min(2.0 ** -126) / E.TOP[fmt]) + 2.0 ** -30)
        ok = ((inv >= lo) & (inv <= hi)) | ((top <= tol) & (inv == 1))
    else:
        ok = ((inv - ref).abs() <= 2.0 ** -22 * ref + tol / E.TOP[fmt]) | ((top <= tol) & (inv == 1))
    assert ok.all(), f"{what}: factors"
    s = (1.0 / inv).repeat_interleave(128, dim=1)
    R.check_codes(q, fmt, v * s, (mag * R.U_F32 + v.abs() * 2.0 ** -22) * s, what)


def _act_case(M, N, act, gated, seed, std=3.0):
    g = torch.Generator().manual_seed(seed)
    W = 2 * N if gated else N
    z = (torch.randn(M, W, generator=g) * std).to(BF)
    z64 = z.to(F64)
    h = R.act(z64[:, :N], act)
    mag = h.abs() + z64[:, :N].abs() * 2.0 ** -20
    if gated:
        h, mag = h * z64[:, N:], mag * z64[:, N:].abs()
    return z, h, mag


def _live(off, M):
    at = E.held(off, M)
    return slice(at[0], at[-1])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", SHAPES)
def test_forward(M, N, act, gated):
    z, h, mag = _act_case(M, N, act, gated, M + act)
    for fmt, pow2 in ((F.E4M3, False), (F.E5M2, True)):
        o = F.fp8_act_block(z.to(DEV), act, gated=gated, q_fmt=fmt, pow2=pow2, keep=True)
        _check_block(o.q, o.scale_inv, fmt, h, mag, pow2, "h")
        q, inv = E.cast(z.float(), F.E4M3, pow2)
        assert torch.equal(o.z_q.cpu(), q) and torch.equal(o.z_scale_inv.cpu(), inv)
        cast = F.fp8_quantize_blocks(z.to(DEV), F.E4M3, F.GRAN_1x128, pow2=pow2)
        assert torch.equal(o.z_q, cast[0]) and torch.equal(o.z_scale_inv, cast[1])
        only = F.fp8_act_block(z.to(DEV), act, gated=gated, q_fmt=fmt, pow2=pow2)
        kept = F.fp8_act_block(z.to(DEV), act, gated=gated, pow2=pow2, want_q=False, keep=True)
        assert only.z_q is None and torch.equal(only.q, o.q) and torch.equal(only.scale_inv, o.scale_inv)
        assert kept.q is None and torch.equal(kept.z_q, o.z_q) and torch.equal(kept.z_scale_inv, o.z_scale_inv)


def test_forward_of_a_large_call():
    """More rows a warp than a small call has."""
    z, h, mag = _act_case(6001, 2048, F.ACT_SILU, True, 1)
    o = F.fp8_act_block(z.to(DEV), F.ACT_SILU, gated=True, keep=True)
    _check_block(o.q, o.scale_inv, F.E4M3, h, mag, False, "h")
    q, inv = E.cast(z.float(), F.E4M3, False)
    assert torch.equal(o.z_q.cpu(), q) and torch.equal(o.z_scale_inv.cpu(), inv)


@pytest.mark.parametrize("M,N", [(70, 256), (5000, 2048)])
@pytest.mark.parametrize("cut", [[0, 30, 64], [5, 5, 70], [9, 40, 20], [-3, 12, 10 ** 6], [0, 0, 0]])
def test_forward_of_experts_rows(M, N, cut):
    z, h, mag = _act_case(M, N, F.ACT_SILU, True, 2)
    s = _live(cut, M)
    z[:s.start], z[s.stop:] = float("nan"), float("nan")
    out = [torch.full((M, w), 9, dtype=torch.uint8, device=DEV) for w in (N, 2 * N)]
    inv = [torch.full((M, w // 128), 7.0, device=DEV) for w in (N, 2 * N)]
    F.fp8_act_block(z.to(DEV), F.ACT_SILU, gated=True, q=out[0], scale_inv=inv[0], z_q=out[1], z_scale_inv=inv[1],
                    offsets=torch.tensor(cut, dtype=torch.int32, device=DEV))
    for t, v in [(t, 9) for t in out] + [(t, 7.0) for t in inv]:
        assert (t[:s.start] == v).all() and (t[s.stop:] == v).all()
    if s.stop > s.start:
        _check_block(out[0][s], inv[0][s], F.E4M3, h[s], mag[s], False, "h")
        q, f = E.cast(z[s].float(), F.E4M3, False)
        assert torch.equal(out[1][s].cpu(), q) and torch.equal(inv[1][s].cpu(), f)


def test_blocks_of_zeros_and_of_what_is_not_finite():
    z = torch.randn(4, 512, generator=torch.Generator().manual_seed(3)).to(BF)
    z[0] = 0
    z[1, 3], z[2, 130], z[3, 260] = float("nan"), float("inf"), -float("inf")
    o = F.fp8_act_block(z.to(DEV), F.ACT_NONE, gated=True, keep=True)
    q, inv = E.cast(z.float(), F.E4M3, False)
    nan = torch.isnan(z)
    assert torch.equal(o.z_q.cpu()[~nan], q[~nan]) and (o.z_q.cpu()[nan] & 0x7F == 0x7F).all()
    assert torch.equal(o.z_scale_inv.cpu(), inv)
    assert (o.z_scale_inv[0] == 1).all() and o.z_scale_inv[1, 0] == 1 and o.z_scale_inv[2, 1] == 1
    h = z.float()[:, :256] * z.float()[:, 256:]
    q, inv = E.cast(h, F.E4M3, False)
    ok = ~torch.isnan(h)
    assert torch.equal(o.q.cpu()[ok], q[ok]) and torch.equal(o.scale_inv.cpu(), inv)


# ------------------------------------------------------------------ gradient

def _bwd_case(M, N, act, gated, seed):
    g = torch.Generator().manual_seed(seed)
    W = 2 * N if gated else N
    d = (torch.randn(M, N, generator=g) * 1e-2).to(BF)
    zq, inv = E.cast((torch.randn(M, W, generator=g) * 2).to(BF).float(), F.E4M3, False)
    z = (E.values(zq, 0).float().unflatten(1, (-1, 128)) * inv[..., None]).flatten(1).to(F64)   # exact but for one rounding
    d64 = d.to(F64)
    gr, a = R.act_grad(z[:, :N], act), R.act(z[:, :N], act)
    m = d64.abs() * (1 + z[:, :N].abs())
    hm = a.abs() + z[:, :N].abs() * 2.0 ** -20
    if gated:
        up = z[:, N:]
        dz, mag = torch.cat([d64 * up * gr, d64 * a], 1), torch.cat([m * up.abs(), m], 1)
        h, hm = a * up, hm * up.abs()
    else:
        dz, mag, h = d64 * gr, m, a
    return d, zq, inv, dz, mag, h, hm


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", SHAPES + [(128, 128), (384, 256), (640, 384)])
def test_backward(M, N, act, gated):
    d, zq, inv, dz, mag, h, hm = _bwd_case(M, N, act, gated, M + act)
    tokens = M % 128 == 0
    for fmt, h_fmt, pow2 in ((F.E5M2, F.E4M3, False), (F.E4M3, F.E5M2, True)):
        o = F.fp8_act_block_bwd(d.to(DEV), zq.to(DEV), inv.to(DEV), act, gated=gated, q_fmt=fmt, h_fmt=h_fmt, pow2=pow2,
                                want_t=tokens, want_h_t=tokens)
        _check_block(o.q, o.scale_inv, fmt, dz, mag, pow2, "dz")
        if not tokens:
            assert o.q_t is None and o.h_t is None
            continue
        _check_block(o.q_t, o.scale_inv_t, fmt, dz.t().contiguous(), mag.t().contiguous(), pow2, "dz^T")
        _check_block(o.h_t, o.h_scale_inv_t, h_fmt, h.t().contiguous(), hm.t().contiguous(), pow2, "h^T")
        for kw, names in ((dict(want_q=False, want_t=True), ("q_t", "scale_inv_t")),
                          (dict(want_q=False, want_h_t=True), ("h_t", "h_scale_inv_t")),
                          (dict(), ("q", "scale_inv"))):
            p = F.fp8_act_block_bwd(d.to(DEV), zq.to(DEV), inv.to(DEV), act, gated=gated, q_fmt=fmt, h_fmt=h_fmt,
                                    pow2=pow2, **kw)
            for name in p._fields:
                got = getattr(p, name)
                assert (got is None) == (name not in names)
                assert got is None or torch.equal(got, getattr(o, name)), name


@pytest.mark.parametrize("cut", [[0, 128, 256], [0, 100, 300], [128, 128, 384], [130, 200, 140], [-1, 5, 10 ** 6],
                                 [0, 0, 0], [512, 512, 512], [255, 256, 257]])
def test_backward_of_experts_rows(cut):
    M, N, act = 512, 256, F.ACT_SILU
    d, zq, inv, dz, mag, h, hm = _bwd_case(M, N, act, True, 5)
    s = _live(cut, M)
    out = torch.ones(M, 1, dtype=F64)
    out[s] = 0
    for t in (dz, mag, h, hm):                  # the others' rows count as zeros
        t *= 1 - out
    d[:s.start], d[s.stop:] = float("nan"), float("inf")
    zq[:s.start], zq[s.stop:] = 0x7F, 0x7F
    inv[:s.start], inv[s.stop:] = float("nan"), float("nan")
    b = lambda *shape: torch.full(shape, 9, dtype=torch.uint8, device=DEV)
    f = lambda *shape: torch.full(shape, 7.0, device=DEV)
    o = F.fp8_act_block_bwd(d.to(DEV), zq.to(DEV), inv.to(DEV), act, gated=True, q=b(M, 2 * N), scale_inv=f(M, 4),
                            q_t=b(2 * N, M), scale_inv_t=f(2 * N, 4), h_t=b(N, M), h_scale_inv_t=f(N, 4),
                            offsets=torch.tensor(cut, dtype=torch.int32, device=DEV))
    assert (o.q[:s.start] == 9).all() and (o.q[s.stop:] == 9).all()
    assert (o.scale_inv[:s.start] == 7).all() and (o.scale_inv[s.stop:] == 7).all()
    if s.stop > s.start:
        _check_block(o.q[s], o.scale_inv[s], F.E5M2, dz[s], mag[s], False, "dz")
    for t in range(4):
        r = slice(128 * t, 128 * t + 128)
        if r.stop <= s.start or r.start >= s.stop:   # a block without rows of experts
            for x, v in ((o.q_t[:, r], 9), (o.h_t[:, r], 9), (o.scale_inv_t[:, t], 7), (o.h_scale_inv_t[:, t], 7)):
                assert (x == v).all()
        else:
            _check_block(o.q_t[:, r], o.scale_inv_t[:, t:t + 1], F.E5M2, dz[r].t().contiguous(),
                         mag[r].t().contiguous(), False, "dz^T")
            _check_block(o.h_t[:, r], o.h_scale_inv_t[:, t:t + 1], F.E4M3, h[r].t().contiguous(),
                         hm[r].t().contiguous(), False, "h^T")


# ------------------------------------------------------------------ transpose

@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("fmt", [F.E4M3, F.E5M2])
@pytest.mark.parametrize("T,C", [(128, 128), (256, 384), (640, 256), (1280, 1152)])
def test_transpose(T, C, fmt, pow2):
    g = torch.Generator().manual_seed(T + C)
    q = E.any_codes(g, fmt, T, C)
    q[:, 5] = 0
    inv = E.exact_factors(g, T, C // 128) * (1.0 if pow2 else 0.1) + (0.0 if pow2 else 0.03)
    x = (q.view(E.TYPE[fmt]).float().unflatten(1, (-1, 128)) * inv[..., None]).flatten(1)
    want, want_inv = E.cast(x.t().contiguous(), fmt, pow2)
    got, got_inv = F.fp8_block_transpose(q.to(DEV), fmt, inv.to(DEV), pow2=pow2)
    assert torch.equal(got.cpu(), want) and torch.equal(got_inv.cpu(), want_inv)


def test_transpose_of_nothing_and_of_nan():
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=DEV)
    q, inv = F.fp8_block_transpose(z(0, 256), F.E4M3, torch.zeros(0, 2, device=DEV))
    assert q.shape == (256, 0) and inv.shape == (256, 0)
    q = z(128, 128)
    q[3, 7], q[:, 9] = 0x7F, 0x38
    got, inv = F.fp8_block_transpose(q, F.E4M3, torch.ones(128, 1, device=DEV))
    assert got[7, 3] == 0x7F and inv[7] == 1 and (got[9] == 0x7E).all() and inv[0] == 1 and (got[0] == 0).all()


def test_no_rows():
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device=DEV)
    o = F.fp8_act_block(z(0, 256, dt=BF), F.ACT_SILU, gated=True, keep=True)
    assert o.q.shape == (0, 128) and o.z_q.shape == (0, 256) and o.z_scale_inv.shape == (0, 2)
    b = F.fp8_act_block_bwd(z(0, 128, dt=BF), o.z_q, o.z_scale_inv, F.ACT_SILU, gated=True, want_t=True, want_h_t=True)
    assert b.q.shape == (0, 256) and b.q_t.shape == (256, 0) and b.h_scale_inv_t.shape == (128, 0)
