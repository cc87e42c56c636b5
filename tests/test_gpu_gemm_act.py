"""The GEMM with bias, activation and residual, and its gradient.

z is held to the GEMM bound 2e-3 sum|a b| s_a s_b of the other GEMM tests;
an activation moves an error by at most 1.13 (GELU's largest slope), the up
factor multiplies it.  Integer operands give exact sums."""
import pytest
import torch

import scaled_fp8_linear_gb300 as F
from tests import block_ref as R

pytestmark = pytest.mark.gpu
DEV, F64, BF = "cuda", torch.float64, torch.bfloat16
BOUND, SLOPE = 2e-3, 1.13


@pytest.fixture(scope="module", autouse=True)
def _status():
    yield
    assert F.fp8_device_status() == 0


def _codes(g, *shape):
    return (torch.randn(*shape, generator=g) * 2).to(torch.float8_e4m3fn)


def _val(q):
    return q.to(torch.float32).to(F64)


def _case(M, N, K, act, gated, bias, res, gran, experts, q_fmt, seed=0, z=True, align=32):
    g = torch.Generator().manual_seed(seed)
    rows = 2 * N if gated else N
    E = experts or 1
    off = None
    if experts:
        off, at = [0], 0
        for e in range(E):               # ragged shares, expert 1 empty
            at = min(M, at + (0 if e == 1 else align * int(torch.randint(0, 2 * M // (align * E) + 2, (1,), generator=g))))
            off.append(at)
        off[-1] = max(off[-1], min(M, 32)) if E > 2 else off[-1]
    a, b = _codes(g, M, K), _codes(g, E, rows, K)
    sa = (torch.rand(M if gran == F.GRAN_ROW else 1, generator=g) + 0.5) * 0.25
    sb = (torch.rand(E, rows, generator=g) + 0.5 if gran == F.GRAN_ROW else torch.rand(E, generator=g) + 0.5) / K ** 0.5
    bi = torch.randn(E, rows, generator=g).to(BF) if bias else None
    rs = torch.randn(M, N, generator=g).to(BF) if res else None
    qs = torch.tensor([20.0])
    d = lambda t: None if t is None else t.to(DEV)
    u8 = lambda t: t.view(torch.uint8).to(DEV)
    flat = lambda t: t if experts else t[0]
    o = F.fp8_gemm_act(u8(a), F.E4M3, flat(u8(b)), F.E4M3, d(sa),
                       d(sb if experts or gran != F.GRAN_ROW else sb[0]), ga=gran, gb=gran, act=act,
                       gated=gated, bias=None if bi is None else d(flat(bi)), residual=d(rs), want_z=z,
                       q_fmt=q_fmt, q_scale=d(qs) if q_fmt is not None else None,
                       want_amax=q_fmt is not None,
                       offsets=None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV))
    off = off or [0, M]
    live = off[-1]
    zr, zm = torch.zeros(live, rows, dtype=F64), torch.zeros(live, rows, dtype=F64)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        av, bv = _val(a[s]), _val(b[e])
        f = (sa.to(F64)[s, None] if gran == F.GRAN_ROW else sa.to(F64)) * sb[e].to(F64)
        zr[s], zm[s] = av @ bv.t() * f, av.abs() @ bv.abs().t() * f
        if bi is not None:
            zr[s] += bi[e].to(F64)
    err = BOUND * zm + R.U_F32 * zr.abs()
    if z:
        R.check(o.z[:live], zr, zr.abs(), "z", err)
    v, ve = R.act(zr[:, :N], act), SLOPE * err[:, :N]
    if gated:
        ve = ve * zr[:, N:].abs() + (v.abs() + ve) * err[:, N:]
        v = v * zr[:, N:]
    mag = v.abs() + zr[:, :N].abs()
    if rs is not None:
        v, mag = v + rs.to(F64)[:live], mag + rs.to(F64)[:live].abs()
    R.check(o.d[:live], v, mag, "d", ve * (1 + R.U_BF16))
    if q_fmt is not None:
        R.check_codes(o.q[:live], q_fmt, v * 20.0, 20.0 * (ve + R.U_F32 * mag), "codes")
        if live:
            top = v.abs().max()
            assert abs(o.amax.item() - top) <= (ve + R.U_F32 * mag).max()
    return o


SHAPES = [(1, 16, 16), (3, 48, 32), (128, 128, 128), (200, 144, 256), (257, 512, 384), (300, 272, 1040),
          (512, 1024, 512), (1000, 2064, 272), (2048, 4096, 256)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(M, N, K, gated):
    _case(M, N, K, F.ACT_SILU, gated, True, True, F.GRAN_TENSOR, 0, None)


@pytest.mark.parametrize("act", [F.ACT_NONE, F.ACT_RELU, F.ACT_SILU, F.ACT_GELU, F.ACT_GELU_TANH])
@pytest.mark.parametrize("gated,bias,res,gran,q_fmt", [
    (False, False, False, F.GRAN_TENSOR, F.E4M3), (False, True, True, F.GRAN_ROW, None),
    (True, False, False, F.GRAN_ROW, F.E5M2), (True, True, True, F.GRAN_TENSOR, F.E4M3)])
@pytest.mark.parametrize("M", [130, 700])
def test_epilogues(M, act, gated, bias, res, gran, q_fmt):
    _case(M, 400, 256, act, gated, bias, res, gran, 0, q_fmt, seed=act)


@pytest.mark.parametrize("M,N,K,E,gated,gran", [
    (64, 64, 128, 3, False, F.GRAN_TENSOR), (1024, 272, 256, 5, True, F.GRAN_ROW),
    (2048, 512, 512, 40, True, F.GRAN_TENSOR), (4096, 1040, 128, 9, False, F.GRAN_ROW),
    (320, 48, 64, 256, True, F.GRAN_TENSOR)])
def test_experts(M, N, K, E, gated, gran):
    _case(M, N, K, F.ACT_SILU, gated, True, True, gran, E, F.E4M3, seed=E)


@pytest.mark.parametrize("align", [1, 16])
@pytest.mark.parametrize("M,N,K,E,gated", [(300, 48, 64, 20, True), (1500, 272, 256, 6, False),
                                           (2000, 528, 128, 17, True), (333, 16, 32, 256, False)])
def test_experts_any_offsets(M, N, K, E, gated, align):
    """Experts that end within a stored box of 32 rows."""
    _case(M, N, K, F.ACT_GELU_TANH, gated, True, True, F.GRAN_ROW, E, F.E4M3, seed=M, align=align)


def test_remainder_beside_pairs():
    """A product whose last rows leave in a launch of their own: the same as
    the row-wise product (700 = 2 x 256 + 188 has none, 600 and 4099 do)."""
    for M, N, K in ((600, 8192, 512), (4099, 4096, 256)):
        _case(M, N, K, F.ACT_SILU, False, True, True, F.GRAN_ROW, 0, F.E4M3, seed=M)


def test_remainder_is_ordered():
    """Between a cast that writes its operand and a norm that reads its result,
    back to back and from a graph: the same bits as with a wait between them."""
    g = torch.Generator(device=DEV).manual_seed(7)
    M, N, K = 600, 8192, 512
    xs = [torch.randn(M, K, generator=g, device=DEV).to(BF) for _ in range(8)]
    w = torch.randint(0, 0x70, (N, K), generator=g, device=DEV, dtype=torch.uint8)
    one, inv = torch.ones(1, device=DEV), torch.full((1,), 2.0 ** -8, device=DEV)
    q = torch.empty(M, K, dtype=torch.uint8, device=DEV)

    def chain(x, wait=lambda: None):
        F.fp8_quantize(x, F.E4M3, scale=one, q=q)
        wait()
        d = F.fp8_gemm_act(q, F.E4M3, w, F.E4M3, one, inv, act=F.ACT_SILU).d
        wait()
        return d, F.fp8_norm_fwd(d, want_x_out=False).y

    want = [chain(x, torch.cuda.synchronize) for x in xs]
    for _ in range(4):
        got = [chain(x) for x in xs]
        assert all(torch.equal(a, b) for p, r in zip(got, want) for a, b in zip(p, r))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [chain(x) for x in xs]
    for _ in range(4):
        for p in got:
            p[0].zero_()
        graph.replay()
        assert all(torch.equal(a, b) for p, r in zip(got, want) for a, b in zip(p, r))


def test_residual_in_place():
    g = torch.Generator().manual_seed(3)
    a, b = _codes(g, 700, 256).view(torch.uint8).to(DEV), _codes(g, 512, 256).view(torch.uint8).to(DEV)
    one, res = torch.ones(1, device=DEV), torch.randn(700, 512, generator=g).to(BF).to(DEV)
    want = F.fp8_gemm_act(a, F.E4M3, b, F.E4M3, one, one, act=F.ACT_GELU, residual=res).d
    F.fp8_gemm_act(a, F.E4M3, b, F.E4M3, one, one, act=F.ACT_GELU, residual=res, d=res)
    assert torch.equal(res, want)


@pytest.mark.parametrize("fa,fb", [(F.E5M2, F.E4M3), (F.E4M3, F.E5M2), (F.E5M2, F.E5M2)])
def test_formats(fa, fb):
    """Small integers are exact in either format."""
    g = torch.Generator().manual_seed(4)
    a, b = (torch.randint(-3, 4, s, generator=g).float() for s in ((300, 128), (272, 128)))
    q = lambda t, f: t.to(torch.float8_e5m2 if f == F.E5M2 else torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    one = torch.ones(1, device=DEV)
    o = F.fp8_gemm_act(q(a, fa), fa, q(b, fb), fb, one, one)
    assert torch.equal(o.d.cpu(), (a @ b.t()).to(BF))


def test_experts_leave_other_rows():
    """Rows past the last offset keep what was there; without any row nothing
    is written."""
    g = torch.Generator().manual_seed(1)
    a, b = _codes(g, 256, 64).view(torch.uint8).to(DEV), _codes(g, 3, 32, 64).view(torch.uint8).to(DEV)
    one = torch.ones(1, device=DEV)
    for off in ([0, 32, 32, 96], [0, 0, 0, 0]):
        d = torch.full((256, 32), 7.0, dtype=BF, device=DEV)
        F.fp8_gemm_act(a, F.E4M3, b, F.E4M3, one, one.repeat(3), d=d,
                       offsets=torch.tensor(off, dtype=torch.int32, device=DEV))
        assert (d[off[-1]:] == 7.0).all()
        assert off[-1] == 0 or not (d[:off[-1]] == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(96, 64, 128), (520, 528, 272), (1024, 4096, 512)])
def test_exact_integers(M, N, K):
    """Operands of -3..3, bias and residual integers: every sum is exact, so D
    is the rounded exact value."""
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randint(-3, 4, s, generator=g).float()
    a, b, bias, res = r(M, K), r(N, K), r(N), r(M, N)
    q = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    one = torch.ones(1, device=DEV)
    o = F.fp8_gemm_act(q(a), F.E4M3, q(b), F.E4M3, one, one, bias=bias.to(BF).to(DEV),
                       residual=res.to(BF).to(DEV), act=F.ACT_RELU)
    want = (a.to(F64) @ b.to(F64).t() + bias).clamp_min(0) + res
    assert torch.equal(o.d.cpu(), want.to(BF))


def test_equal_calls_give_equal_bits():
    a = _case(700, 512, 512, F.ACT_GELU, True, True, True, F.GRAN_ROW, 0, F.E4M3, seed=5)
    b = _case(700, 512, 512, F.ACT_GELU, True, True, True, F.GRAN_ROW, 0, F.E4M3, seed=5)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_no_rows():
    one = torch.ones(1, device=DEV)
    w = torch.zeros(64, 64, dtype=torch.uint8, device=DEV)
    o = F.fp8_gemm_act(w[:0], F.E4M3, w, F.E4M3, one, one, want_z=True, q_fmt=F.E4M3, q_scale=one,
                       want_amax=True)
    assert o.d.shape == (0, 64) and o.amax.item() == 0.0
    x = torch.empty(0, 64, dtype=BF, device=DEV)
    o = F.fp8_act_bwd(x, x, F.ACT_SILU, want_dbias=True)
    assert not o.dbias.any()


@pytest.mark.parametrize("act", [F.ACT_NONE, F.ACT_RELU, F.ACT_SILU, F.ACT_GELU, F.ACT_GELU_TANH])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N", [(1, 16), (65, 272), (200, 1024)])
def test_gradient(M, N, act, gated):
    g = torch.Generator().manual_seed(act)
    rows = 2 * N if gated else N
    d = torch.randn(M, N, generator=g).to(BF)
    z = (torch.randn(M, rows, generator=g) * 3).to(BF)
    z[0, :4] = torch.tensor([0.0, -0.0, 30.0, -30.0])     # the kink and both tails
    d64, z64 = d.to(F64), z.to(F64)
    gr, a = R.act_grad(z64[:, :N], act), R.act(z64[:, :N], act)
    want = torch.cat([d64 * z64[:, N:] * gr, d64 * a], 1) if gated else d64 * gr
    # |act'| <= 1.13, |act| <= |z|; the derivative's terms are each at most 1 + |z|
    m = d64.abs() * (1 + z64[:, :N].abs())
    mag = torch.cat([m * z64[:, N:].abs(), m], 1) if gated else m
    # an output below bf16's smallest normal number is off by its step there
    tiny = torch.full_like(want, 2.0 ** -133)
    for fmt in (F.E4M3, F.E5M2):
        o = F.fp8_act_bwd(d.to(DEV), z.to(DEV), act, gated=gated, q_fmt=fmt,
                          q_scale=torch.full((1,), 4.0, device=DEV), want_amax=True, want_dbias=True)
        R.check(o.dz, want, mag, "dz", tiny)
        R.check_codes(o.q, fmt, want * 4, mag * 4 * R.U_F32, "codes")
        R.check(o.dbias, want.sum(0), mag.sum(0), "dbias")
        R.check(o.amax, want.abs().max().view(1), mag.max().view(1), "amax")
    more = o.dbias.clone()
    F.fp8_act_bwd(d.to(DEV), z.to(DEV), act, gated=gated, dbias=more, accumulate=True, want_dz=False)
    R.check(more, 2 * want.sum(0), 2 * mag.sum(0), "dbias added")


def test_offsets_past_32_bits():
    """More than 2^31 elements of D and z: the last rows equal the same rows alone."""
    M, N, K = (1 << 18) + 40, 8192, 32
    g = torch.Generator(device=DEV).manual_seed(1)
    code = lambda *s: torch.randint(0, 0x70, s, generator=g, device=DEV, dtype=torch.uint8)
    a, b = code(M, K), code(N, K)
    sa, sb = torch.rand(M, device=DEV) * 2 ** -9, torch.rand(N, device=DEV)
    res = torch.empty(M, N, dtype=BF, device=DEV)
    res.normal_(generator=g)
    run = lambda a, sa, res: F.fp8_gemm_act(a, F.E4M3, b, F.E4M3, sa, sb, ga=F.GRAN_ROW, gb=F.GRAN_ROW,
                                            act=F.ACT_SILU, residual=res, want_z=True)
    o, t = run(a, sa, res), run(a[-40:].contiguous(), sa[-40:].contiguous(), res[-40:].contiguous())
    assert torch.equal(o.d[-40:], t.d) and torch.equal(o.z[-40:], t.z)
    q = F.fp8_act_bwd(res, o.z, F.ACT_SILU).dz[-40:]
    assert torch.equal(q, F.fp8_act_bwd(res[-40:].contiguous(), t.z, F.ACT_SILU).dz)
