"""The epilogue's gradient over experts' rows: rows that no expert has are not
read, written or counted, and the bias gradient is one sum an expert.

Bounds as in tests/test_gpu_gemm_act.py: |act'| <= 1.13, |act| <= |z|, a
derivative's terms are each at most 1 + |z|; a column sum adds a CTA's 64 rows
in order, then the row blocks (at most 64 here) in eight slices and those in
order: under 128 roundings of 2^-24, which is 2^-17."""
import pytest
import torch

import scaled_fp8_linear_gb300 as F
from tests import block_ref as R

pytestmark = pytest.mark.gpu
DEV, F64, BF = "cuda", torch.float64, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _status():
    yield
    assert F.fp8_device_status() == 0


def _held(off, M):
    """Offsets as the call takes them: within 0..M, never falling."""
    out, top = [], 0
    for o in off:
        top = max(top, min(max(o, 0), M))
        out.append(top)
    return out


def _check(M, N, off, act, gated, seed=0):
    g = torch.Generator().manual_seed(seed)
    rows, E = (2 * N if gated else N), len(off) - 1
    at = _held(off, M)
    first, live = at[0], at[-1]
    d = torch.randn(M, N, generator=g).to(BF)
    z = (torch.randn(M, rows, generator=g) * 3).to(BF)
    for t in (d, z):                       # what nobody may read
        t[:first], t[live:] = float("nan"), float("nan")
    d64, z64 = d.to(F64)[first:live], z.to(F64)[first:live]
    gr, a = R.act_grad(z64[:, :N], act), R.act(z64[:, :N], act)
    want = torch.cat([d64 * z64[:, N:] * gr, d64 * a], 1) if gated else d64 * gr
    m = d64.abs() * (1 + z64[:, :N].abs())
    mag = torch.cat([m * z64[:, N:].abs(), m], 1) if gated else m
    tiny = torch.full_like(want, 2.0 ** -133)
    sums, sum_mag = torch.zeros(E, rows, dtype=F64), torch.zeros(E, rows, dtype=F64)
    for e in range(E):
        s = slice(at[e] - first, at[e + 1] - first)
        sums[e], sum_mag[e] = want[s].sum(0), mag[s].sum(0)
    o_dev = torch.tensor(off, dtype=torch.int32, device=DEV)
    call = lambda **kw: F.fp8_act_bwd(d.to(DEV), z.to(DEV), act, gated=gated, q_fmt=F.E5M2, offsets=o_dev,
                                      q_scale=torch.full((1,), 4.0, device=DEV), want_amax=True, **kw)
    dz = torch.full((M, rows), 7.0, dtype=BF, device=DEV)
    q = torch.full((M, rows), 9, dtype=torch.uint8, device=DEV)
    o = call(dz=dz, q=q, want_dbias=True)
    R.check(o.dz[first:live], want, mag, "dz", tiny)
    R.check_codes(o.q[first:live], F.E5M2, want * 4, mag * 4 * R.U_F32, "codes")
    for t, v in ((dz, 7.0), (q, 9)):
        assert (t[:first] == v).all() and (t[live:] == v).all()
    if live > first:
        R.check(o.amax, want.abs().max().view(1), mag.max().view(1), "amax")
    else:
        assert o.amax.item() == 0.0
    assert o.dbias.shape == (E, rows)
    R.check(o.dbias, sums, sum_mag, "dbias")
    again = call(want_dbias=True)
    assert torch.equal(again.dbias, o.dbias) and torch.equal(again.dz[first:live], o.dz[first:live])
    more = o.dbias.clone()
    F.fp8_act_bwd(d.to(DEV), z.to(DEV), act, gated=gated, dbias=more, accumulate=True, want_dz=False, offsets=o_dev)
    R.check(more, 2 * sums, 2 * sum_mag, "dbias added")
    only = call()
    assert torch.equal(only.dz[first:live], o.dz[first:live]) and torch.equal(only.amax, o.amax)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", [F.ACT_NONE, F.ACT_RELU, F.ACT_SILU, F.ACT_GELU, F.ACT_GELU_TANH])
def test_activations(act, gated):
    _check(300, 272, [0, 64, 64, 160, 224], act, gated, seed=act)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,off", [
    (1, 16, [0, 1]), (5, 48, [0, 0, 0]), (70, 16, [0, 3, 3, 67, 68]),          # any rows, empty experts
    (500, 528, [32, 96, 480]), (257, 32, [10, 10, 257]),                       # rows before the first
    (200, 64, [0, 120, 50, 180]), (200, 64, [-5, 40, 1000, 300]),              # falling, outside
    (4000, 1024, [0, 1, 2000, 3999]), (90, 32, [200, 300])])
def test_offsets(M, N, off, gated):
    _check(M, N, off, F.ACT_SILU, gated, seed=M)


def test_many_experts():
    g = torch.Generator().manual_seed(1)
    off = [0] + torch.cumsum(torch.randint(0, 9, (256,), generator=g), 0).tolist()
    _check(off[-1] + 40, 64, off, F.ACT_GELU, True, seed=2)


def test_after_a_product():
    """The forward's z in memory that held NaN, and its gradient."""
    E, N, K, M = 3, 64, 64, 200
    g = torch.Generator().manual_seed(5)
    code = lambda *s: (torch.randn(*s, generator=g) * 2).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    off = torch.tensor([0, 32, 32, 96], dtype=torch.int32, device=DEV)
    one = torch.ones(1, device=DEV)
    z = torch.full((M, 2 * N), float("nan"), dtype=BF, device=DEV)
    d = torch.full((M, N), float("nan"), dtype=BF, device=DEV)
    F.fp8_gemm_act(code(M, K), F.E4M3, code(E, 2 * N, K), F.E4M3, one / 64, one.repeat(E), act=F.ACT_SILU,
                   gated=True, z=z, d=d, offsets=off)
    o = F.fp8_act_bwd(d, z, F.ACT_SILU, gated=True, q_fmt=F.E5M2, q_scale=one, want_amax=True, want_dbias=True,
                      offsets=off)
    assert torch.isfinite(o.amax).all() and torch.isfinite(o.dbias).all() and not o.dbias[1].any()
    part = F.fp8_act_bwd(d[:96], z[:96], F.ACT_SILU, gated=True, q_fmt=F.E5M2, q_scale=one, want_amax=True)
    assert torch.equal(o.dz[:96], part.dz) and torch.equal(o.q[:96], part.q) and torch.equal(o.amax, part.amax)


def test_no_rows():
    x = torch.empty(0, 64, dtype=BF, device=DEV)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    o = F.fp8_act_bwd(x, x, F.ACT_SILU, want_dbias=True, offsets=off)
    assert o.dbias.shape == (3, 64) and not o.dbias.any()
    old = torch.ones(3, 64, device=DEV)
    F.fp8_act_bwd(x, x, F.ACT_SILU, dbias=old, accumulate=True, offsets=off)
    assert (old == 1).all()


def test_from_a_graph():
    """Offsets are read when the graph runs."""
    d = torch.randn(256, 64, device=DEV).to(BF)
    z = torch.randn(256, 64, device=DEV).to(BF)
    off = torch.tensor([0, 64, 128], dtype=torch.int32, device=DEV)
    db = torch.empty(2, 64, device=DEV)
    run = lambda: F.fp8_act_bwd(d, z, F.ACT_RELU, dbias=db, want_dz=False, offsets=off)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    off.copy_(torch.tensor([0, 100, 250]))
    graph.replay()
    got = db.clone()
    run()
    assert torch.equal(got, db)
    want = (d * (z > 0)).double()
    assert (got[0].double() - want[:100].sum(0)).abs().max() < 1e-4
