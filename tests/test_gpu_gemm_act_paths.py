"""Which kernels a product of fp8_gemm_act takes, and products whose last rows
leave in a launch of their own (test_remainder_beside_pairs' second shape runs
in pairs alone).  The kernels are those of the launches captured into a CUDA
graph, so a change of the choice cannot drop a path from these tests unseen."""
import re

import pytest
import torch

import scaled_fp8_linear_gb300 as F
from tests import block_ref as R
from tests.test_gpu_gemm_act import _case

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _status():
    yield
    assert F.fp8_device_status() == 0


def _kernels(call, tmp_path):
    """The product kernels of one call: ("pair", gated) or (columns, gated)."""
    call()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        call()
    dot = tmp_path / "graph.dot"
    graph.debug_dump(str(dot))
    names = set(re.findall(r"gemm_act_(pair|tile)_kernelI(?:Li(\d+)E)?Lb(\d)E", dot.read_text()))
    return {(kind if kind == "pair" else int(cols), gated == "1") for kind, cols, gated in names}


def _product(M, N, K, gated):
    a = torch.zeros(M, K, dtype=torch.uint8, device=DEV)
    b = torch.zeros(2 * N if gated else N, K, dtype=torch.uint8, device=DEV)
    one = torch.ones(1, device=DEV)
    return lambda: F.fp8_gemm_act(a, F.E4M3, b, F.E4M3, one, one, act=F.ACT_SILU, gated=gated)


# by the rule of launch_gemm_act the same at 148 to 152 SMs
PATHS = [(256, 512, False, {64}), (1000, 2064, False, {128}), (4096, 8192, False, {"pair"}),
         (600, 8192, False, {"pair", 256}), (1100, 4112, False, {"pair", 256}), (4099, 8192, False, {"pair", 256}),
         (600, 4096, True, {"pair", 256}), (513, 4112, True, {"pair", 256}), (1100, 2048, True, {"pair", 256})]


@pytest.mark.filterwarnings("ignore:DEBUG")
@pytest.mark.parametrize("M,N,gated,want", PATHS)
def test_path(M, N, gated, want, tmp_path):
    got = _kernels(_product(M, N, 128, gated), tmp_path)
    assert got == {(k, gated) for k in want}


@pytest.mark.parametrize("M,N,gated", [(600, 8192, False), (1100, 4112, False), (4099, 8192, False),
                                       (600, 4096, True), (513, 4112, True), (1100, 2048, True)])
@pytest.mark.parametrize("gran,q_fmt", [(F.GRAN_ROW, F.E4M3), (F.GRAN_TENSOR, None)])
def test_remainder(M, N, gated, gran, q_fmt):
    _case(M, N, 272, F.ACT_SILU, gated, True, True, gran, 0, q_fmt, seed=M)


@pytest.mark.parametrize("M,N,gated", [(600, 8192, False), (600, 4096, True)])
def test_remainder_onto_its_residual(M, N, gated):
    g = torch.Generator(device=DEV).manual_seed(3)
    code = lambda *s: torch.randint(0, 0x70, s, generator=g, device=DEV, dtype=torch.uint8)
    a, b = code(M, 256), code(2 * N if gated else N, 256)
    one, inv = torch.ones(1, device=DEV), torch.full((1,), 2.0 ** -10, device=DEV)
    res = torch.randn(M, N, generator=g, device=DEV).to(BF)
    call = lambda **k: F.fp8_gemm_act(a, F.E4M3, b, F.E4M3, one, inv, act=F.ACT_GELU, gated=gated, residual=res, **k)
    want = call().d
    call(d=res)
    assert torch.equal(res, want)


@pytest.mark.parametrize("off", [[-7, 40, 20, 1000, 300], [50, 50, 170, 171, 400], [0, 300, 100, 260, 260],
                                 [500, 600, 700, 800, 900], [10, 5, 3, 2, 1]])
@pytest.mark.parametrize("gated", [False, True])
def test_any_offsets(off, gated):
    """Offsets that fall, start past 0 or lie outside the rows are held to
    0..M and never fall; rows that no expert has keep what was there."""
    M, N, K, E = 400, 80, 64, 4
    g = torch.Generator().manual_seed(9)
    code = lambda *s: (torch.randn(*s, generator=g) * 2).to(torch.float8_e4m3fn)
    a, b = code(M, K), code(E, 2 * N if gated else N, K)
    top, at = 0, []
    for o in off:
        top = max(top, min(max(o, 0), M))
        at.append(top)
    one = torch.ones(1, device=DEV)
    z = torch.full((M, b.shape[1]), 5.0, dtype=BF, device=DEV)
    d = torch.full((M, N), 7.0, dtype=BF, device=DEV)
    q = torch.full((M, N), 9, dtype=torch.uint8, device=DEV)
    o = F.fp8_gemm_act(a.view(torch.uint8).to(DEV), F.E4M3, b.view(torch.uint8).to(DEV), F.E4M3, one, one.repeat(E),
                       act=F.ACT_RELU, gated=gated, z=z, d=d, q=q, q_fmt=F.E4M3, q_scale=one, want_amax=True,
                       offsets=torch.tensor(off, dtype=torch.int32, device=DEV))
    F64 = torch.float64
    zr, zm = torch.full(z.shape, 5.0, dtype=F64), torch.zeros(z.shape, dtype=F64)
    dr, dm = torch.full(d.shape, 7.0, dtype=F64), torch.zeros(d.shape, dtype=F64)
    top = 0.0
    for e in range(E):
        s = slice(at[e], at[e + 1])
        av, bv = a[s].to(torch.float32).to(F64), b[e].to(torch.float32).to(F64)
        zr[s], zm[s] = av @ bv.t(), av.abs() @ bv.abs().t()
        v, m = zr[s, :N].clamp_min(0), zm[s, :N]
        dr[s], dm[s] = (v * zr[s, N:], m * zm[s, N:]) if gated else (v, m)
        top = max([top] + dr[s].reshape(-1).abs().tolist())
    # the products' bound of the other GEMM tests; of a gated one's two factors, twice
    R.check(z, zr, zm, "z", 2e-3 * zm)
    R.check(d, dr, dm, "d", 2 * 2e-3 * dm * 1.01)
    inside = torch.zeros(M, dtype=torch.bool)
    inside[at[0]:at[-1]] = True
    assert (q.cpu()[~inside] == 9).all() and (d.cpu()[~inside] == 7.0).all() and (z.cpu()[~inside] == 5.0).all()
    assert abs(o.amax.item() - top) <= 1e-2 * dm.max().item() + 1e-30


@pytest.mark.parametrize("gated", [False, True])
def test_nan_and_infinity_stay_in_their_rows(gated):
    """A NaN code, a NaN residual and an infinite factor: their rows are not
    finite, the others are, amax is NaN; an infinity saturates its code."""
    M, N, K = 300, 272, 64
    g = torch.Generator().manual_seed(2)
    a = (torch.randn(M, K, generator=g) * 2).to(torch.float8_e4m3fn).view(torch.uint8)
    b = (torch.randn(2 * N if gated else N, K, generator=g) * 2).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    clean = a.clone()
    a[3, 5] = 0x7F                                  # E4M3's NaN
    sa, res = torch.full((M,), 2.0 ** -6), torch.randn(M, N, generator=g).to(BF)
    bad_sa, bad_res = sa.clone(), res.clone()
    bad_sa[130], bad_res[280, 17], bad_res[290, 18] = float("inf"), float("nan"), float("inf")
    one = torch.ones(1, device=DEV)
    run = lambda a, sa, res: F.fp8_gemm_act(
        a.to(DEV), F.E4M3, b, F.E4M3, sa.to(DEV), one.repeat(b.shape[0]), ga=F.GRAN_ROW, gb=F.GRAN_ROW, act=F.ACT_RELU,
        gated=gated, residual=res.to(DEV), q_fmt=F.E4M3, q_scale=one, want_amax=True, want_z=True)
    o, want = run(a, bad_sa, bad_res), run(clean, sa, res)
    rows = torch.ones(M, dtype=torch.bool, device=DEV)
    rows[[3, 130, 280, 290]] = False
    assert torch.equal(o.d[rows], want.d[rows]) and torch.equal(o.z[rows], want.z[rows])
    assert torch.equal(o.q[rows], want.q[rows])
    assert torch.isnan(o.z[3]).all() and torch.isnan(o.d[3]).all() and (o.q[3] & 0x7F == 0x7F).all()
    assert not torch.isfinite(o.z[130]).any()
    assert torch.isnan(o.d[280, 17]) and o.q[280, 17].item() & 0x7F == 0x7F
    assert o.d[290, 18].item() == float("inf") and o.q[290, 18].item() == 0x7E      # 448
    keep = torch.ones(N, dtype=torch.bool, device=DEV)
    keep[17] = False
    assert torch.equal(o.d[280, keep], want.d[280, keep])
    assert torch.isnan(o.amax).all()
    only_inf = run(clean, sa, torch.where(torch.isnan(bad_res), res, bad_res))
    assert only_inf.amax.item() == float("inf")


def test_nan_and_infinity_in_the_gradient():
    M, N = 130, 272
    g = torch.Generator().manual_seed(4)
    d, z = torch.randn(M, N, generator=g).to(BF), torch.randn(M, N, generator=g).to(BF)
    bad = d.clone()
    bad[70, 9], bad[129, 271] = float("nan"), float("inf")
    z[129, 271] = 2.0
    one = torch.ones(1, device=DEV)
    run = lambda d: F.fp8_act_bwd(d.to(DEV), z.to(DEV), F.ACT_SILU, q_fmt=F.E5M2, q_scale=one, want_amax=True,
                                  want_dbias=True)
    o, want = run(bad), run(d)
    same = torch.ones(M, N, dtype=torch.bool, device=DEV)
    same[70, 9] = same[129, 271] = False
    assert torch.equal(o.dz[same], want.dz[same]) and torch.equal(o.q[same], want.q[same])
    assert torch.isnan(o.dz[70, 9]) and o.q[70, 9].item() & 0x7F > 0x7C
    assert o.dz[129, 271].item() == float("inf") and o.q[129, 271].item() == 0x7B    # 57344
    cols = torch.ones(N, dtype=torch.bool, device=DEV)
    cols[[9, 271]] = False
    assert torch.equal(o.dbias[cols], want.dbias[cols])
    assert torch.isnan(o.dbias[9]) and o.dbias[271].item() == float("inf") and torch.isnan(o.amax).all()
