"""Products of experts and their weight gradients in blocks of 128, against 64
bits.  Exact inputs (tests/expert_ref.py) bit for bit; codes over the whole
range within the framework's bound for its FP8 GEMMs, 2e-3 of the sum of the
terms' magnitudes, with half a step of bf16, 2^-8, for its rounding."""
import pytest
import torch

import scaled_fp8_linear_gb300 as F
from tests import expert_ref as E
from tests.helpers import BOUND

pytestmark = pytest.mark.gpu
DEV, F64 = "cuda", torch.float64


@pytest.fixture(scope="module", autouse=True)
def _status():
    yield
    assert F.fp8_device_status() == 0


def _i32(off):
    return torch.tensor(off, dtype=torch.int32, device=DEV)


def _near(got, want, mag, what):
    g, tol = got.to(F64).cpu(), BOUND * mag
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert ((g - want).abs() <= tol).all(), f"{what}: largest {((g - want).abs() - tol).max()}"


# ------------------------------------------------------------------ products

def _product(M, N, K, off, fa=0, fb=0, out=F.OUT_BF16, pow2=False, exact=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = len(off) - 1
    codes = E.exact_codes if exact else E.any_codes
    a, b = codes(g, fa, M, K), codes(g, fb, n, N, K)
    if exact or pow2:
        sa, sb = E.exact_factors(g, M, K // 128), E.exact_factors(g, n, N // 128, K // 128)
    else:
        sa, sb = torch.rand(M, K // 128, generator=g) + 0.1, torch.rand(n, N // 128, K // 128, generator=g) + 0.1
    want, mag, live = E.products(E.by_rows(a, sa, fa), E.by_tiles(b, sb, fb), off)
    d = torch.full((M, N), 7.0, dtype=torch.float32 if out == F.OUT_F32 else torch.bfloat16, device=DEV)
    a_dev, sa_dev = a.to(DEV), sa.to(DEV)
    if not live.all():                       # what nobody may read into a result
        a_dev[~live], sa_dev[~live] = 0x7F, float("nan")
    got = F.fp8_gemm_experts(a_dev, fa, b.to(DEV), fb, sa_dev, sb.to(DEV), _i32(off), out=out, pow2=pow2, d=d)
    assert got is d
    d = d.cpu()
    assert (d[~live] == 7.0).all()
    if exact:
        assert torch.equal(d[live], want[live].to(d.dtype))
    else:
        _near(d[live], want[live], mag[live], "product")


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("out", [F.OUT_BF16, F.OUT_F32])
@pytest.mark.parametrize("M,N,K,off", [
    (1, 128, 128, [0, 1]),
    (1, 128, 256, [0, 0, 1, 1]),
    (5, 256, 384, [0, 2, 2, 5]),
    (17, 384, 128, [0, 16, 17]),
    (33, 128, 1152, [0, 1, 33]),
    (64, 640, 640, [0, 15, 31, 48, 64]),
    (100, 256, 512, [3, 40, 40, 97]),            # rows of no expert before and after
    (130, 128, 256, [0, 129, 130]),
    (255, 384, 384, [0, 255]),
    (300, 512, 256, [0, 100, 90, 400]),          # falling, and past the rows
    (600, 256, 2048, [0, 257, 258, 600]),
    (1000, 384, 640, [0, 1000, 1000, 1000]),
    (1100, 128, 384, [-5, 256, 300, 813, 1024]),
    (40, 256, 256, [0, 0, 0, 0]),                # no rows at all
])
def test_products_exact(M, N, K, off, out, pow2):
    _product(M, N, K, off, out=out, pow2=pow2)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("fa,fb", [(0, 0), (1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("M,off", [(29, [0, 7, 20, 29]), (700, [0, 130, 600, 700])])
def test_products_of_any_codes(M, off, fa, fb, pow2):
    _product(M, 384, 896, off, fa, fb, out=F.OUT_F32, pow2=pow2, exact=False, seed=1)


# more rows an expert and more tiles than the kernels of few rows take
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("out", [F.OUT_BF16, F.OUT_F32])
@pytest.mark.parametrize("K,off", [
    (128, [0, 3000]),
    (384, [5, 700, 700, 1411, 2990]),            # rows of no expert before and after
    (640, [0, 1500, 1400, 4000]),                # falling, and past the rows
    (256, [-5, 256, 512, 813, 941, 1069, 1070, 2222]),
    (2176, [0, 1, 130, 3000]),
    (256, [0, 0, 0, 0]),                         # no rows at all
    (512, [2999, 2999, 3000]),
])
def test_products_of_many_tiles(K, off, out, pow2):
    _product(3000, 1152, K, off, out=out, pow2=pow2)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("fa,fb", [(0, 0), (1, 0), (0, 1), (1, 1)])
def test_products_of_many_tiles_of_any_codes(fa, fb, pow2):
    _product(2700, 1280, 896, [0, 601, 1300, 2600], fa, fb, out=F.OUT_F32, pow2=pow2, exact=False, seed=1)


@pytest.mark.parametrize("pow2", [False, True])
def test_nan_stays_in_its_row_among_many_tiles(pow2):
    g = torch.Generator().manual_seed(3)
    M, N = 3000, 1152
    a, b = E.exact_codes(g, 0, M, 256), E.exact_codes(g, 0, 2, N, 256)
    sa, sb = E.exact_factors(g, M, 2), E.exact_factors(g, 2, N // 128, 2)
    a[11, 5] = a[1400, 200] = 0x7F
    got = F.fp8_gemm_experts(a.to(DEV), 0, b.to(DEV), 0, sa.to(DEV), sb.to(DEV), _i32([0, 1300, M]), pow2=pow2).cpu()
    nan = torch.zeros(M, dtype=torch.bool)
    nan[[11, 1400]] = True
    assert torch.isnan(got[nan]).all() and not torch.isnan(got[~nan]).any()


@pytest.mark.parametrize("M,rows", [(200, 3), (4096, 100), (6000, 2000)])
def test_many_experts(M, rows):
    g = torch.Generator().manual_seed(rows)
    for n in (1, 31, 33, 256):
        cuts = torch.randint(0, M + 1, (n - 1,), generator=g).sort().values.tolist()
        _product(M, 128, 128, [0] + cuts + [M], out=F.OUT_F32, seed=n)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 256, 257])
def test_rows_around_the_tiles(rows):
    """One busy expert among idle ones, and all of them alike."""
    _product(rows, 256, 256, [0, 0, rows, rows, rows], out=F.OUT_F32, seed=rows)
    _product(4 * rows, 256, 256, [0, rows, 2 * rows, 3 * rows, 4 * rows], seed=rows)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows", [8, 9, 72, 73, 224, 225])
def test_rows_around_the_choice_of_the_kernel(rows, pow2):
    off = [0, rows // 2, rows // 2, 2 * rows + 3, 4 * rows]
    _product(4 * rows, 384, 640, off, fa=1, pow2=pow2, seed=rows)


@pytest.mark.parametrize("out", [F.OUT_BF16, F.OUT_F32])
@pytest.mark.parametrize("K", [128, 512, 640, 1152, 2048, 4224, 7168])
@pytest.mark.parametrize("M,N,off", [
    (1, 128, [0, 1]), (3, 384, [0, 1, 1, 3]), (16, 1024, [0, 16]), (17, 256, [0, 0, 17]), (9, 128, [2, 2, 7]),
    (40, 128, [0, 40]), (129, 512, [0, 129]), (200, 256, [3, 100, 199]), (30, 256, [0, 0, 0])])
def test_few_tiles_with_a_long_reduction(M, N, K, off, out):
    """K cut into ranges, and groups of four K blocks that do not divide evenly."""
    _product(M, N, K, off, fa=1, out=out, seed=K + M)
    if K == 7168:
        _product(M, N, K, off, out=out, exact=False, seed=M)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,N,off", [(300, 256, [0, 300]), (1000, 384, [0, 450, 450, 1000]),
                                     (4800, 512, [0, 4799]), (5000, 512, [0, 4999])])   # 148 and 160 tiles of 128 rows
def test_many_rows_in_few_tiles(M, N, off, pow2):
    _product(M, N, 1152, off, fb=1, pow2=pow2, seed=M)


def test_equal_calls_give_equal_bits_when_k_is_cut():
    g = torch.Generator().manual_seed(9)
    for M in (5, 70):
        a, b = E.any_codes(g, 0, M, 7168).to(DEV), E.any_codes(g, 0, 2, 256, 7168).to(DEV)
        sa, sb = (torch.rand(M, 56, generator=g) + 0.1).to(DEV), (torch.rand(2, 2, 56, generator=g) + 0.1).to(DEV)
        off = _i32([0, M // 2, M])
        first = F.fp8_gemm_experts(a, 0, b, 0, sa, sb, off, out=F.OUT_F32)
        for _ in range(20):
            assert torch.equal(F.fp8_gemm_experts(a, 0, b, 0, sa, sb, off, out=F.OUT_F32), first)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("n", [7, 31, 256])
def test_many_experts_of_many_rows(n, pow2):
    g = torch.Generator().manual_seed(n)
    M = 290 * n if n < 256 else 60000
    cuts = torch.randint(0, M + 1, (n - 1,), generator=g).sort().values.tolist()
    _product(M, 256, 128, [0] + cuts + [M - 1], out=F.OUT_F32, pow2=pow2, seed=n)


def test_nan_stays_in_its_row():
    g = torch.Generator().manual_seed(3)
    for M in (40, 600):
        a, b = E.exact_codes(g, 0, M, 256), E.exact_codes(g, 0, 2, 256, 256)
        sa, sb = E.exact_factors(g, M, 2), E.exact_factors(g, 2, 2, 2)
        a[11, 5] = 0x7F
        got = F.fp8_gemm_experts(a.to(DEV), 0, b.to(DEV), 0, sa.to(DEV), sb.to(DEV), _i32([0, 20, M])).cpu()
        assert torch.isnan(got[11]).all() and not torch.isnan(got[torch.arange(M) != 11]).any()


def test_no_tokens():
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device=DEV)
    d = F.fp8_gemm_experts(z(0, 128), 0, z(2, 128, 128), 0, z(0, 1, dt=torch.float32), z(2, 1, 1, dt=torch.float32),
                           _i32([0, 0, 0]))
    assert d.shape == (0, 128)
    dw = F.fp8_wgrad_experts(z(128, 0), 1, z(256, 0), 0, z(128, 0, dt=torch.float32), z(256, 0, dt=torch.float32),
                             _i32([0, 0, 0]))
    assert dw.shape == (2, 128, 256) and (dw == 0).all()


# ------------------------------------------------------------------ weight gradients

def _wgrad(M, N, K, off, pow2=False, accumulate=False, exact=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    n, tb = len(off) - 1, M // 128
    codes = E.exact_codes if exact else E.any_codes
    dy, x = codes(g, 1, N, M), codes(g, 0, K, M)
    if exact or pow2:
        sy, sx = E.exact_factors(g, N, tb), E.exact_factors(g, K, tb)
    else:
        sy, sx = torch.rand(N, tb, generator=g) + 0.1, torch.rand(K, tb, generator=g) + 0.1
    a, b = E.by_rows(dy, sy, 1), E.by_rows(x, sx, 0)
    at = E.held(off, M)
    want = torch.stack([a[:, s:t] @ b[:, s:t].t() for s, t in zip(at, at[1:])])
    mag = torch.stack([a[:, s:t].abs() @ b[:, s:t].abs().t() for s, t in zip(at, at[1:])])
    dev = [t.to(DEV) for t in (dy, x, sy, sx)]
    for t in dev[:2]:                        # tokens of no expert
        t[:, :at[0]], t[:, at[-1]:] = 0x7F, 0x7F
    dw = None
    if accumulate:
        old = torch.randint(-100, 100, (n, N, K), generator=g).float()
        want, mag, dw = want + old, mag + old.abs(), old.to(DEV)
    got = F.fp8_wgrad_experts(dev[0], 1, dev[1], 0, dev[2], dev[3], _i32(off), pow2=pow2, dW=dw, accumulate=accumulate)
    assert dw is None or got is dw
    if exact:
        assert torch.equal(got.cpu(), want.float())
    else:
        _near(got.cpu(), want, mag, "weight gradient")


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("M,N,K,off", [
    (128, 128, 128, [0, 128]),
    (128, 256, 128, [0, 0, 128, 128]),
    (256, 128, 384, [128, 256]),
    (512, 384, 256, [0, 128, 128, 384, 512]),
    (640, 256, 256, [128, 256, 640, 640]),
    (1024, 512, 128, [0, 640, 512, 2000]),      # falling, and past the tokens
    (1280, 128, 640, [0, 0, 1152]),
    (2688, 384, 384, [0, 128, 2304, 2432]),     # 17 blocks from the second on
    (384, 128, 128, [0, 0, 0]),                 # no tokens of any expert
])
def test_wgrad_exact(M, N, K, off, pow2, accumulate):
    _wgrad(M, N, K, off, pow2, accumulate)


@pytest.mark.parametrize("pow2", [False, True])
def test_wgrad_of_any_codes(pow2):
    _wgrad(896, 384, 256, [0, 256, 256, 896], pow2, exact=False, seed=2)


@pytest.mark.parametrize("n", [31, 33, 256])
def test_wgrad_many_experts(n):
    g = torch.Generator().manual_seed(n)
    M = 40 * 128
    cuts = (torch.randint(0, 41, (n - 1,), generator=g).sort().values * 128).tolist()
    for pow2 in (False, True):
        _wgrad(M, 128, 128, [0] + cuts + [M], pow2, seed=n)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("accumulate", [False, True])
def test_wgrad_refuses_offsets_within_a_block(pow2, accumulate):
    """Those experts' gradients are NaN and the status word says so; the others
    are right."""
    g = torch.Generator().manual_seed(5)
    M, N, K, off = 512, 256, 128, [0, 128, 200, 384, 512]
    dy, x = E.exact_codes(g, 1, N, M), E.exact_codes(g, 0, K, M)
    sy, sx = E.exact_factors(g, N, 4), E.exact_factors(g, K, 4)
    a, b = E.by_rows(dy, sy, 1), E.by_rows(x, sx, 0)
    assert F.fp8_device_status() == 0
    dw = torch.zeros(4, N, K, device=DEV) if accumulate else None
    got = F.fp8_wgrad_experts(dy.to(DEV), 1, x.to(DEV), 0, sy.to(DEV), sx.to(DEV), _i32(off), pow2=pow2, dW=dw,
                              accumulate=accumulate).cpu()
    assert torch.isnan(got[1]).all() and torch.isnan(got[2]).all()
    for e in (0, 3):
        s = slice(off[e], off[e + 1])
        assert torch.equal(got[e], (a[:, s] @ b[:, s].t()).float())
    with pytest.raises(ValueError, match="multiples of 128"):
        F.check_device_status()
    F.check_device_status()


def test_equal_calls_give_equal_bits():
    g = torch.Generator().manual_seed(9)
    M, N, K = 1500, 512, 1024
    a, b = E.any_codes(g, 0, M, K).to(DEV), E.any_codes(g, 0, 5, N, K).to(DEV)
    sa, sb = torch.rand(M, 8, generator=g).to(DEV), torch.rand(5, 4, 8, generator=g).to(DEV)
    for off in ([0, 20, 20, 30, 44, 60], [0, 400, 400, 777, 1100, 1500]):
        m = off[-1]
        call = lambda: F.fp8_gemm_experts(a[:m], 0, b, 0, sa[:m], sb, _i32(off), out=F.OUT_F32)
        want = call()
        assert all(torch.equal(call(), want) for _ in range(5))
