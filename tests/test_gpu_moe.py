"""Tokens sorted by expert and back: the plan equals a walk over the slots,
copies are exact, sums are held to tests/block_ref.py's bounds."""
import pytest
import torch

import scaled_fp8_linear_gb300 as F
from tests import block_ref as R

pytestmark = pytest.mark.gpu
DEV, F64, BF = "cuda", torch.float64, torch.bfloat16

ROUTES = [(1, 1, 1, 1), (1, 2, 8, 16), (3, 2, 5, 32), (64, 8, 256, 32), (257, 4, 7, 128),
          (1000, 2, 33, 1), (1024, 2, 64, 16), (2049, 1, 3, 32), (5000, 8, 1024, 4), (20000, 8, 60, 32),
          (300, 64, 100, 2)]


def _ids(T, k, E, seed, drop=0.1, skew=False):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if skew:
        ids = torch.where(torch.rand(T, k, generator=g) < 0.8, torch.full_like(ids, E // 2), ids)
    out = torch.rand(T, k, generator=g)
    ids[out < drop / 2] = -1
    ids[out > 1 - drop / 2] = E          # past the last expert: dropped as well
    return ids


@pytest.mark.parametrize("skew", [False, True])
@pytest.mark.parametrize("T,k,E,align", ROUTES)
def test_plan(T, k, E, align, skew):
    ids = _ids(T, k, E, 7, skew=skew)
    p = F.fp8_moe_plan(ids.to(DEV), E, align=align)
    for got, want, name in zip(p, R.plan(ids, E, align, p.src.numel()), p._fields):
        assert torch.equal(got.cpu(), want), name


@pytest.mark.parametrize("fill", [-1, 0, 3])
def test_plan_one_expert_or_none(fill):
    ids = torch.full((100, 2), fill, dtype=torch.int32)
    p = F.fp8_moe_plan(ids.to(DEV), 4, align=32)
    for got, want, name in zip(p, R.plan(ids, 4, 32, p.src.numel()), p._fields):
        assert torch.equal(got.cpu(), want), name


def test_no_tokens():
    ids = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    p = F.fp8_moe_plan(ids, 4, align=32, rows=64)
    assert not p.offsets.any() and (p.src == -1).all()
    x = torch.empty(0, 128, dtype=BF, device=DEV)
    xs, _ = F.fp8_moe_permute(x, p.row_of, p.src)
    assert not xs.any()
    assert F.fp8_moe_unpermute(xs, p.row_of).shape == (0, 128)
    dys, dw = F.fp8_moe_unpermute_bwd(x, xs, p.row_of, p.src, torch.empty(0, 2, device=DEV))
    assert not dys.any() and dw.shape == (0, 2)


WIDTHS = [1, 3, 8, 20, 100, 256, 1000, 2048, 7168]


@pytest.mark.parametrize("dtype", [BF, torch.float32, torch.uint8])
@pytest.mark.parametrize("C", WIDTHS)
def test_permute(C, dtype):
    T, k, E = 70, 3, 9
    ids = _ids(T, k, E, 1)
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(T, C, generator=g) * 50).to(dtype)
    scale = torch.rand(T, generator=g) if dtype == torch.uint8 else None
    p = F.fp8_moe_plan(ids.to(DEV), E, align=16)
    xs, ss = F.fp8_moe_permute(x.to(DEV), p.row_of, p.src, scale=None if scale is None else scale.to(DEV))
    src = p.src.cpu().long()
    want = x[src.clamp_min(0) // k] * (src >= 0)[:, None].to(dtype)
    assert torch.equal(xs.cpu(), want)
    if scale is not None:
        assert torch.equal(ss.cpu(), scale[src.clamp_min(0) // k] * (src >= 0))


@pytest.mark.parametrize("C,dtype", [(40001, torch.uint8), (40000, torch.uint8), (16385, BF), (20000, torch.float32)])
def test_permute_long_rows(C, dtype):
    """Rows that a kernel takes in several parts."""
    ids = _ids(9, 2, 4, 1)
    x = (torch.randn(9, C, generator=torch.Generator().manual_seed(2)) * 50).to(dtype)
    p = F.fp8_moe_plan(ids.to(DEV), 4, align=4)
    xs, _ = F.fp8_moe_permute(x.to(DEV), p.row_of, p.src)
    src = p.src.cpu().long()
    assert torch.equal(xs.cpu(), x[src.clamp_min(0) // 2] * (src >= 0)[:, None].to(dtype))


@pytest.mark.parametrize("C", [12000, 20001])
def test_wide_weighted_sum(C):
    """Rows past what a CTA's registers hold."""
    ids = _ids(5, 3, 4, 1)
    g = torch.Generator().manual_seed(3)
    p = F.fp8_moe_plan(ids.to(DEV), 4, align=4)
    row = p.row_of.cpu().long()
    ys, dy = torch.randn(p.src.numel(), C, generator=g).to(BF), torch.randn(5, C, generator=g).to(BF)
    w = torch.rand(5, 3, generator=g)
    v = ys[row.clamp_min(0)].to(F64) * (row >= 0)[..., None]
    R.check(F.fp8_moe_unpermute(ys.to(DEV), p.row_of, weights=w.to(DEV)), (v * w.to(F64)[..., None]).sum(1),
            (v * w.to(F64)[..., None]).abs().sum(1), "y")
    _, dw = F.fp8_moe_unpermute_bwd(dy.to(DEV), ys.to(DEV), p.row_of, p.src, w.to(DEV))
    t = v * dy.to(F64)[:, None, :]
    R.check(dw, t.sum(2), t.abs().sum(2), "dweights")


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("k", [1, 2, 8, 13])
def test_weighted_sum_and_gradient(C, dtype, k):
    T, E = 67, 11
    ids = _ids(T, k, E, 3)
    ids[5] = -1                       # a token without experts
    g = torch.Generator().manual_seed(4)
    p = F.fp8_moe_plan(ids.to(DEV), E, align=16)
    row, src = p.row_of.cpu().long(), p.src.cpu().long()
    w = torch.rand(T, k, generator=g)
    ys = torch.randn(src.numel(), C, generator=g).to(dtype)
    ys[src < 0] = float("nan")        # pad rows are not read
    dy = torch.randn(T, C, generator=g).to(dtype)
    here = (row >= 0)[..., None]
    v = torch.where(here, ys[row.clamp_min(0)].to(F64), torch.zeros(1, dtype=F64))
    for weights in (w, None):
        wt = (torch.ones_like(w) if weights is None else w).to(F64)[..., None]
        y = F.fp8_moe_unpermute(ys.to(DEV), p.row_of, weights=None if weights is None else w.to(DEV))
        R.check(y, (v * wt).sum(1), (v * wt).abs().sum(1), "y")
        dys, dw = F.fp8_moe_unpermute_bwd(dy.to(DEV), ys.to(DEV), p.row_of, p.src,
                                          None if weights is None else w.to(DEV))
        at = src.clamp_min(0)
        want = dy.to(F64)[at // k] * wt.reshape(-1)[at][:, None] * (src >= 0)[:, None]
        R.check(dys, want, want.abs(), "dys")
        if weights is not None:
            t = v * dy.to(F64)[:, None, :]
            # 7168 terms: 28 a thread in order, then two trees
            R.check(dw, t.sum(2), t.abs().sum(2), "dweights")
            assert not dw[5].any()


def test_there_and_back():
    """With weight one and k copies, the way there and back multiplies by k:
    the permutation's gradient is the unweighted sum."""
    x = torch.randn(300, 512, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    ids = torch.stack([torch.arange(300) % 7, (torch.arange(300) + 3) % 7], 1).int().to(DEV)
    p = F.fp8_moe_plan(ids, 7, align=32)
    xs, _ = F.fp8_moe_permute(x, p.row_of, p.src)
    assert torch.equal(F.fp8_moe_unpermute(xs, p.row_of), x + x)


def test_rows_past_2_31_elements():
    """Row offsets pass 32 bits: the last rows of a buffer of 2^31 + elements."""
    C, rows = 16384, (1 << 17) + 64
    ys = torch.zeros(rows, C, dtype=BF, device=DEV)
    ys[-1] = 3.0
    row_of = torch.tensor([[rows - 1, -1], [0, rows - 1]], dtype=torch.int32, device=DEV)
    y = F.fp8_moe_unpermute(ys, row_of)
    assert (y == 3.0).all()
