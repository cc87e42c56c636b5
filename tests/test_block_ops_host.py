"""The operators between the linears, on the host: the references' gradients
against differences, and the refusals (checked before any CUDA call)."""
import ctypes

import pytest
import torch

import scaled_fp8_linear_gb300 as F
from scaled_fp8_linear_gb300 import block_ops as B
from tests import block_ref as R

F64 = torch.float64
FAKE = 0x10000   # a 16-byte-aligned address that is never dereferenced


def _diff(f, x, v, eps=1e-6):
    """Directional derivative of f at x along v, by central differences."""
    return (f(x + eps * v) - f(x - eps * v)) / (2 * eps)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("post", [False, True])
def test_norm_gradient_against_differences(kind, post):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)
    T, C, alpha, eps = 6, 10, 0.7, 1e-5
    v = {"x": r(T, C), "h": r(T, C), "gate": r(2, C), "w_post": r(C), "b_post": r(C) if kind else None,
         "w_pre": r(C), "b_pre": r(C) if kind else None}
    if not post:
        v["w_post"] = v["b_post"] = None
    dy, dxo = r(T, C), r(T, C)

    def loss(**kw):
        a = dict(v, **kw)
        xo, _, y, _, _ = R.norm_fwd(a["x"], a["h"], a["gate"], kind, eps, alpha, post, a["w_post"],
                                    a["b_post"], a["w_pre"], a["b_pre"])
        return (xo * dxo).sum() + (y * dy).sum()

    xo, _, _, _, st = R.norm_fwd(v["x"], v["h"], v["gate"], kind, eps, alpha, post, v["w_post"],
                                 v["b_post"], v["w_pre"], v["b_pre"])
    out = R.norm_bwd(dy, xo, dxo, v["h"], v["gate"], st, kind, alpha, post, v["w_post"], v["b_post"],
                     v["w_pre"])
    for name, t in v.items():
        if t is None:
            continue
        d = r(*t.shape)
        want = _diff(lambda x: loss(**{name: x}), t, d)
        assert abs((out["d" + name][0] * d).sum() - want) < 1e-5 * (1 + abs(want)), name


@pytest.mark.parametrize("act", range(5))
def test_activation_gradient_against_differences(act):
    z = torch.linspace(-6, 6, 241, dtype=F64) + 0.013
    want = _diff(lambda t: R.act(t, act), z, torch.ones_like(z))
    assert (R.act_grad(z, act) - want).abs().max() < 1e-8



@pytest.mark.parametrize("args", [B.NormFwdArgsC, B.NormBwdArgsC, B.GemmActArgsC, B.ActBwdArgsC])
def test_packed_arguments_have_the_struct_layout(args):
    """Each field lands where the C struct has it."""
    pack = B._packer(args)
    for i, (name, kind) in enumerate(args._fields_):
        values = [0] * len(args._fields_)
        values[i] = 1.5 if kind is ctypes.c_float else 77
        got = args.from_buffer_copy(pack(*values).ljust(ctypes.sizeof(args), b"\0"))
        for j, (other, _) in enumerate(args._fields_):
            assert (getattr(got, other) or 0) == values[j], (name, other)


def test_norm_refusals():
    L = B._lib()
    p = FAKE

    def fwd(**kw):
        f = dict(rows=4, width=64, kind=0, stream_type=0, eps=1e-5, alpha=1.0, x=p, h=p, y=p, x_out=p,
                 q_format=0, q_granularity=0)
        f.update(kw)
        return L.fp8_norm_fwd(ctypes.byref(B.NormFwdArgsC(**f)), None)

    assert L.fp8_norm_fwd(None, None) == -1
    assert fwd(rows=-1) == -2 and fwd(width=0) == -2 and fwd(rows=1 << 31) == -2
    assert fwd(width=16385) == -6
    assert fwd(kind=2) == -1 and fwd(stream_type=2) == -1 and fwd(eps=-1.0) == -1
    assert fwd(eps=float("nan")) == -1
    assert fwd(x=None, h=None) == -1 and fwd(h=None, post_norm=1) == -1 and fwd(h=None, gate=p, gate_rows=1) == -1
    assert fwd(gate=p, gate_rows=3) == -2 and fwd(gate=p, gate_rows=0) == -2 and fwd(gate_rows=2) == -2
    assert fwd(w_post=p) == -1                                   # without the post norm
    assert fwd(b_pre=p) == -6                                    # RMS takes no bias
    assert fwd(y=None, x_out=None) == -1                         # no output
    assert fwd(q=p) == -1 and fwd(q_scale=p) == -1 and fwd(amax=p) == -1
    assert fwd(q=p, q_scale=p, q_format=2) == -1
    assert fwd(q=p, q_scale_inv=p, q_granularity=1) == -6 and fwd(q=p, q_scale=p, q_granularity=7) == -1
    assert fwd(q=p, q_scale=p, q_granularity=3) == -1            # per row: q_scale_inv
    assert fwd(q=p, q_scale_inv=p, amax=p, q_granularity=3) == -1
    assert fwd(x=p + 8) == -3 and fwd(y=p + 2) == -3 and fwd(stats=p + 2) == -3
    assert "aligned" in F.fp8_last_error()

    def bwd(ws=p, ws_bytes=1 << 30, **kw):
        f = dict(rows=4, width=64, kind=0, stream_type=0, alpha=1.0, dy=p, x_out=p, h=p, stats=p, dx=p)
        f.update(kw)
        return L.fp8_norm_bwd(ctypes.byref(B.NormBwdArgsC(**f)), ws, ws_bytes, None)

    assert L.fp8_norm_bwd(None, None, 0, None) == -1
    assert bwd(rows=-1) == -2 and bwd(width=16385) == -6 and bwd(kind=5) == -1
    assert bwd(h=None, dh=p) == -1 and bwd(dw_post=p) == -1 and bwd(db_pre=p) == -6
    assert bwd(dgate=p) == -1 and bwd(dy=None) == -1 and bwd(x_out=None) == -1 and bwd(stats=None) == -1
    assert bwd(dy=None, dx_out=p, dw_pre=p) == -1
    assert bwd(dx=p + 4) == -3 and bwd(ws=p + 4) == -3
    assert bwd(ws=None) == -1 and bwd(ws_bytes=16) == -1
    assert "workspace" in F.fp8_last_error()
    assert F.fp8_norm_bwd_workspace_size(0, 64) == 0 and F.fp8_norm_bwd_workspace_size(4, 16385) == 0
    assert F.fp8_norm_bwd_workspace_size(5, 64, 2) == 0


def test_gemm_act_refusals():
    L = B._lib()
    p = FAKE

    def call(**kw):
        f = dict(A=p, B=p, M=128, N=64, K=64, scale_inv_a=p, scale_inv_b=p, d=p, experts=1)
        f.update(kw)
        return L.fp8_gemm_act(ctypes.byref(B.GemmActArgsC(**f)), None)

    assert L.fp8_gemm_act(None, None) == -1
    assert call(fa=2) == -1 and call(fb=-1) == -1 and call(act=5) == -1 and call(ga=9) == -1
    assert call(ga=1, gb=2) == -6 and call(ga=16) == -1
    assert call(M=-1) == -2 and call(N=0) == -2 and call(K=0) == -2 and call(N=72) == -2 and call(K=24) == -2
    assert call(M=1 << 31) == -2 and call(N=1 << 31) == -2
    assert call(experts=2) == -2 and call(experts=0, offsets=p) == -2 and call(experts=257, offsets=p) == -2
    assert call(A=None) == -1 and call(B=None) == -1 and call(scale_inv_a=None) == -1
    assert call(d=None) == -1 and call(q=p) == -1 and call(q_scale=p) == -1 and call(amax=p) == -1
    assert call(q=p, q_scale=p, q_format=3) == -1
    assert call(A=p + 8) == -3 and call(residual=p + 2) == -3 and call(bias=p + 8) == -3
    assert call(offsets=p + 2) == -3 and call(scale_inv_a=p + 1) == -3

    def bwd(ws=None, ws_bytes=0, **kw):
        f = dict(M=128, N=64, act=2, dD=p, z=p, dz=p)
        f.update(kw)
        return L.fp8_act_bwd(ctypes.byref(B.ActBwdArgsC(**f)), ws, ws_bytes, None)

    assert L.fp8_act_bwd(None, None, 0, None) == -1
    assert bwd(act=-1) == -1 and bwd(M=-1) == -2 and bwd(N=8) == -2 and bwd(dD=None) == -1
    assert bwd(dz=None) == -1 and bwd(q=p) == -1 and bwd(amax=p) == -1 and bwd(q=p, q_scale=p, q_format=2) == -1
    assert bwd(dbias=p) == -1 and bwd(dz=p + 8) == -3 and bwd(ws=p + 4, ws_bytes=1 << 20, dbias=p) == -3


def test_moe_refusals():
    L = B._lib()
    p = FAKE

    def plan(ids=p, tokens=8, slots=2, experts=4, align=16, offsets=p, counts=p, row_of=p, src=p,
             rows=256, ws=None, ws_bytes=0):
        return L.fp8_moe_plan(ids, tokens, slots, experts, align, offsets, counts, row_of, src, rows,
                              ws, ws_bytes, None)

    assert plan(tokens=-1) == -2 and plan(slots=0) == -2 and plan(slots=65) == -2
    assert plan(experts=0) == -2 and plan(experts=1025) == -2 and plan(align=0) == -2 and plan(align=4097) == -2
    assert plan(rows=16) == -2 and plan(tokens=1 << 30, rows=1 << 31) == -2
    assert "2^30" in F.fp8_last_error()
    assert plan(ids=None) == -1 and plan(offsets=None) == -1 and plan(src=None) == -1
    assert plan(ids=p + 2) == -3
    assert plan(tokens=5000, rows=20000) == -1                  # no workspace
    assert L.fp8_moe_permute(None, None, 4, 1, 64, p, p, 8, p, None, None) == -1
    assert L.fp8_moe_permute(p, p, 4, 1, 64, p, p, 8, p, None, None) == -1
    assert L.fp8_moe_permute(p, None, 4, 1, 0, p, p, 8, p, None, None) == -2
    assert L.fp8_moe_permute(p + 4, None, 4, 1, 64, p, p, 8, p, None, None) == -3
    assert L.fp8_moe_unpermute(p, 5, p, None, 4, 1, 64, 8, p, None) == -1
    assert L.fp8_moe_unpermute(p, 0, None, None, 4, 1, 64, 8, p, None) == -1
    assert L.fp8_moe_unpermute(p, 0, p, None, 4, 1, -1, 8, p, None) == -2
    assert L.fp8_moe_unpermute(p, 0, p, None, 4, 1, 64, 8, p + 2, None) == -3
    assert L.fp8_moe_unpermute_bwd(p, p, 7, p, p, None, 4, 1, 64, 8, p, None, None) == -1
    assert L.fp8_moe_unpermute_bwd(p, None, 0, p, p, None, 4, 1, 64, 8, p, None, None) == -1
    assert L.fp8_moe_unpermute_bwd(p, p, 0, p, None, None, 4, 1, 64, 8, p, None, None) == -1
    assert L.fp8_moe_unpermute_bwd(p + 8, p, 0, p, p, None, 4, 1, 64, 8, p, None, None) == -3
    assert F.fp8_moe_rows(8, 2, 4, 16) == 16 + 4 * 15 and F.fp8_moe_rows(1, 2, 256, 32) == 2 + 2 * 31
    with pytest.raises(ValueError):
        F.fp8_moe_rows(8, 0, 4)


def test_binding_refusals():
    """Shapes and types that the binding checks itself."""
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        F.fp8_norm_fwd(None, None)
    with pytest.raises(ValueError):
        F.fp8_norm_fwd(t(4, 8, 2))
    with pytest.raises(TypeError):
        F.fp8_norm_fwd(torch.zeros(4, 8, dtype=torch.float16))
    with pytest.raises(ValueError):
        F.fp8_norm_bwd(t(4, 8), t(4, 8), None, w_pre=torch.ones(8), accumulate=True)
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    with pytest.raises(ValueError):
        F.fp8_gemm_act(u(4, 32), 0, u(16, 48), 0, None, None)
    with pytest.raises(ValueError):
        F.fp8_gemm_act(u(4, 32), 0, u(17, 32), 0, None, None, gated=True)
    with pytest.raises(ValueError):
        F.fp8_gemm_act(u(4, 32), 0, u(16, 32), 0, None, None, offsets=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        F.fp8_act_bwd(t(4, 16), t(4, 16), 1, accumulate=True)
    with pytest.raises(TypeError):
        F.fp8_moe_unpermute(u(4, 16), torch.zeros(2, 1, dtype=torch.int32))
