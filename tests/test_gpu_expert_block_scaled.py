"""The block-scaled experts of examples/expert_block.py: against the same block in
64 bits, from a graph, and against the plain form of the same chain of casts.

Bounds of the first: as in tests/test_gpu_expert_block.py, relative 2-norm
errors.  A forward product's operands are off by at most 2^-4 each, two products
in a row; the weight gradients' kept operands are rounded once more (the
transposed re-cast, the 8-bit pre-activations): 0.25 for gradients covers the
E5M2 gradient, at most 2^-3, and three roundings of at most 2^-4 beside it in
quadrature with the chain before."""
import importlib.util
import os

import pytest
import torch

import scaled_fp8_linear_gb300 as F

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _status():
    yield
    assert F.fp8_device_status() == 0


def _block(*a, **kw):
    spec = importlib.util.spec_from_file_location("expert_block", os.path.join(ROOT, "examples", "expert_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m.BlockScaledExperts(*a, **kw)


def _inputs(tokens, width, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda s: (torch.randn(tokens, width, generator=g, device="cuda") * s).to(torch.bfloat16)
    return r(1.0), r(1e-2), r(1e-2)


def _rms(v, w):
    return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-5) * w


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("tokens,experts,slots", [(256, 4, 2), (700, 3, 1), (33, 8, 3), (1, 8, 2)])
def test_block(tokens, experts, slots, pow2):
    width, hidden = 512, 256
    block = _block(width, hidden, experts, slots, alpha=0.9, pow2=pow2)
    x, d_out, d_z = _inputs(tokens, width)
    x_out, z, s = block.forward(x)
    grads = block.backward(d_out, d_z, s)
    F.check_device_status()

    f64 = lambda t: t.detach().double().requires_grad_(True)
    p = {n: f64(getattr(block, n)) for n in ("w_pre", "w_post", "w_next", "gate", "w_in", "w_out")}
    p["x"], p["w"] = f64(x), f64(s["w"])
    y = _rms(p["x"], p["w_pre"])
    b = torch.zeros_like(y)
    for j in range(slots):
        for e in range(experts):
            t = (s["ids"][:, j] == e).nonzero()[:, 0]
            if t.numel():
                v = y[t] @ p["w_in"][e].t()
                h = torch.nn.functional.silu(v[:, :hidden]) * v[:, hidden:]
                b = b.index_add(0, t, (h @ p["w_out"][e].t()) * p["w"][t, j, None])
    b.retain_grad()
    xo = 0.9 * p["x"] + p["gate"] * _rms(b, p["w_post"])
    zo = _rms(xo, p["w_next"])
    off = lambda got, want: ((got.double() - want).norm() / want.norm()).item()
    assert off(x_out, xo) < 2 ** -2.5 and off(z, zo) < 2 ** -2.5
    ((xo * d_out.double()).sum() + (zo * d_z.double()).sum()).backward()
    for name, t in p.items():
        if name == "w" and slots == 1:
            # b = w o, and N_post(w o) does not depend on w but for the norm's epsilon:
            # dw = <db, o> is a sum whose terms cancel, and what is left of it is the
            # roundings of db and o, at most 0.25 of |db| |o| together
            o = (b / t).detach()
            assert (grads[name][:, 0].abs() <= 0.25 * b.grad.norm(dim=1) * o.norm(dim=1)).all()
            continue
        assert off(grads[name].view(t.shape), t.grad) < 0.25, name
    idle = torch.bincount(s["ids"].flatten().long(), minlength=experts) == 0
    assert (grads["w_in"][idle] == 0).all() and (grads["w_out"][idle] == 0).all()


def test_from_a_graph():
    """Forward and backward in one graph, replayed with other tokens and another
    routing: the bits of eager calls."""
    block = _block(512, 256, 8, 2, pow2=False)
    first, second = _inputs(300, 512, 2), _inputs(300, 512, 3)
    held = [t.clone() for t in first]

    def step(x, d_out, d_z):
        x_out, z, s = block.forward(x)
        return {"x_out": x_out, "z": z, **block.backward(d_out, d_z, s)}

    want = [{k: v.clone() for k, v in step(*t).items()} for t in (first, second)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*held)
    for t, w in zip((first, second), want):
        for a, b in zip(held, t):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for k, v in w.items():
            assert torch.equal(got[k], v), k


def test_chain_against_its_plain_form():
    """Each step of one expert's block from the codes that the step before left,
    in 64 bits: the weight gradients within 2^-16 of their terms' magnitudes (FP32
    sums of at most 3 blocks of 128 products each)."""
    block = _block(512, 256, 2, 1, pow2=False)
    x, d_out, d_z = _inputs(200, 512, 4)
    _, _, s = block.forward(x)
    plan, up = s["plan"], s["up"]
    do = F.fp8_moe_unpermute_bwd(d_out, s["o"], plan.row_of, plan.src, s["w"])[0]
    do_q, do_inv, do_t, do_inv_t = F.fp8_quantize_blocks(do, F.E5M2, F.GRAN_1x128, transpose=True)
    dh = F.fp8_gemm_experts(do_q, F.E5M2, block.out_qt, F.E4M3, do_inv, block.out_inv_t, plan.offsets)
    a = F.fp8_act_block_bwd(dh, up.z_q, up.z_scale_inv, F.ACT_SILU, gated=True, want_t=True, want_h_t=True,
                            offsets=plan.offsets)
    xs_t, xs_inv_t = F.fp8_block_transpose(s["xs"], F.E4M3, s["xs_inv"])
    dw = F.fp8_wgrad_experts(a.q_t, F.E5M2, xs_t, F.E4M3, a.scale_inv_t, xs_inv_t, plan.offsets)
    wide = lambda inv: inv.double().repeat_interleave(128, dim=1)
    v = lambda q, t, inv: q.view(t).double() * wide(inv)
    off = plan.offsets.tolist()
    dz_t, x_t = v(a.q_t, torch.float8_e5m2, a.scale_inv_t), v(xs_t, torch.float8_e4m3fn, xs_inv_t)
    for e in range(2):
        r = slice(off[e], off[e + 1])
        want, mag = dz_t[:, r] @ x_t[:, r].t(), dz_t[:, r].abs() @ x_t[:, r].abs().t()
        assert ((dw[e].double() - want).abs() <= 2.0 ** -16 * mag).all()
    # the re-cast input is the kept one to within half a step of the second rounding
    x_rows = v(s["xs"], torch.float8_e4m3fn, s["xs_inv"])[:off[-1]]
    step = 2.0 ** -4 * x_rows.abs() + 2.0 ** -10 * wide(xs_inv_t).t()[:off[-1]]
    assert ((x_t.t()[:off[-1]] - x_rows).abs() <= step * (1 + 2.0 ** -20)).all()
