"""Experts and activations in blocks of 128 at what depends on the device (the
choice of the products' kernel goes by its SMs), with offsets that change between
replays, factors that are not finite where nobody's tokens are, and checkpoints
of zeros.  Everything is exact: inputs as in tests/expert_ref.py, and numbers that
the codes hold."""
import pytest
import torch

import scaled_fp8_linear_gb300 as F
from tests import expert_ref as E

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _status():
    yield
    assert F.fp8_device_status() == 0


def _i32(off):
    return torch.tensor(off, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("N", [256, 640])
@pytest.mark.parametrize("past", [0, 1])
def test_rows_around_one_tile_an_sm(N, past, pow2):
    """The most rows whose 128 x 128 tiles fit on the device's SMs at once, and one
    more: the two sides of the rule, whatever the device."""
    num_n = N // 128
    M = torch.cuda.get_device_properties(0).multi_processor_count // num_n * 128 + past
    g = torch.Generator().manual_seed(N + past)
    a, b = E.exact_codes(g, 0, M, 384), E.exact_codes(g, 0, 1, N, 384)
    sa, sb = E.exact_factors(g, M, 3), E.exact_factors(g, 1, num_n, 3)
    got = F.fp8_gemm_experts(a.to(DEV), 0, b.to(DEV), 0, sa.to(DEV), sb.to(DEV), _i32([0, M]), out=F.OUT_F32, pow2=pow2)
    want, _, _ = E.products(E.by_rows(a, sa, 0), E.by_tiles(b, sb, 0), [0, M])
    assert torch.equal(got.cpu(), want.float())


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradients_beside_factors_that_are_not_finite(pow2, accumulate):
    """The factors of tokens of no expert, within the same group of four K blocks as
    others' and on their own."""
    for off in ([128, 640], [0, 128, 128, 256], [640, 640, 1152], [0, 0]):
        g = torch.Generator().manual_seed(off[-1])
        M, N, K, n = 1280, 384, 256, len(off) - 1
        dy, x = E.exact_codes(g, 1, N, M), E.exact_codes(g, 0, K, M)
        sy, sx = E.exact_factors(g, N, M // 128), E.exact_factors(g, K, M // 128)
        a, b = E.by_rows(dy, sy, 1), E.by_rows(x, sx, 0)
        want = torch.stack([a[:, s:t] @ b[:, s:t].t() for s, t in zip(off, off[1:])])
        for t, bad in ((sy, float("nan")), (sx, float("inf"))):
            t[:, :off[0] // 128], t[:, off[-1] // 128:] = bad, bad
        dw = torch.ones(n, N, K, device=DEV) if accumulate else None
        got = F.fp8_wgrad_experts(dy.to(DEV), 1, x.to(DEV), 0, sy.to(DEV), sx.to(DEV), _i32(off), pow2=pow2, dW=dw,
                                  accumulate=accumulate)
        assert torch.equal(got.cpu(), (want + accumulate).float())


@pytest.mark.parametrize("call", ["wgrad", "wgrad_pow2", "act", "act_bwd", "act_bwd_tokens"])
def test_offsets_change_between_replays(call):
    """A graph reads the offsets of the replay, not of the capture: the bits of eager
    calls, whose rows and blocks without experts stay as they were too."""
    g = torch.Generator().manual_seed(2)
    M, N, o = 640, 256, _i32([0, 0, 0])
    fill = lambda *s: torch.empty(*s, dtype=torch.uint8, device=DEV)
    f32 = lambda *s: torch.empty(*s, device=DEV)
    if call.startswith("wgrad"):
        q = [E.any_codes(g, f, N, M).to(DEV) for f in (1, 0)]
        inv = [E.exact_factors(g, N, M // 128).to(DEV) for _ in q]
        out = [f32(2, N, N)]
        run = lambda: F.fp8_wgrad_experts(q[0], 1, q[1], 0, inv[0], inv[1], o, pow2=call == "wgrad_pow2", dW=out[0])
    elif call == "act":
        z = torch.randn(M, 2 * N, generator=g).to(BF).to(DEV)
        out = [fill(M, N), f32(M, N // 128), fill(M, 2 * N), f32(M, 2 * N // 128)]
        run = lambda: F.fp8_act_block(z, F.ACT_SILU, gated=True, q=out[0], scale_inv=out[1], z_q=out[2],
                                      z_scale_inv=out[3], offsets=o)
    else:
        d = torch.randn(M, N, generator=g).to(BF).to(DEV)
        zq, z_inv = [t.to(DEV) for t in E.cast(torch.randn(M, 2 * N, generator=g), 0, False)]
        out = [fill(M, 2 * N), f32(M, 2 * N // 128)]
        kw = dict(q=out[0], scale_inv=out[1])
        if call == "act_bwd_tokens":
            out += [fill(2 * N, M), f32(2 * N, M // 128), fill(N, M), f32(N, M // 128)]
            kw.update(q_t=out[2], scale_inv_t=out[3], h_t=out[4], h_scale_inv_t=out[5])
        run = lambda: F.fp8_act_block_bwd(d, zq, z_inv, F.ACT_GELU, gated=True, offsets=o, **kw)

    def reset():
        for t in out:
            t.view(torch.uint8).fill_(0x3A)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for off in ([0, 128, 640], [128, 384, 384], [256, 256, 256], [0, 512, 512]):
        o.copy_(_i32(off))
        reset()
        run()
        want = [t.clone() for t in out]
        reset()
        graph.replay()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, want))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tokens", [False, True])
@pytest.mark.parametrize("act,slope", [(F.ACT_NONE, 1.0), (F.ACT_RELU, 0.0), (F.ACT_SILU, 0.5), (F.ACT_GELU, 0.5),
                                       (F.ACT_GELU_TANH, 0.5)])
def test_gradient_of_a_checkpoint_of_zeros(act, slope, tokens, gated):
    """act(0) = 0, and its derivative there: ReLU's is 0.  d holds powers of two, so
    codes with power-of-two factors hold every gradient, and a derivative that is
    half but for 1e-6 rounds to the same."""
    M, N = 128, 256
    g = torch.Generator().manual_seed(act)
    d = (2.0 ** torch.randint(-3, 4, (M, N), generator=g).float() * (torch.randint(0, 2, (M, N), generator=g) * 2 - 1))
    zq = torch.zeros(M, 2 * N if gated else N, dtype=torch.uint8)
    if gated:
        zq[:, N:] = 0x38                       # 1
    inv = torch.full((M, zq.shape[1] // 128), 2.0)
    o = F.fp8_act_block_bwd(d.to(BF).to(DEV), zq.to(DEV), inv.to(DEV), act, gated=gated, q_fmt=F.E4M3, pow2=True,
                            want_t=tokens, want_h_t=tokens)
    want = torch.zeros(M, zq.shape[1])
    want[:, :N] = d * slope * (2.0 if gated else 1.0)
    assert torch.equal(E.by_rows(o.q, o.scale_inv, 0), want.to(E.F64))
    if tokens:
        assert torch.equal(E.by_rows(o.q_t, o.scale_inv_t, 0), want.t().to(E.F64))
        assert (o.h_t & 0x7F == 0).all() and (o.h_scale_inv_t == 1).all()
