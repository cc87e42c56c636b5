"""The experts' products and the activations in blocks on other streams than the
current one, with no wait between independent calls, and from graphs: the same
bits as one call after the other."""
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


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _offsets(off):
    return torch.tensor(off, dtype=torch.int32, device=DEV)


def _product(off, pow2):
    def make(seed):
        g, m = _gen(seed), off[-1]
        a, b = E.any_codes(g, 0, m, 1024).to(DEV), E.any_codes(g, 0, 4, 512, 1024).to(DEV)
        sa, sb = E.exact_factors(g, m, 8).to(DEV), E.exact_factors(g, 4, 4, 8).to(DEV)
        o = _offsets(off)
        return lambda **k: (F.fp8_gemm_experts(a, 0, b, 0, sa, sb, o, out=F.OUT_F32, pow2=pow2, **k),)
    return make


def _wgrad(pow2):
    def make(seed):
        g = _gen(seed)
        dy, x = E.any_codes(g, 1, 512, 1024).to(DEV), E.any_codes(g, 0, 384, 1024).to(DEV)
        sy, sx = E.exact_factors(g, 512, 8).to(DEV), E.exact_factors(g, 384, 8).to(DEV)
        o = _offsets([0, 256, 256, 896])
        return lambda **k: (F.fp8_wgrad_experts(dy, 1, x, 0, sy, sx, o, pow2=pow2, **k),)
    return make


def _act(seed):
    z = (torch.randn(2000, 2048, generator=_gen(seed)) * 2).to(BF).to(DEV)
    return lambda **k: F.fp8_act_block(z, F.ACT_GELU, gated=True, keep=True, **k)


def _act_bwd(tokens):
    def make(seed):
        g = _gen(seed)
        d = torch.randn(2048, 1024, generator=g).to(BF).to(DEV)
        q, inv = E.cast(torch.randn(2048, 2048, generator=g), 0, False)
        q, inv = q.to(DEV), inv.to(DEV)
        return lambda **k: F.fp8_act_block_bwd(d, q, inv, F.ACT_SILU, gated=True, want_t=tokens, want_h_t=tokens, **k)
    return make


def _transpose(seed):
    g = _gen(seed)
    q, inv = E.any_codes(g, 0, 2048, 1024).to(DEV), E.exact_factors(g, 2048, 8).to(DEV)
    return lambda **k: F.fp8_block_transpose(q, F.E4M3, inv, **k)


CALLS = {"few": _product([0, 9, 9, 20, 31], False), "some": _product([0, 50, 90, 190, 200], False),
         "many": _product([0, 300, 301, 700, 1200], False), "many_pow2": _product([0, 300, 301, 700, 1200], True),
         "wgrad": _wgrad(False), "wgrad_pow2": _wgrad(True), "act": _act, "act_bwd": _act_bwd(False),
         "act_bwd_tokens": _act_bwd(True), "transpose": _transpose}


def _same(a, b):
    return all(x is y is None or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_independent_calls_on_two_streams(name, raw):
    here, there = CALLS[name](1), CALLS[name](2)
    want = here(), there()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [(here(), there(stream=s.cuda_stream if raw else s)) for _ in range(6)]
    torch.cuda.synchronize()
    assert all(_same(a, want[0]) and _same(b, want[1]) for a, b in got)


@pytest.mark.parametrize("name", CALLS)
def test_from_a_graph(name):
    call = CALLS[name](4)
    want = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(2):
        for t in got:
            if t is not None:
                t.view(torch.uint8).fill_(0x55)
        graph.replay()
        torch.cuda.synchronize()
        assert _same(got, want)


def test_offsets_change_between_replays():
    """A graph reads the offsets of the replay, not of the capture."""
    g = _gen(5)
    a, b = E.exact_codes(g, 0, 600, 256), E.exact_codes(g, 0, 3, 256, 256)
    sa, sb = E.exact_factors(g, 600, 2), E.exact_factors(g, 3, 2, 2)
    o, dev = _offsets([0, 0, 0, 0]), [t.to(DEV) for t in (a, b, sa, sb)]
    d = torch.zeros(600, 256, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.fp8_gemm_experts(dev[0], 0, dev[1], 0, dev[2], dev[3], o, out=F.OUT_F32, d=d)
    for off in ([0, 10, 300, 600], [5, 500, 500, 600], [0, 0, 0, 1]):
        d.fill_(7)
        o.copy_(_offsets(off))
        graph.replay()
        want, _, live = E.products(E.by_rows(a, sa, 0), E.by_tiles(b, sb, 0), off)
        got = d.cpu()
        assert torch.equal(got[live], want[live].float()) and (got[~live] == 7).all()


# ------------------------------------------------------------------ offsets past 32 bits

def test_long_rows_of_a_product():
    """D past 2^31 elements: the last rows."""
    g = _gen(6)
    M, N, tail = (1 << 31) // 8192 + 300, 8192, 400
    a = torch.zeros(M, 128, dtype=torch.uint8, device=DEV)
    sa = torch.ones(M, 1, device=DEV)
    at, st = E.exact_codes(g, 0, tail, 128), E.exact_factors(g, tail, 1)
    a[-tail:], sa[-tail:] = at.to(DEV), st.to(DEV)
    b, sb = E.exact_codes(g, 0, 2, N, 128), E.exact_factors(g, 2, N // 128, 1)
    for pow2 in (False, True):
        d = F.fp8_gemm_experts(a, 0, b.to(DEV), 0, sa, sb.to(DEV), _offsets([0, M - 150, M]), pow2=pow2)
        want, _, _ = E.products(E.by_rows(at, st, 0), E.by_tiles(b, sb, 0), [0, tail - 150, tail])
        assert torch.equal(d[-tail:].cpu(), want.to(BF)) and (d[:1000] == 0).all()
        del d


def test_long_weight_gradients():
    g = _gen(7)
    n, N, K = 33, 8192, 8192                       # 2.2e9 numbers
    dy, x = E.exact_codes(g, 1, N, 256), E.exact_codes(g, 0, K, 256)
    sy, sx = E.exact_factors(g, N, 2), E.exact_factors(g, K, 2)
    off = [0] + [128] * (n - 1) + [256]
    want = E.by_rows(dy, sy, 1)[-256:, 128:] @ E.by_rows(x, sx, 0)[:, 128:].t()
    for pow2 in (False, True):
        dw = F.fp8_wgrad_experts(dy.to(DEV), 1, x.to(DEV), 0, sy.to(DEV), sx.to(DEV), _offsets(off), pow2=pow2)
        assert torch.equal(dw[-1, -256:].cpu(), want.float()) and (dw[1:-1] == 0).all()
        del dw


def test_long_activations():
    g = _gen(8)
    N, tail = 16384, 256
    M = ((1 << 31) // (2 * N) + 512) // 128 * 128
    z = torch.zeros(M, 2 * N, dtype=BF, device=DEV)
    zt = torch.randn(tail, 2 * N, generator=g).to(BF).to(DEV)
    z[-tail:] = zt
    o, small = (F.fp8_act_block(t, F.ACT_SILU, gated=True, keep=True) for t in (z, zt))
    for a, b in zip(o, small):
        assert torch.equal(a[-tail:], b)
    del z
    d = torch.zeros(M, N, dtype=BF, device=DEV)
    dt = torch.randn(tail, N, generator=g).to(BF).to(DEV)
    d[-tail:] = dt
    for tokens in (True, False):
        kw = dict(gated=True, want_t=tokens, want_h_t=tokens)
        big = F.fp8_act_block_bwd(d, o.z_q, o.z_scale_inv, F.ACT_SILU, **kw)
        few = F.fp8_act_block_bwd(dt, small.z_q, small.z_scale_inv, F.ACT_SILU, **kw)
        for name, a, b in zip(big._fields, big, few):
            if a is not None:
                cut = a[-tail:] if name in ("q", "scale_inv") else a[:, -b.shape[1]:]
                assert torch.equal(cut, b), name
        del big
    t, inv = F.fp8_block_transpose(o.z_q, F.E4M3, o.z_scale_inv)
    ts, invs = F.fp8_block_transpose(small.z_q, F.E4M3, small.z_scale_inv)
    assert torch.equal(t[:, -tail:], ts) and torch.equal(inv[:, -2:], invs)
