"""The operators between the linears on other streams than the current one,
with no wait between independent calls, and from graphs: the same bits as one
call after the other."""
import pytest
import torch

import scaled_fp8_linear_gb300 as F

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _status():
    yield
    assert F.fp8_device_status() == 0


def _norm_bwd(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    T, C = 4096, 4096
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    dy, x, h, gate = r(T, C).to(BF), r(T, C).to(BF), r(T, C).to(BF), r(4, C).to(BF)
    w1, w2, st = 1 + 0.1 * r(C), 1 + 0.1 * r(C), 0.5 + torch.rand(4, T, generator=g, device=DEV)
    return lambda **k: F.fp8_norm_bwd(dy, x, st, dx_out=dy, h=h, gate=gate, post_norm=True, w_post=w1, w_pre=w2, **k)


def _act_bwd(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    d, z = (torch.randn(4096, 2048, generator=g, device=DEV).to(BF) for _ in range(2))
    return lambda **k: F.fp8_act_bwd(d, z, F.ACT_GELU, want_dbias=True, **k)


def _act_bwd_experts(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    d, z = (torch.randn(4096, 2048, generator=g, device=DEV).to(BF) for _ in range(2))
    off = torch.tensor([0, 700, 701, 4096], dtype=torch.int32, device=DEV)
    return lambda **k: F.fp8_act_bwd(d, z, F.ACT_SILU, want_dbias=True, offsets=off, **k)


def _plan(seed):
    ids = torch.randint(-1, 64, (20000, 8), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).to(DEV)
    return lambda **k: F.fp8_moe_plan(ids, 64, align=16, **k)


def _there_and_back(seed):
    """The sort, the copy, the weighted sum and its gradient."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    ids = torch.randint(-1, 16, (3000, 4), generator=g, device=DEV, dtype=torch.int32)
    x, w = torch.randn(3000, 1000, generator=g, device=DEV).to(BF), torch.rand(3000, 4, generator=g, device=DEV)

    def call(**k):
        p = F.fp8_moe_plan(ids, 16, align=8, **k)
        xs, _ = F.fp8_moe_permute(x, p.row_of, p.src, **k)
        y = F.fp8_moe_unpermute(xs, p.row_of, weights=w, **k)
        return (*p, xs, y, *F.fp8_moe_unpermute_bwd(x, xs, p.row_of, p.src, w, **k))
    return call


def _product(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    a, b = (torch.randint(0, 0x70, s, generator=g, device=DEV, dtype=torch.uint8) for s in ((2048, 1024), (1024, 1024)))
    one = torch.full((1,), 2.0 ** -8, device=DEV)
    return lambda **k: F.fp8_gemm_act(a, F.E4M3, b, F.E4M3, one, one, act=F.ACT_SILU, want_z=True, q_fmt=F.E4M3,
                                      q_scale=one, want_amax=True, **k)


CALLS = [_norm_bwd, _act_bwd, _act_bwd_experts, _plan, _there_and_back, _product]


def _same(a, b):
    return all(x is y is None or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("make", CALLS)
@pytest.mark.parametrize("raw", [False, True])
def test_independent_calls_on_two_streams(make, raw):
    here, there = make(1), make(2)
    want = here(), there()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(6):
        a = here()
        b = there(stream=s.cuda_stream if raw else s)
        got.append((a, b))
    torch.cuda.synchronize()
    assert all(_same(a, want[0]) and _same(b, want[1]) for a, b in got)


@pytest.mark.parametrize("make", CALLS)
def test_default_stream_by_handle(make):
    """Handle 0 while another stream is current."""
    call = make(3)
    want = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call(stream=0)
        mine = call()
        assert torch.cuda.current_stream() == s
    torch.cuda.synchronize()
    assert _same(got, want) and _same(mine, want)


@pytest.mark.parametrize("make", CALLS)
def test_from_a_graph(make):
    call = make(4)
    want = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for t in got:
        if t is not None:
            t.view(torch.uint8).fill_(0x55)
    graph.replay()
    torch.cuda.synchronize()
    assert _same(got, want)


def _casts_and_products(seed):
    """The linears' own calls: casts (one adds to counters that it sets to
    zero itself) and a product."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(4096, 2048, generator=g, device=DEV).to(BF)
    w = torch.randint(0, 0x70, (1024, 2048), generator=g, device=DEV, dtype=torch.uint8)
    one, inv = torch.full((1,), 300.0, device=DEV), torch.full((1,), 2.0 ** -12, device=DEV)

    def call(**k):
        q, q_t, amax, counts = F.fp8_quantize_counted(x, F.E4M3, one, transpose=True, want_amax=True, **k)
        blocks = F.fp8_quantize_blocks(x, F.E4M3, F.GRAN_1x128, transpose=True, **k)
        return (q, q_t, amax, counts, *blocks, F.fp8_amax(x, **k),
                F.fp8_gemm(q, F.E4M3, w, F.E4M3, inv, inv, out=F.OUT_F32, **k))
    return call


def _layer(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    layer = F.Fp8Linear(2048, 1024, 1024, F.Recipe(F.SCALING_DYNAMIC))
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)
    x, w, dy = r(2048, 1024), r(1024, 1024), r(2048, 1024)
    return lambda **k: (layer.forward(x, w, **k), *layer.backward(dy, **k))


@pytest.mark.parametrize("make", [_casts_and_products, _layer])
def test_the_linears_on_two_streams(make):
    here, there = make(1), make(2)
    want = here(), there()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [(here(), there(stream=s)) for _ in range(6)]
    torch.cuda.synchronize()
    assert all(_same(a, want[0]) and _same(b, want[1]) for a, b in got)
