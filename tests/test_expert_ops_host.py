"""The experts' products and the activations in blocks on the host: the references'
gradient against differences, refusals (checked before any CUDA call), packed
arguments, the device and the memory of a call."""
import ctypes

import pytest
import torch

import scaled_fp8_linear_gb300 as F
from scaled_fp8_linear_gb300 import block_ops as B
from scaled_fp8_linear_gb300 import expert_ops as X
from tests import block_ref as R
from tests import expert_ref as E

BF, U8, F32, I32, F64 = torch.bfloat16, torch.uint8, torch.float32, torch.int32, torch.float64
FAKE = 0x10000   # a 16-byte-aligned address that is never dereferenced


# ------------------------------------------------------------------ references

def test_cast_reference_against_torch():
    """Codes times factors are within half a step of what was cast."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 256, generator=g) * 10
    for fmt, half in ((0, 2.0 ** -4), (1, 2.0 ** -3)):
        for pow2 in (False, True):
            q, inv = E.cast(x, fmt, pow2)
            back, f = E.by_rows(q, inv, fmt), inv.to(F64).repeat_interleave(128, dim=1)
            low = 2.0 ** (-10 if fmt == 0 else -17)     # half the smallest step
            assert ((back - x.to(F64)).abs() <= half * x.to(F64).abs() * (1 + 2.0 ** -20) + low * f).all()
            if pow2:
                assert (torch.frexp(inv)[0] == 0.5).all()
    q, inv = E.cast(torch.zeros(1, 128), 0, False)
    assert (q == 0).all() and inv.item() == 1


@pytest.mark.parametrize("act", range(5))
def test_gated_gradient_against_differences(act):
    """dz of h = act(z_g) z_u, as the tests of the kernel take it."""
    g = torch.Generator().manual_seed(act)
    zg, zu, d = (torch.randn(50, generator=g, dtype=F64) for _ in range(3))
    zg = zg + 0.01 * torch.sign(zg)                  # away from ReLU's corner
    eps = 1e-6
    f = lambda a, b: (d * R.act(a, act) * b)
    dg = (f(zg + eps, zu) - f(zg - eps, zu)) / (2 * eps)
    du = (f(zg, zu + eps) - f(zg, zu - eps)) / (2 * eps)
    assert (d * zu * R.act_grad(zg, act) - dg).abs().max() < 1e-7
    assert (d * R.act(zg, act) - du).abs().max() < 1e-7


def test_products_by_offsets():
    """The reference's rows by any offsets."""
    a, b = torch.ones(4, 2, dtype=F64), torch.tensor([[[1.0, 0]], [[0, 3.0]]], dtype=F64)
    d, _, live = E.products(a, b, [-1, 2, 1])
    assert d[:, 0].tolist() == [1, 1, 0, 0] and live.tolist() == [True, True, False, False]
    assert E.held([3, 1, 9], 5) == [3, 3, 5]


# ------------------------------------------------------------------ refusals of the library

def _call(name, struct, base):
    f, keep = getattr(X._lib(), name), []

    def call(**kw):
        s = struct(**{**base, **kw})
        keep.append(s)
        return f(ctypes.byref(s), None)
    return call


def test_gemm_experts_refusals():
    p = FAKE
    call = _call("fp8_gemm_experts", X.GemmExpertsArgsC,
                 dict(A=p, B=p, M=300, N=256, K=384, scale_inv_a=p, scale_inv_b=p, d=p, offsets=p, experts=4))
    assert X._lib().fp8_gemm_experts(None, None) == -1
    assert call(fa=2) == -1 and call(fb=-1) == -1 and call(out=2) == -1 and call(out=-1) == -1
    assert call(M=-1) == -2 and call(N=0) == -2 and call(K=0) == -2
    assert call(N=192) == -2 and call(K=64) == -2 and call(N=-128) == -2
    assert call(experts=0) == -2 and call(experts=257) == -2
    assert call(M=1 << 31) == -2 and call(K=1 << 31) == -2 and call(N=1 << 31) == -2
    assert call(N=1 << 24, experts=256) == -2 and call(M=1 << 30, N=1 << 20) == -2
    assert "range" in F.fp8_last_error()
    for name in ("A", "B", "scale_inv_a", "scale_inv_b", "d", "offsets"):
        assert call(**{name: None}) == -1, name
    for name in ("A", "B", "d"):
        assert call(**{name: p + 8}) == -3, name
    for name in ("scale_inv_a", "scale_inv_b", "offsets"):
        assert call(**{name: p + 2}) == -3, name
    assert call(M=0, A=None, d=None, scale_inv_a=None) == 0        # no tokens


def test_wgrad_experts_refusals():
    p = FAKE
    call = _call("fp8_wgrad_experts", X.WgradExpertsArgsC,
                 dict(dY_t=p, X_t=p, f_dy=1, M=384, N=256, K=128, scale_inv_dy=p, scale_inv_x=p, dW=p, offsets=p, experts=2))
    assert X._lib().fp8_wgrad_experts(None, None) == -1
    assert call(f_dy=2) == -1 and call(f_x=-1) == -1
    assert call(M=-128) == -2 and call(M=100) == -2 and call(N=64) == -2 and call(K=0) == -2 and call(K=130) == -2
    assert call(experts=0) == -2 and call(experts=257) == -2
    assert call(M=1 << 31) == -2 and call(N=1 << 31) == -2 and call(N=1 << 24, experts=256) == -2
    assert call(N=1 << 22, K=1 << 22, experts=256) == -2
    for name in ("dY_t", "X_t", "scale_inv_dy", "scale_inv_x", "dW", "offsets"):
        assert call(**{name: None}) == -1, name
    for name in ("dY_t", "X_t", "dW"):
        assert call(**{name: p + 8}) == -3, name
    assert call(scale_inv_x=p + 1) == -3 and call(offsets=p + 2) == -3
    assert call(M=0, dW=None) == -1 and call(M=0, dW=p, accumulate=1) == 0


def test_act_block_refusals():
    p = FAKE
    call = _call("fp8_act_block", X.ActBlockArgsC, dict(M=10, N=256, act=2, z=p, q=p, scale_inv=p, offsets=p, experts=2))
    assert X._lib().fp8_act_block(None, None) == -1
    assert call(act=5) == -1 and call(act=-1) == -1 and call(q_format=2) == -1
    assert call(M=-1) == -2 and call(N=0) == -2 and call(N=64) == -2 and call(M=1 << 31) == -2
    assert call(N=1 << 31) == -2 and call(N=1 << 30, gated=1) == -2 and call(M=1 << 30, N=1 << 10) == -2
    assert call(experts=0) == -2 and call(experts=257) == -2
    assert call(z=None) == -1 and call(q=None, scale_inv=None) == -1
    assert call(scale_inv=None) == -1 and call(q=None) == -1 and call(z_q=p) == -1 and call(z_scale_inv=p) == -1
    assert call(z=p + 8) == -3 and call(q=p + 4) == -3 and call(z_q=p + 8, z_scale_inv=p) == -3
    assert call(scale_inv=p + 2) == -3 and call(offsets=p + 2) == -3
    assert call(M=0, z=None, q=None, scale_inv=None) == 0

    bwd = _call("fp8_act_block_bwd", X.ActBlockBwdArgsC,
                dict(M=256, N=256, act=2, dD=p, z_q=p, z_scale_inv=p, q=p, scale_inv=p, q_format=1))
    assert X._lib().fp8_act_block_bwd(None, None) == -1
    assert bwd(act=5) == -1 and bwd(q_format=2) == -1 and bwd(h_t=p, h_scale_inv_t=p, h_format=2) == -1
    assert bwd(M=-1) == -2 and bwd(N=100) == -2 and bwd(offsets=p, experts=0) == -2
    assert bwd(M=200, q_t=p, scale_inv_t=p) == -2 and bwd(M=200, h_t=p, h_scale_inv_t=p) == -2
    assert "multiple of 128" in F.fp8_last_error()
    for name in ("dD", "z_q", "z_scale_inv", "scale_inv", "q"):
        assert bwd(**{name: None}) == -1, name
    assert bwd(q=None, scale_inv=None) == -1
    assert bwd(q_t=p) == -1 and bwd(scale_inv_t=p) == -1 and bwd(h_t=p) == -1 and bwd(h_scale_inv_t=p) == -1
    assert bwd(dD=p + 8) == -3 and bwd(z_q=p + 8) == -3 and bwd(q_t=p + 8, scale_inv_t=p) == -3
    assert bwd(z_scale_inv=p + 2) == -3 and bwd(h_t=p, h_scale_inv_t=p + 2) == -3
    assert bwd(M=0, dD=None, z_q=None, z_scale_inv=None, q=None, scale_inv=None) == 0


def test_block_transpose_refusals():
    L, p = X._lib(), FAKE

    def call(q=p, inv=p, rows=256, cols=128, fmt=0, q_t=p, inv_t=p):
        return L.fp8_block_transpose(q, inv, rows, cols, fmt, 0, q_t, inv_t, None)

    assert call(rows=-128) == -2 and call(rows=100) == -2 and call(cols=0) == -2 and call(cols=64) == -2
    assert call(rows=1 << 31) == -2 and call(cols=1 << 31) == -2 and call(rows=1 << 30, cols=1 << 30) == -2
    assert call(fmt=2) == -1 and call(q=None) == -1 and call(inv=None) == -1 and call(q_t=None) == -1
    assert call(q=p + 8) == -3 and call(q_t=p + 8) == -3 and call(inv=p + 2) == -3 and call(inv_t=p + 1) == -3
    assert call(rows=0, q=None, inv=None, q_t=None, inv_t=None) == 0


def test_binding_refusals():
    u, f, i = (lambda *s: torch.zeros(*s, dtype=U8)), (lambda *s: torch.zeros(*s)), (lambda *s: torch.zeros(*s, dtype=I32))
    with pytest.raises(ValueError, match="experts"):
        F.fp8_gemm_experts(u(4, 128), 0, u(128, 128), 0, f(4, 1), f(1, 1), i(2))
    with pytest.raises(ValueError, match="A's K"):
        F.fp8_gemm_experts(u(4, 256), 0, u(1, 128, 128), 0, f(4, 2), f(1, 1, 1), i(2))
    with pytest.raises(ValueError, match="128"):
        F.fp8_gemm_experts(u(4, 64), 0, u(1, 128, 64), 0, f(4, 1), f(1, 1, 1), i(2))
    with pytest.raises(ValueError, match="out"):
        F.fp8_gemm_experts(u(4, 128), 0, u(1, 128, 128), 0, f(4, 1), f(1, 1, 1), i(2), out=5)
    with pytest.raises(ValueError, match="tokens"):
        F.fp8_wgrad_experts(u(128, 100), 1, u(128, 100), 0, f(128, 1), f(128, 1), i(2))
    with pytest.raises(ValueError, match="accumulate"):
        F.fp8_wgrad_experts(u(128, 128), 1, u(128, 128), 0, f(128, 1), f(128, 1), i(2), accumulate=True)
    with pytest.raises(ValueError, match="offsets"):
        F.fp8_wgrad_experts(u(128, 128), 1, u(128, 128), 0, f(128, 1), f(128, 1), None)
    with pytest.raises(ValueError, match="even"):
        F.fp8_act_block(torch.zeros(4, 129, dtype=BF), 1, gated=True)
    with pytest.raises(ValueError, match="128"):
        F.fp8_act_block(torch.zeros(4, 128, dtype=BF), 1, gated=True)
    with pytest.raises(ValueError, match="multiple of 128"):
        F.fp8_act_block_bwd(torch.zeros(4, 128, dtype=BF), u(4, 128), f(4, 1), 1, want_t=True)
    with pytest.raises(ValueError, match="rows"):
        F.fp8_block_transpose(u(4, 128), 0, f(4, 1))
    with pytest.raises(ValueError):
        F.fp8_block_transpose(u(128), 0, f(4, 1))
    with pytest.raises(ValueError, match="CUDA"):              # host tensors
        F.fp8_block_transpose(u(128, 128), 0, f(128, 1))


@pytest.mark.parametrize("args", [X.GemmExpertsArgsC, X.WgradExpertsArgsC, X.ActBlockArgsC, X.ActBlockBwdArgsC])
def test_packed_arguments_have_the_struct_layout(args):
    pack = B._packer(args)
    for i, (name, _) in enumerate(args._fields_):
        values = [0] * len(args._fields_)
        values[i] = 77
        got = args.from_buffer_copy(pack(*values).ljust(ctypes.sizeof(args), b"\0"))
        for j, (other, _) in enumerate(args._fields_):
            assert (getattr(got, other) or 0) == values[j], (name, other)


def test_status_word(monkeypatch):
    """Each bit of the device status word has its error."""
    for bit, error in ((F.STATUS_TIMEOUT, F.Fp8Error), (F.STATUS_OFFSETS, ValueError), (F.STATUS_NONFINITE, F.Fp8NumericsError)):
        monkeypatch.setattr(F, "fp8_device_status", lambda clear=True, bit=bit: bit)
        with pytest.raises(error):
            F.check_device_status()
    monkeypatch.setattr(F, "fp8_device_status", lambda clear=True: 0)
    F.check_device_status()


# ------------------------------------------------------------------ devices and memory

class _On(torch.Tensor):
    number = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.number


def _on(number, dtype, *shape):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(_On)
    t.number = number
    return t


CALLS = {
    F.fp8_gemm_experts: (dict(A=(U8, 8, 128), B=(U8, 2, 128, 128), scale_inv_a=(F32, 8, 1), scale_inv_b=(F32, 2, 1, 1),
                              offsets=(I32, 3), d=(BF, 8, 128)), dict(fa=0, fb=0)),
    F.fp8_wgrad_experts: (dict(dY_t=(U8, 256, 128), X_t=(U8, 128, 128), scale_inv_dy=(F32, 256, 1), scale_inv_x=(F32, 128, 1),
                               offsets=(I32, 3), dW=(F32, 2, 256, 128)), dict(f_dy=1, f_x=0)),
    F.fp8_act_block: (dict(z=(BF, 8, 256), q=(U8, 8, 128), scale_inv=(F32, 8, 1), z_q=(U8, 8, 256), z_scale_inv=(F32, 8, 2),
                           offsets=(I32, 3)), dict(act=2, gated=True)),
    F.fp8_act_block_bwd: (dict(dD=(BF, 128, 128), z_q=(U8, 128, 256), z_scale_inv=(F32, 128, 2), q=(U8, 128, 256),
                               scale_inv=(F32, 128, 2), q_t=(U8, 256, 128), scale_inv_t=(F32, 256, 1), h_t=(U8, 128, 128),
                               h_scale_inv_t=(F32, 128, 1), offsets=(I32, 3)), dict(act=2, gated=True)),
    F.fp8_block_transpose: (dict(q=(U8, 128, 256), scale_inv=(F32, 128, 2), q_t=(U8, 256, 128), scale_inv_t=(F32, 256, 1)),
                            dict(fmt=0)),
}
CASES = [(call, name) for call, (tensors, _) in CALLS.items() for name in tensors]
OUTPUTS = {"d", "dW", "q", "scale_inv", "z_q", "z_scale_inv", "q_t", "scale_inv_t", "h_t", "h_scale_inv_t"}


class _Library:
    def __init__(self, log=None):
        self.log = log

    def __getattr__(self, name):
        def call(*a):
            if self.log is None:
                raise AssertionError(f"{name} was called")
            self.log.append((name, a[-1]))
            return 0
        return call


@pytest.fixture
def two_devices(monkeypatch):
    monkeypatch.setattr(X, "_ready", _Library())
    monkeypatch.setattr(F, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(F, "_devices", 2, raising=False)
    monkeypatch.setattr(X, "_on", lambda *a: 0)


def _run(call, numbers):
    tensors, rest = CALLS[call]
    return call(**{n: _on(numbers.get(n, numbers["rest"]), *spec) for n, spec in tensors.items()}, **rest)


@pytest.mark.parametrize("call,name", CASES, ids=lambda v: getattr(v, "__name__", v))
def test_one_tensor_elsewhere(two_devices, call, name):
    with pytest.raises(ValueError, match="cuda:1"):
        _run(call, {"rest": 0, name: 1})


@pytest.mark.parametrize("call", list(CALLS), ids=lambda v: v.__name__)
def test_all_tensors_elsewhere_or_here(two_devices, call):
    with pytest.raises(ValueError, match="current device"):
        _run(call, {"rest": 1})
    with pytest.raises(AssertionError, match="was called"):     # they pass the checks
        _run(call, {"rest": 0})


@pytest.mark.parametrize("call,name", CASES, ids=lambda v: getattr(v, "__name__", v))
def test_shapes_and_types(two_devices, call, name):
    """Every tensor of another shape or type is refused."""
    tensors, rest = CALLS[call]
    dt, *shape = tensors[name]
    make = lambda n, spec: _on(0, *spec)
    good = {n: make(n, spec) for n, spec in tensors.items()}
    with pytest.raises((ValueError, TypeError)):
        call(**{**good, name: _on(0, torch.float64, *shape)}, **rest)
    if name == "offsets" and call in (F.fp8_act_block, F.fp8_act_block_bwd):
        return                                       # they say how many experts there are
    with pytest.raises((ValueError, TypeError)):
        call(**{**good, name: _on(0, dt, *shape[:-1], shape[-1] + 1)}, **rest)


@pytest.mark.parametrize("call", list(CALLS), ids=lambda v: v.__name__)
def test_memory_comes_from_the_stream_of_the_call(monkeypatch, call):
    """With stream= every new tensor is allocated with that stream current."""
    class World:
        now, allocated, launched = 1, [], []

    class Stream:
        device_index = 0

        def __init__(self, number):
            self.stream_id = self.cuda_stream = number

    World.allocated, World.launched = [], []
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(F, "_get_stream", lambda device: (World.now, 0, 1), raising=False)
    monkeypatch.setattr(F, "_set_stream", lambda i, d, t: setattr(World, "now", i), raising=False)
    monkeypatch.setattr(F, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(X, "_on", lambda *a: World.now)
    monkeypatch.setattr(X, "_here", lambda t: 0)
    monkeypatch.setattr(X, "_given", lambda t, what, dtype, shape, *a: t.data_ptr() or 16)
    monkeypatch.setattr(X, "_ready", _Library(World.launched))
    tensors, rest = CALLS[call]
    inputs = {n: torch.zeros(*spec[1:], dtype=spec[0]) for n, spec in tensors.items()
              if n not in OUTPUTS or (call is F.fp8_act_block_bwd and n in ("z_q", "z_scale_inv"))
              or (call is F.fp8_block_transpose and n in ("q", "scale_inv"))}
    more = {F.fp8_act_block: dict(keep=True), F.fp8_act_block_bwd: dict(want_t=True, want_h_t=True)}.get(call, {})
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: World.allocated.append(World.now) or empty(*a, **kw))
    for stream in (7, Stream(7)):
        World.allocated.clear(), World.launched.clear()
        call(**inputs, **rest, **more, stream=stream)
        assert World.allocated and set(World.allocated) == {7} and [s for _, s in World.launched] == [7]
        assert World.now == 1
    World.allocated.clear(), World.launched.clear()
    call(**inputs, **rest, **more)
    assert set(World.allocated) == {1} and [s for _, s in World.launched] == [1]
