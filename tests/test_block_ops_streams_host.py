"""Where a call with stream= takes its memory, without a GPU: torch's
allocator hands out blocks by the stream that is current, so every tensor
that a call allocates has to be allocated with the given stream current.  One
from another stream's pool may still be in use by that stream's work."""
import pytest
import torch

import scaled_fp8_linear_gb300 as F
from scaled_fp8_linear_gb300 import block_ops as B

BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


class _Library:
    """The C calls, noting the stream that they get; sizes as if there were
    a GPU."""

    def __init__(self, log):
        self.log = log

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 4096
        if name == "fp8_moe_rows":
            return lambda *a: 64
        return lambda *a: self.log.append((name, a[-1])) or 0


@pytest.fixture
def world(monkeypatch):
    """Streams are numbers, current one in world.now; allocations and launches
    are noted with it."""
    class World:
        now, allocated, launched = 1, [], []
    World.allocated, World.launched = [], []

    class Stream:
        device_index = 0

        def __init__(self, number):
            self.stream_id = self.cuda_stream = number

    def set_stream(stream_id, device_index, device_type):
        World.now = stream_id

    def noted(make):
        def call(*a, **kw):
            World.allocated.append(World.now)
            return make(*a, **kw)
        return call

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(F, "_get_stream", lambda device: (World.now, 0, 1), raising=False)
    monkeypatch.setattr(F, "_set_stream", set_stream, raising=False)
    monkeypatch.setattr(F, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(F, "_devices", 1, raising=False)
    World.Stream = Stream
    monkeypatch.setattr(B, "_on", lambda *a: World.now)
    monkeypatch.setattr(F, "_stream", lambda stream: World.now if stream is None else int(stream))
    monkeypatch.setattr(F, "_ptr", lambda t, *a: None if t is None else t.data_ptr() or 16)
    monkeypatch.setattr(F, "_lib", _Library(World.launched))
    monkeypatch.setattr(B, "_given", lambda t, what, dtype, shape, *a: t.data_ptr() or 16)
    monkeypatch.setattr(B, "_here", lambda t: 0, raising=False)
    monkeypatch.setattr(B, "_ready", _Library(World.launched))
    monkeypatch.setattr(torch, "empty", noted(torch.empty))
    monkeypatch.setattr(torch, "empty_like", noted(torch.empty_like))
    monkeypatch.setattr(torch, "zeros", noted(torch.zeros))
    for cached in (B.fp8_act_bwd_workspace_size, B.fp8_moe_rows, B.fp8_moe_workspace_size):
        cached.cache_clear()
    yield World
    for cached in (B.fp8_act_bwd_workspace_size, B.fp8_moe_rows, B.fp8_moe_workspace_size):
        cached.cache_clear()


def _calls():
    t = lambda dt, *s: torch.full(s, 0, dtype=dt)
    x, w, ids = t(BF, 8, 32), t(F32, 32), t(I32, 8, 2)
    one, code, off = t(F32, 1), t(U8, 8, 32), t(I32, 3)
    plan = (t(I32, 8, 2), t(I32, 64))
    X, W = t(BF, 128, 128), t(BF, 128, 128)
    codes = lambda: dict(A=t(U8, 8, 32), fa=0, B=t(U8, 16, 32), fb=0, scale_inv_a=one, scale_inv_b=one)
    group = codes()
    layer = F.Fp8Linear(128, 128, 128, F.Recipe(F.SCALING_DYNAMIC), device="cpu")
    return {
        "linear_forward": lambda **k: layer.forward(X, W, **k),
        "linear_backward": lambda **k: layer.backward(X, **k),
        "amax": lambda **k: F.fp8_amax(x, **k),
        "quantize": lambda **k: F.fp8_quantize(X, F.E4M3, F.GRAN_ROW, transpose=True, want_amax=True, **k),
        "quantize_counted": lambda **k: F.fp8_quantize_counted(x, F.E4M3, one, transpose=True, want_amax=True, **k),
        "quantize_sr": lambda **k: F.fp8_quantize_sr(x, F.E4M3, one, 1, transpose=True, want_amax=True, **k),
        "quantize_blocks": lambda **k: F.fp8_quantize_blocks(X, F.E4M3, F.GRAN_1x128, transpose=True, **k),
        "gemm": lambda **k: F.fp8_gemm(**codes(), **k),
        "gemm_group": lambda **k: F.fp8_gemm_group(group, group, **k),
        "norm_fwd": lambda **k: F.fp8_norm_fwd(x, x, w_pre=w, want_stats=True, q_fmt=F.E4M3, q_gran=F.GRAN_ROW, **k),
        "norm_bwd": lambda **k: F.fp8_norm_bwd(x, x, t(F32, 4, 8), h=x, gate=t(BF, 1, 32), post_norm=True, w_post=w,
                                               w_pre=w, **k),
        "gemm_act": lambda **k: F.fp8_gemm_act(code, 0, t(U8, 16, 32), 0, one, one, want_z=True, q_fmt=F.E4M3,
                                               q_scale=one, want_amax=True, **k),
        "act_bwd": lambda **k: F.fp8_act_bwd(x, x, F.ACT_SILU, q_fmt=F.E5M2, q_scale=one, want_amax=True,
                                             want_dbias=True, **k),
        "act_bwd_experts": lambda **k: F.fp8_act_bwd(x, x, F.ACT_SILU, want_dbias=True, offsets=off, **k),
        "plan": lambda **k: F.fp8_moe_plan(ids, 4, **k),
        "permute": lambda **k: F.fp8_moe_permute(x, *plan, scale=t(F32, 8), **k),
        "unpermute": lambda **k: F.fp8_moe_unpermute(t(BF, 64, 32), plan[0], **k),
        "unpermute_bwd": lambda **k: F.fp8_moe_unpermute_bwd(x, t(BF, 64, 32), *plan, t(F32, 8, 2), **k),
    }


NAMES = ["act_bwd", "act_bwd_experts", "amax", "gemm", "gemm_act", "gemm_group", "linear_backward", "linear_forward",
         "norm_bwd", "norm_fwd", "permute", "plan", "quantize", "quantize_blocks", "quantize_counted", "quantize_sr",
         "unpermute", "unpermute_bwd"]


@pytest.mark.parametrize("by_object", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_comes_from_the_stream_of_the_call(world, name, by_object):
    call = _calls()[name]
    world.allocated.clear()     # what the arguments themselves took
    call(stream=world.Stream(7) if by_object else 7)
    assert world.allocated and set(world.allocated) == {7}
    assert [s for _, s in world.launched] == [7]
    assert world.now == 1
    world.allocated.clear()
    world.launched.clear()
    call()
    assert set(world.allocated) == {1} and [s for _, s in world.launched] == [1]


def test_stream_given_by_position(world):
    x, ids = torch.full((8, 32), 0, dtype=BF), torch.full((8, 2), 0, dtype=I32)
    F.fp8_moe_plan(ids, 4, 1, None, None, None, None, None, None, 7)
    F.fp8_moe_unpermute(x, ids, None, None, 9)
    assert [s for _, s in world.launched] == [7, 9] and set(world.allocated) == {7, 9}


def test_an_error_leaves_the_stream(world):
    with pytest.raises(TypeError):
        F.fp8_moe_unpermute(torch.zeros(4, 16, dtype=U8), torch.zeros(2, 1, dtype=I32), stream=7)
    assert world.now == 1
