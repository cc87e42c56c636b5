"""Tensors of another device than the current one, without a GPU: the library
launches on the current device, so every call refuses them before a launch.
The tensors here are host tensors that say they are on a device."""
import pytest
import torch

import scaled_fp8_linear_gb300 as F
from scaled_fp8_linear_gb300 import block_ops as B

BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


class _On(torch.Tensor):
    number = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.number


def _on(number, dtype, *shape):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(_On)
    t.number = number
    return t


class _Library:
    """Sizes as if there were a GPU; no call may come through."""

    def __getattr__(self, name):
        def call(*a):
            if name.endswith("_size") or name == "fp8_moe_rows":
                return 64
            raise AssertionError(f"{name} was called")
        return call


@pytest.fixture(autouse=True)
def world(monkeypatch):
    monkeypatch.setattr(B, "_ready", _Library())
    monkeypatch.setattr(F, "_lib", _Library())
    monkeypatch.setattr(F, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(F, "_devices", 2, raising=False)
    monkeypatch.setattr(F, "_stream", lambda stream: 0)
    monkeypatch.setattr(B, "_on", lambda *a: 0)
    cached = (B.fp8_act_bwd_workspace_size, B.fp8_moe_rows, B.fp8_moe_workspace_size)
    for c in cached:
        c.cache_clear()
    yield
    for c in cached:
        c.cache_clear()


# each call with its tensors: (dtype, shape) by argument name
CALLS = {
    F.fp8_norm_fwd: (dict(x=(BF, 8, 32), h=(BF, 8, 32), gate=(BF, 2, 32), w_post=(F32, 32), w_pre=(F32, 32),
                          x_out=(BF, 8, 32), y=(BF, 8, 32), q=(U8, 8, 32), q_scale=(F32, 1), amax=(F32, 1),
                          stats=(F32, 4, 8)), dict(post_norm=True)),
    F.fp8_norm_bwd: (dict(dy=(BF, 8, 32), x_out=(BF, 8, 32), stats=(F32, 4, 8), dx_out=(BF, 8, 32), h=(BF, 8, 32),
                          gate=(BF, 2, 32), w_pre=(F32, 32), dx=(BF, 8, 32), dh=(BF, 8, 32), dw_pre=(F32, 32),
                          dgate=(F32, 2, 32), workspace=(U8, 4096)), {}),
    F.fp8_gemm_act: (dict(A=(U8, 8, 32), B=(U8, 2, 16, 32), scale_inv_a=(F32, 1), scale_inv_b=(F32, 2),
                          bias=(BF, 2, 16), residual=(BF, 8, 16), z=(BF, 8, 16), d=(BF, 8, 16), q=(U8, 8, 16),
                          q_scale=(F32, 1), amax=(F32, 1), offsets=(I32, 3)), dict(fa=0, fb=0)),
    F.fp8_act_bwd: (dict(dD=(BF, 8, 16), z=(BF, 8, 16), dz=(BF, 8, 16), q=(U8, 8, 16), q_scale=(F32, 1),
                         amax=(F32, 1), dbias=(F32, 2, 16), workspace=(U8, 4096), offsets=(I32, 3)), dict(act=1)),
    F.fp8_moe_plan: (dict(ids=(I32, 8, 2), offsets=(I32, 5), counts=(I32, 4), row_of=(I32, 8, 2), src=(I32, 64),
                          workspace=(U8, 4096)), dict(experts=4)),
    F.fp8_moe_permute: (dict(x=(U8, 8, 32), row_of=(I32, 8, 2), src=(I32, 64), scale=(F32, 8), xs=(U8, 64, 32),
                             scale_s=(F32, 64)), {}),
    F.fp8_moe_unpermute: (dict(ys=(BF, 64, 32), row_of=(I32, 8, 2), weights=(F32, 8, 2), y=(BF, 8, 32)), {}),
    F.fp8_moe_unpermute_bwd: (dict(dy=(BF, 8, 32), ys=(BF, 64, 32), row_of=(I32, 8, 2), src=(I32, 64),
                                   weights=(F32, 8, 2), dys=(BF, 64, 32), dweights=(F32, 8, 2)), {}),
    F.fp8_amax: (dict(x=(BF, 8, 32), amax=(F32, 1)), {}),
    F.fp8_update_scale: (dict(amax=(F32, 1), history=(F32, 4), pos=(I32, 1), scale=(F32, 1), scale_inv=(F32, 1)),
                         dict(history_len=4, algo=0, fmt=0, margin=0, pow2=False)),
    F.fp8_quantize: (dict(x=(BF, 8, 32), scale=(F32, 1), q=(U8, 8, 32), q_t=(U8, 32, 8), amax_out=(F32, 1)),
                     dict(fmt=0)),
    F.fp8_quantize_counted: (dict(x=(BF, 8, 32), scale=(F32, 1), counts=(torch.int64, 2), q=(U8, 8, 32)), dict(fmt=0)),
    F.fp8_quantize_sr: (dict(x=(BF, 8, 32), scale=(F32, 1), q=(U8, 8, 32)), dict(fmt=0, seed=1)),
    F.fp8_gemm: (dict(A=(U8, 8, 32), B=(U8, 16, 32), scale_inv_a=(F32, 1), scale_inv_b=(F32, 1), bias=(BF, 16),
                      D=(BF, 8, 16)), dict(fa=0, fb=0)),
}
CASES = [(call, name) for call, (tensors, _) in CALLS.items() for name in tensors]


def _run(call, numbers):
    tensors, rest = CALLS[call]
    return call(**{n: _on(numbers.get(n, numbers["rest"]), *spec) for n, spec in tensors.items()}, **rest)


@pytest.mark.parametrize("call,name", CASES, ids=lambda v: getattr(v, "__name__", v))
def test_one_tensor_elsewhere(call, name):
    with pytest.raises(ValueError, match="cuda:1"):
        _run(call, {"rest": 0, name: 1})


@pytest.mark.parametrize("call", list(CALLS), ids=lambda v: v.__name__)
def test_all_tensors_elsewhere(call):
    with pytest.raises(ValueError, match="current device"):
        _run(call, {"rest": 1})


@pytest.mark.parametrize("call", list(CALLS), ids=lambda v: v.__name__)
def test_all_tensors_here(call):
    """They pass the checks: the library is called."""
    with pytest.raises(AssertionError, match="was called"):
        _run(call, {"rest": 0})


def test_one_device_only(monkeypatch):
    """Numbers are not asked for, host tensors are refused all the same."""
    monkeypatch.setattr(F, "_devices", 1)
    with pytest.raises(AssertionError, match="was called"):
        _run(F.fp8_norm_fwd, {"rest": 0})
    x = torch.zeros(8, 32, dtype=BF)
    with pytest.raises(ValueError, match="CUDA"):
        F.fp8_norm_fwd(x, x)
    monkeypatch.setattr(F, "_devices", 2)
    with pytest.raises(ValueError, match="CUDA"):
        F.fp8_norm_fwd(x, x)
