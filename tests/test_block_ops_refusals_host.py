"""Refusals of the operators between the linears, beside those of
test_block_ops_host.py: checked before any CUDA call."""
import ctypes

import pytest
import torch

import scaled_fp8_linear_gb300 as F
from scaled_fp8_linear_gb300 import block_ops as B

FAKE = 0x10000   # a 16-byte-aligned address that is never dereferenced


def test_act_bwd_offsets():
    L, p = B._lib(), FAKE

    def bwd(ws=None, ws_bytes=0, **kw):
        f = dict(M=128, N=64, act=2, dD=p, z=p, dz=p, offsets=p, experts=4)
        f.update(kw)
        return L.fp8_act_bwd(ctypes.byref(B.ActBwdArgsC(**f)), ws, ws_bytes, None)

    assert bwd(experts=0) == -2 and bwd(experts=257) == -2 and bwd(experts=-1) == -2
    assert bwd(M=1 << 31) == -2
    assert bwd(offsets=p + 2) == -3
    need = F.fp8_act_bwd_workspace_size(128, 64, False, 4)
    assert need == (2 + 3) * 64 * 4 + 5 * 4      # row blocks of 64, cut by four experts; a table
    assert bwd(ws=p, ws_bytes=need - 1, dbias=p) == -1 and bwd(dbias=p) == -1
    assert "workspace" in F.fp8_last_error()
    t = torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        F.fp8_act_bwd(t, t, 1, offsets=torch.zeros(1, dtype=torch.int32), want_dz=False)
