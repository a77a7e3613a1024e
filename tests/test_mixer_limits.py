"""Sizes and factors at the ends of their types, in the calls of sliding-window
attention and the RMS norm."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

import mamba_chunked_ssd_amd as ssd

INVALID = 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.LIB_PATH):
        from mamba_chunked_ssd_amd import build
        build.build()
    return ssd.load_library()


@pytest.mark.parametrize("scale,ok", [(2.3e38, True), (2.4e38, False), (3.4e38, False), (1e-45, True)])
def test_scale_times_log2_e(lib, scale, ok):
    # the workspace queries are 0 for shapes that their calls refuse
    shape = ssd.AttnShape(1, 64, 2, 1, 64, 8, 2, scale, ssd.SSD_DTYPE_F32)
    assert (lib.ssd_window_attn_bwd_workspace_size(ctypes.byref(shape)) > 0) == ok
    if not ok and not torch.cuda.is_available():  # (addresses of nothing)
        a = [(1 << 44) + (i << 36) for i in range(5)]
        st = lib.ssd_window_attn_fwd(ctypes.byref(shape), a[0], a[1], a[2], None, None, None, None, a[3], a[4], None)
        assert st == INVALID


@pytest.mark.gpu
def test_window_and_sinks_beyond_64_bits():
    q = torch.randn((1, 20, 2, 32), device="cuda")
    k = torch.randn((1, 20, 1, 32), device="cuda")
    want = ssd.window_attention_fwd(q, k, k)
    assert torch.equal(ssd.window_attention_fwd(q, k, k, (1 << 63) - 1), want)
    for kw in (dict(window=(1 << 64) + 5), dict(window=1 << 63), dict(window=5, sinks=(1 << 64) + 2), dict(window=-(1 << 64) + 5)):
        with pytest.raises(ValueError, match="64 bits"):
            ssd.window_attention_fwd(q, k, k, **kw)
    kc = torch.zeros((1, 1, 5, 32), device="cuda")
    at = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="64 bits"):
        ssd.window_attention_step(q[:, 0], k[:, 0], k[:, 0], kc, kc.clone(), at, (1 << 64) + 5)
