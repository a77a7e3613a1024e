"""The RMS norm at sizes of u far from 1, up to the ends that its formulas leave
fp32: u r is of order 1 there, r^3 and products of u with itself are not.

Bounds as derived in test_gpu_norm.py, in units of EPS = 2^-24: they are
relative to the terms' magnitudes, and no intermediate value may leave fp32's
normal range where inputs, results and the sum of squares do not.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mamba_chunked_ssd_amd as ssd
from oracle import mixer_ops as mo

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def host(t):
    return t.double().cpu().numpy()


def half_step(dtype, ref):
    return 2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0


# rows of a wave, of a block, of neither
@pytest.mark.parametrize("c", [200, 2560, 5000, 17000])
@pytest.mark.parametrize("size", [1e-18, 1e-13, 1e-6, 1e12, 1e14, 1e15, 1e16, 1e17])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward(c, size, dtype):
    g = torch.Generator().manual_seed(c)
    u = (size * torch.randn((2, 3, c), generator=g)).to(TYPES[dtype]).cuda()
    dy = torch.randn((2, 3, c), generator=g).to(TYPES[dtype]).cuda()
    w = (1 + 0.3 * torch.randn(c, generator=g)).cuda()
    got = ssd.rms_norm_bwd(dy, u, w, eps=0.0, dx_dtype=TYPES[dtype], want_dresidual=True)
    du, dw, mag, wmag = mo.norm_bwd(host(dy), host(u), host(w), eps=0.0)
    for k in ("dx", "dresidual"):
        assert np.all(np.abs(host(got[k]) - du) <= 256 * EPS * mag + half_step(dtype, du)), k
    assert np.all(np.abs(host(got["dweight"]) - dw) <= 512 * EPS * wmag)


@pytest.mark.parametrize("c", [200, 5000, 17000])
@pytest.mark.parametrize("size", [1e-13, 1e16])
def test_backward_along_u(c, size):
    # dy w along u: the two terms cancel but for eps and the rounding of dy, du is what is left of them
    g = torch.Generator().manual_seed(c + 1)
    u = (size * torch.randn((1, 2, c), generator=g)).cuda()
    got = ssd.rms_norm_bwd(u / size, u, eps=0.0)
    du, _, mag, _ = mo.norm_bwd(host(u / size), host(u), eps=0.0)
    assert np.all(np.abs(host(got["dx"]) - du) <= 256 * EPS * mag)


@pytest.mark.parametrize("c", [200, 2560, 5000, 17000])
@pytest.mark.parametrize("size,weight", [(1e17, 1e22), (1e-13, 1e-28), (1e-13, 1e20), (1e16, 1e-30)])
@pytest.mark.parametrize("block", [0, 128])
def test_scales_where_u_times_weight_leaves_the_range(c, size, weight, block):
    # y = u r w is of order w; the scale is off by 64 EPS of itself, a code by half a step of e4m3 and 130 EPS
    g = torch.Generator().manual_seed(c)
    x = (size * torch.randn((2, 3, c), generator=g)).cuda()
    w = (weight * (1 + 0.3 * torch.randn(c, generator=g))).cuda()
    q, s = ssd.rms_norm_fwd(x, w, eps=0.0, y_dtype=torch.float8_e4m3fn, scale_block=block)
    _, y = mo.norm(host(x), host(w), eps=0.0)
    want, per = mo.scales(y, block)
    assert np.all(np.abs(host(s) - want) <= 64 * EPS * want)
    z = y / per
    assert np.all(np.abs(host(q.float()) - z) <= 2.0 ** -4 * np.maximum(np.abs(z), 2.0 ** -6) + 130 * EPS * np.abs(z))
    # in fp32 the same y
    assert np.all(np.abs(host(ssd.rms_norm_fwd(x, w, eps=0.0)) - y) <= 64 * EPS * np.abs(y))
