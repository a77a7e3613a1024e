"""The softmax's sums over many tokens of like weight, in sliding-window attention.

A lane adds eight weights, those of 16 tokens being shared by two lanes, and takes
their sum into its running one: over n tokens the running sum is off by (n / 16 +
32) EPS of itself at most (its n / 16 additions, eight weights' own, the joining of
lanes and waves), EPS = 2^-24, where weight by weight it would be n / 2.  A score here
is a single product, off by EPS of itself, its exponent by 4 EPS: lse within (n / 16 +
32 + 16) EPS + 4 EPS |lse|, for every n up to 65 536.
"""
from __future__ import annotations

import math

import pytest
import torch

import mamba_chunked_ssd_amd as ssd

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


# weights of 0.7 beside the first token's: each is rounded the same way as it enters a sum
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_sums_of_like_weights(d, dtype):
    L, h = 65536, 3
    q, k, v = (torch.zeros((1, L, n, d), dtype=dtype, device="cuda") for n in (h, 1, 1))
    q[..., 0], k[..., 0], v[...] = 1, 0.640625, 1
    k[:, 0, :, 0] = 1
    _, lse = ssd.window_attention_fwd(q, k, v, scale=1.0, return_lse=True)
    n = torch.arange(1, L + 1, dtype=torch.float64, device="cuda")
    want = torch.log(math.e + (n - 1) * math.exp(0.640625))
    assert bool(((lse[0].double() - want).abs() <= (n / 16 + 48 + 4 * want.abs()) * EPS).all())
