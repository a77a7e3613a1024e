"""The attention step's weights: 16 bits of each in bf16 too.

Bounds as in test_gpu_attn.py, with E = (2 (D + 8) A + 2 n + 32) EPS for n slots
and A the largest scale sum |q||k|, but for the weights' rounding: what bf16 takes
off them (2^-8 relatively at most) goes into the product as an operand of its
own, again rounded by 2^-8, so that 2^-16 is left.  y is off by (E + 2^-16) sum p
|v|, and 2^-8 |y| for its own rounding.  Scores are small here, so that E is.
"""
from __future__ import annotations

import pytest
import torch

import mamba_chunked_ssd_amd as ssd

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


# one block for a cache and several; groups of one head, of some, of more than 32
@pytest.mark.parametrize("b,h,kv,d,w,n", [
    (3, 4, 4, 64, 5, 0), (40, 8, 2, 64, 12, 3), (2, 8, 1, 128, 30, 2), (5, 40, 1, 32, 9, 1), (64, 8, 4, 128, 100, 4),
    (1, 8, 2, 64, 5000, 4), (2, 12, 1, 128, 3001, 0), (1, 4, 2, 32, 6000, 100)])
def test_weights_keep_16_bits(b, h, kv, d, w, n):
    g = torch.Generator().manual_seed(w + d)
    rows = lambda *dims, size=1.0: (size * torch.randn(dims, generator=g)).bfloat16().cuda()  # noqa: E731
    q, k, v = rows(b, h, d, size=0.1), rows(b, kv, d, size=0.1), rows(b, kv, d)
    kc, vc = rows(b, kv, w + n, d, size=0.1), rows(b, kv, w + n, d)
    at = torch.arange(b, dtype=torch.int32, device="cuda") + 2 * (w + n)
    y = ssd.window_attention_step(q, k, v, kc, vc, at, w, n).double()
    # the caches now hold the new token too, and all of a cache is seen
    kk, vv = (x.double().repeat_interleave(h // kv, 1) for x in (kc, vc))
    p = torch.softmax((kk * q.double()[:, :, None]).sum(-1) * d ** -0.5, -1)[..., None]
    want, mag = (p * vv).sum(2), (p * vv.abs()).sum(2)
    a = d ** -0.5 * float(q.double().abs().flatten(0, 1).amax(0) @ kc.double().abs().flatten(0, 2).amax(0))
    e = (2 * (d + 8) * a + 2 * (w + n) + 32) * EPS
    assert bool(((y - want).abs() <= (e + 2.0 ** -16) * mag + 2.0 ** -8 * want.abs()).all())
