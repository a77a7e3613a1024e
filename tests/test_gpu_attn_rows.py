"""Every element of sliding-window attention's gradients where no kernel for few
blocks is taken: tiles, blocks and groups of waves of the large sizes, whose
remainders of rows a norm over the whole gradient would not show.

Bounds per element as derived in test_gpu_attn.py: dq and dk within 4 (E + R) of
the sums of their terms' magnitudes, dv within E + R, each and R (bf16 2^-8) and
EPS of itself; y within (E + R) sum p |v| and R |y|.
"""
from __future__ import annotations

import math

import pytest
import torch

import mamba_chunked_ssd_amd as ssd

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f32": 0.0}
LENGTHS = [300, 0, 1, 299, 129, 128, 127, 33, 200, 257, 65]


def reference(q, k, v, dy, w, n, scale, ends):
    """y, gradients and their terms' magnitudes, lse, in fp64, heads first, rows behind a sequence's end 0."""
    g = q.shape[2] // k.shape[2]
    L = q.shape[1]
    live = (torch.arange(L, device="cuda") < ends[:, None])[:, None, :, None].double()
    q, dy = (x.double().transpose(1, 2) * live for x in (q, dy))
    k, v = (x.double().repeat_interleave(g, 2).transpose(1, 2) for x in (k, v))
    t = torch.arange(L, device="cuda")
    back = t[:, None] - t
    on = (back >= 0) & ((back < w) | (t < n))
    across = lambda x: x.transpose(2, 3).contiguous()  # noqa: E731
    z = (q @ across(k) * scale).masked_fill(~on, -math.inf)
    p = torch.softmax(z, -1) * live
    dp, part = dy @ across(v), dy.abs() @ across(v.abs())
    ds = scale * p * (dp - (p * dp).sum(-1, keepdim=True))
    dsm = scale * p * (part + (p * part).sum(-1, keepdim=True))
    share = lambda x: x.unflatten(1, (-1, g)).sum(2)  # noqa: E731
    return dict(y=(p @ v, p @ v.abs()), dq=(ds @ k, dsm @ k.abs()), dk=(share(across(ds) @ q), share(across(dsm) @ q.abs())),
                dv=(share(across(p) @ dy), share(across(p) @ dy.abs()))), torch.logsumexp(z, -1) * live[..., 0]


def check(q, k, v, dy, w, n, ends, dtype):
    d = q.shape[-1]
    scale = d ** -0.5
    lengths = torch.tensor(ends, dtype=torch.int32, device="cuda")
    y, lse = ssd.window_attention_fwd(q, k, v, w, n, lengths=lengths, return_lse=True)
    got = dict(ssd.window_attention_bwd(q, k, v, y, lse, dy, w, n, lengths=lengths), y=y)
    want, rlse = reference(q, k, v, dy, w, n, scale, lengths)
    a = scale * float(q.double().abs().flatten(0, -2).amax(0) @ k.double().abs().flatten(0, -2).amax(0))
    e, r = (2 * (d + 8) * a + 2 * (w + n) + 32) * EPS, ROUND[dtype]
    assert bool(((lse.double() - rlse).abs() <= (2 * (d + 8) * a + w + n + 8 + 4 * rlse.abs()) * EPS * (rlse != 0)).all())
    for name, (ref, mag) in want.items():
        m = 4 if name in ("dq", "dk") else 1
        bad = (got[name].double().transpose(1, 2) - ref).abs() > m * (e + r) * mag + (r + EPS) * ref.abs()
        assert not bool(bad.any()), (name, bad.nonzero()[:5].tolist(), int(bad.sum()))


def inputs(b, L, h, kv, d, dtype, layout, seed):
    g = torch.Generator().manual_seed(seed + d)
    out = [torch.randn((b, L, n, d), generator=g).to(TYPES[dtype]).cuda() for n in (h, kv, kv, h)]
    if layout == "heads":
        out = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in out]
    if layout == "sliced":
        out = [torch.nn.functional.pad(x.flatten(2), (16, 24))[..., 16:-24].unflatten(-1, (-1, d)) for x in out]
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("w,n,layout", [(9, 1, "sliced"), (40, 3, "heads"), (1, 2, "dense"), (129, 0, "sliced"), (33, 70, "heads")])
def test_elements(w, n, layout, d, dtype):
    q, k, v, dy = inputs(len(LENGTHS), 300, 16, 8, d, dtype, layout, 1)
    check(q, k, v, dy, w, n, LENGTHS, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("w,n", [(200, 4), (65, 33), (128, 1), (64, 0)])
def test_weight_on_the_edges_of_what_is_seen(w, n, d, dtype):
    # each query lies along one key, which then holds most of its weight: the oldest of its window, the first sink, the
    # last sink, itself.  A single lost, doubled or misplaced term is an error of the whole row's size
    L, h, kv = 300, 32, 8
    q, k, v, dy = inputs(len(LENGTHS), L, h, kv, d, dtype, "dense", 2)
    t = torch.arange(L, device="cuda")
    first = (t - w + 1).clamp(min=0)
    edges = [first, torch.zeros_like(t) if n else first, torch.minimum(t, torch.full_like(t, n - 1)) if n else first, t]
    for head in range(h):
        q[:, :, head] = k[:, edges[head % 4], head // (h // kv)]
    check(q, k, v, dy, w, n, LENGTHS, dtype)
    check(q, k, v, dy, w, n, [L] * len(LENGTHS), dtype)
