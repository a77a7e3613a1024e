"""Parity of sliding-window attention with sinks (ssd_window_attn_fwd, _bwd,
_step) against the fp64 oracle and, at larger sizes, its definition in fp64
torch.

Bounds.  EPS = 2^-24, R = 2^-8 (half a step of bf16) for bf16 and 0 for fp32.
Inputs are exact.  A score is a sum of D products in fp32, off by (D + 4) EPS A,
A the largest scale sum |q||k|; the exponent adds 4 EPS A.  So a weight is off by
2 (D + 8) EPS A relatively (itself and the sum it is divided by), the sum of n
weights by n EPS, exponential, quotient and the rest by 32 EPS: E = (2 (D + 8) A
+ 2 n + 32) EPS.  As an operand of the second product it is rounded by R.
  y:  (E + R) sum p |v|, and R |y| for its own rounding.
  lse: (2 (D + 8) A + n + 8) EPS + 4 EPS |lse|.
  delta is dy . y of the rounded y: E + 2 R of sum p (|dy| . |v|), dS another E,
  its rounding R: dq and dk are within (4 E + 4 R) of the sums of their terms'
  magnitudes (parts of dP - delta separately), dv within E + R, each and R of
  itself.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import mamba_chunked_ssd_amd as ssd
from oracle import mixer_ops as mo

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f32": 0.0}


def host(t):
    return None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def inputs(b, L, h, kv, d, dtype="f32", layout="dense", lengths=None, cache=None, positions=None, seed=0, size=1.0):
    g = torch.Generator().manual_seed(1000 * seed + 7 * L + h + d)
    t = TYPES[dtype]
    q, k, v, dy = (size * torch.randn((b, L, n, d), generator=g) for n in (h, kv, kv, h))
    s = {}
    if layout == "sliced":
        wide = torch.full((b, L, (2 * h + 2 * kv) * d + 64), float("nan")).to(t).cuda()
        at = 16
        for name, x in (("q", q), ("k", k), ("v", v), ("dy", dy)):
            n = x.shape[2] * d
            wide[..., at:at + n] = x.flatten(2).to(t)
            s[name] = wide[..., at:at + n].unflatten(-1, (-1, d))
            at += n
    else:
        for name, x in (("q", q), ("k", k), ("v", v), ("dy", dy)):
            s[name] = x.to(t).cuda()
            if layout == "turned":  # (seqlen, batch, ..) storage
                s[name] = s[name].transpose(0, 1).contiguous().transpose(0, 1)
            if layout == "heads":  # (batch, heads, seqlen, ..) storage
                s[name] = s[name].transpose(1, 2).contiguous().transpose(1, 2)
    s["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    s["positions"] = None if positions is None else torch.tensor(positions, dtype=torch.int32, device="cuda")
    if cache is not None:
        s["kc"], s["vc"] = (size * torch.randn((b, kv, cache, d), generator=g).to(t).cuda() for _ in range(2))
    return s


def spread(s, scale, window, sinks, d):
    """E of the bounds above."""
    q, k = s["q"].double().abs(), s["k"].double().abs()
    if "kc" in s:
        k = torch.cat([k.transpose(1, 2).flatten(0, 2), s["kc"].double().abs().flatten(0, 2)])
    a = scale * float(q.flatten(0, -2).amax(0) @ k.reshape(-1, d).amax(0)) if q.numel() else 0.0
    return (2 * (d + 8) * a + 2 * (window + sinks) + 32) * EPS, a


# (b, L, h, kv, d, window, sinks, dtype, layout, lengths): one token, the waves' 32 queries and the blocks' 128, tiles
# of 32 and 64 keys; windows of one, odd ones, longer than the sequence; sinks of none, one, within, beyond and past
# the window; shared heads
CASES = [
    (1, 1, 1, 1, 32, 1, 0, "f32", "dense", None),
    (2, 1, 4, 2, 64, 7, 3, "bf16", "dense", None),
    (1, 33, 2, 1, 64, 1, 0, "f32", "dense", None),
    (2, 40, 3, 3, 32, 5, 2, "f32", "sliced", [40, 17]),
    (1, 65, 4, 1, 128, 16, 1, "bf16", "dense", None),
    (3, 70, 6, 2, 64, 33, 5, "f32", "turned", [70, 0, 33]),
    (1, 129, 2, 2, 32, 500, 0, "f32", "dense", None),
    (2, 130, 5, 1, 64, 64, 64, "bf16", "sliced", [130, 129]),
    (1, 150, 2, 1, 128, 20, 9, "f32", "dense", None),
    (1, 200, 1, 1, 32, 10, 150, "f32", "heads", None),
    (2, 140, 6, 3, 64, 3, 40, "bf16", "heads", [140, 1]),
    (1, 260, 2, 1, 32, 128, 4, "f32", "sliced", None),
]


def ids(c):
    return "b%d_L%d_h%d_kv%d_d%d_w%d_s%d_%s_%s%s" % (c[:9] + ("_ragged" * (c[9] is not None),))


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward(case):
    b, L, h, kv, d, w, n, dtype, layout, lengths = case
    s = inputs(b, L, h, kv, d, dtype, layout, lengths)
    y, lse = ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n, lengths=s["lengths"], return_lse=True)
    torch.cuda.synchronize()
    ref, rlse, mag = mo.attention(host(s["q"]), host(s["k"]), host(s["v"]), w, n, lengths=host(s["lengths"]))
    e, a = spread(s, d ** -0.5, min(w, L), n, d)
    r = ROUND[dtype]
    assert y.dtype == TYPES[dtype]
    assert np.all(np.abs(host(y) - ref) <= (e + r) * mag + r * np.abs(ref))
    assert np.all(np.abs(host(lse) - rlse) <= ((2 * (d + 8) * a + L + 8) + 4 * np.abs(rlse)) * EPS * (rlse != 0))


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_backward(case):
    b, L, h, kv, d, w, n, dtype, layout, lengths = case
    s = inputs(b, L, h, kv, d, dtype, layout, lengths)
    y, lse = ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n, lengths=s["lengths"], return_lse=True)
    if layout == "heads":
        y = y.transpose(1, 2).contiguous().transpose(1, 2)
    got = ssd.window_attention_bwd(s["q"], s["k"], s["v"], y, lse, s["dy"], w, n, lengths=s["lengths"])
    torch.cuda.synchronize()
    ref, mag = mo.attention_bwd(*[host(s[x]) for x in ("q", "k", "v", "dy")], w, n, lengths=host(s["lengths"]))
    e, _ = spread(s, d ** -0.5, min(w, L), n, d)
    r = ROUND[dtype]
    for name in ref:
        m = 1 if name == "dv" else 4
        assert got[name].dtype == TYPES[dtype]
        assert np.all(np.abs(host(got[name]) - ref[name]) <= m * (e + r) * mag[name] + (r + EPS) * np.abs(ref[name])), name


def dense(s, w, n, scale):
    """The definition over all pairs in fp64, differentiable; y, lse, sum p |v|."""
    q, k, v = s
    b, L, h, d = q.shape
    g = h // k.shape[2]
    k, v = (x.repeat_interleave(g, 2).transpose(1, 2) for x in (k, v))
    t = torch.arange(L, device=q.device)
    back = t[:, None] - t[None, :]
    seen = (back >= 0) & ((back < w) | (t[None, :] < n))
    z = (q.transpose(1, 2) @ k.transpose(2, 3) * scale).masked_fill(~seen, -math.inf)
    p = torch.softmax(z, -1)
    return (p @ v).transpose(1, 2), torch.logsumexp(z, -1), (p @ v.abs()).transpose(1, 2)


# larger ones: many tiles of a window, sinks in two tiles, several chunks of far queries
LARGE = [
    (1, 1500, 2, 1, 64, 300, 4, "f32", 0.25),
    (2, 1100, 4, 2, 128, 257, 70, "bf16", None),
    (1, 1801, 3, 1, 32, 64, 140, "f32", None),
    (1, 900, 2, 2, 128, 10000, 0, "f32", 0.01),
    (1, 2000, 2, 1, 64, 700, 1, "bf16", 0.3),
]


@pytest.mark.parametrize("case", LARGE, ids=lambda c: "b%d_L%d_h%d_kv%d_d%d_w%d_s%d_%s" % c[:8])
def test_larger_sizes(case):
    b, L, h, kv, d, w, n, dtype, scale = case
    s = inputs(b, L, h, kv, d, dtype, seed=3)
    y, lse = ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n, scale=scale, return_lse=True)
    got = ssd.window_attention_bwd(s["q"], s["k"], s["v"], y, lse, s["dy"], w, n, scale=scale)
    scale = d ** -0.5 if scale is None else scale
    x = [s[m].double().requires_grad_() for m in "qkv"]
    ref, rlse, mag = dense(x, w, n, scale)
    (ref * s["dy"].double()).sum().backward()
    e, a = spread(s, scale, min(w, L), n, d)
    r = ROUND[dtype]
    assert bool(((y.double() - ref).abs() <= (e + r) * mag + r * ref.abs()).all())
    assert bool(((lse.double() - rlse).abs() <= (2 * (d + 8) * a + L + 8 + 4 * rlse.abs()) * EPS).all())
    # the sums' magnitudes, by the square root of n against n terms: 2-norms within the operands' roundings
    for name, z in zip(("dq", "dk", "dv"), x):
        off = float((got[name].double() - z.grad).norm() / z.grad.norm())
        assert off <= (4 * r if r else 2e-6), (name, off)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_queries_that_see_one_token_alone(dtype):
    # their weight is 1 whatever the score: dq of token 0 is 0, and with a window of one and no sinks all of dq and dk
    for d in (32, 64, 128):
        s = inputs(2, 150, 4, 2, d, dtype, lengths=[150, 40], seed=12)
        for w, n in ((1, 0), (1, 1), (30, 0)):
            y, lse = ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n, lengths=s["lengths"], return_lse=True)
            g = ssd.window_attention_bwd(s["q"], s["k"], s["v"], y, lse, s["dy"], w, n, lengths=s["lengths"])
            assert not bool(g["dq"][:, 0].any())
            if (w, n) == (1, 0):
                assert not bool(g["dq"].any()) and not bool(g["dk"].any())
                # (the exponential of a score less its own rounded product is 1 within E)
                v, (e, _) = s["v"][0].repeat_interleave(2, 1).double(), spread(s, d ** -0.5, w, n, d)
                assert bool(((y[0].double() - v).abs() <= (e + 2 * ROUND[dtype]) * v.abs()).all())


# enough blocks of 128 queries, and of 128 keys, that none of the kernels for few is taken
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("h,kv,w,n,layout", [(8, 8, 40, 3, "sliced"), (24, 8, 200, 70, "dense"), (8, 8, 1, 0, "heads"),
                                             (8, 8, 129, 0, "turned"), (16, 8, 9, 1, "dense")])
def test_many_blocks(h, kv, w, n, layout, d, dtype):
    b, L = 9, 300
    lengths = [300, 0, 1, 299, 129, 128, 127, 33, 200]
    s = inputs(b, L, h, kv, d, dtype, layout, lengths, seed=14)
    y, lse = ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n, lengths=s["lengths"], return_lse=True)
    got = ssd.window_attention_bwd(s["q"], s["k"], s["v"], y, lse, s["dy"], w, n, lengths=s["lengths"])
    x = [s[m].double().nan_to_num().requires_grad_() for m in "qkv"]
    ref, rlse, mag = dense(x, w, n, d ** -0.5)
    on = (torch.arange(L, device="cuda")[None, :] < s["lengths"][:, None])[..., None, None]
    (torch.where(on, ref, 0) * s["dy"].double()).sum().backward()
    e, a = spread(s, d ** -0.5, w, n, d)
    r = ROUND[dtype]
    assert bool(((y.double() - torch.where(on, ref, 0)).abs() <= (e + r) * mag * on + r * ref.abs() * on).all())
    live = on[..., 0].transpose(1, 2)
    assert bool(((lse.double() - torch.where(live, rlse, 0)).abs() <= live * (2 * (d + 8) * a + L + 8 + 4 * rlse.abs()) * EPS).all())
    for name, z in zip(("dq", "dk", "dv"), x):
        if (w, n) == (1, 0) and name != "dv":
            assert not bool(got[name].any())
            continue
        # 2-norms, whose errors average: the operands' roundings (a few short windows: no more than four of them)
        off = float((got[name].double() - z.grad).norm() / z.grad.norm())
        assert off <= (4 * r if r else 4e-6), (name, off)
        for i, end in enumerate(lengths):
            assert not bool(got[name][i, end:].any())


@pytest.mark.parametrize("d,dtype", [(32, "f32"), (64, "bf16"), (128, "bf16"), (128, "f32")])
@pytest.mark.parametrize("w,n,positions", [(16, 4, [0, 3, 17, 500]), (100, 0, [64, 99, 100, 333]), (33, 80, [10, 81, 200, 0])])
def test_many_blocks_with_a_past(w, n, positions, d, dtype):
    # the same four sequences once (few blocks) and twelve times (many): every copy gives the same
    L, h, kv = 200, 4, 2
    s = inputs(4, L, h, kv, d, dtype, "dense", [200, 131, 0, 64], w + n, positions, seed=15)
    many = {k: v.repeat(12, *[1] * (v.dim() - 1)) for k, v in s.items()}

    def call(z):
        y, lse = ssd.window_attention_fwd(z["q"], z["k"], z["v"], w, n, lengths=z["lengths"], positions=z["positions"],
                                          k_cache=z["kc"], v_cache=z["vc"], return_lse=True)
        return y, lse, z["kc"], z["vc"]

    few, all_ = call(s), call(many)
    e, _ = spread(s, d ** -0.5, w, n, d)
    most = max(1.0, float(s["vc"].abs().max()), float(s["v"].abs().max()))
    for k, (p, q) in enumerate(zip(few, all_)):
        q = q.unflatten(0, (12, 4))
        assert all(torch.equal(q[0], c) for c in q[1:])
        if k >= 2:
            assert torch.equal(q[0], p)
        else:  # two calculations, each within its bound
            assert float((q[0].double() - p.double()).abs().max()) <= 2 * (e + 2 * ROUND[dtype]) * (most if k == 0 else 20)


# (b, L, h, kv, d, window, sinks, dtype, lengths, positions): nothing behind, less than the sinks, than the window, a
# ring that has turned, one far along; new tokens that fill the sinks, that overrun the whole ring
PAST = [
    (4, 5, 2, 1, 64, 9, 3, "f32", None, [0, 2, 7, 1000]),
    (3, 40, 4, 2, 32, 16, 4, "f32", [40, 39, 0], [3, 17, 50]),
    (3, 70, 3, 1, 128, 100, 0, "bf16", None, [0, 64, 333]),
    (2, 1, 2, 2, 64, 40, 70, "f32", None, [5, 200]),
    (2, 150, 2, 1, 64, 33, 80, "bf16", [150, 7], [10, 81]),
    (3, 200, 1, 1, 32, 64, 64, "f32", None, [-5, 63, 64]),
]


@pytest.mark.parametrize("case", PAST, ids=lambda c: "b%d_L%d_h%d_kv%d_d%d_w%d_s%d_%s" % c[:8])
def test_prompts_with_a_past(case):
    b, L, h, kv, d, w, n, dtype, lengths, positions = case
    s = inputs(b, L, h, kv, d, dtype, "sliced", lengths, w + n, positions)
    kc, vc = s["kc"].clone(), s["vc"].clone()
    # slots that no token has reached hold anything
    for i, p in enumerate(positions):
        kc[i, :, max(p, 0):] = float("nan")
        vc[i, :, max(p, 0):] = float("nan")
    got = [kc.clone(), vc.clone()]
    y, lse = ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n, lengths=s["lengths"], positions=s["positions"],
                                      k_cache=got[0], v_cache=got[1], return_lse=True)
    torch.cuda.synchronize()
    ref, rlse, mag = mo.attention(host(s["q"]), host(s["k"]), host(s["v"]), w, n, lengths=host(s["lengths"]),
                                  positions=positions, kc=host(s["kc"]), vc=host(s["vc"]))
    e, a = spread(s, d ** -0.5, w, n, d)
    r = ROUND[dtype]
    assert np.all(np.abs(host(y) - ref) <= (e + r) * mag + r * np.abs(ref))
    assert np.all(np.abs(host(lse) - rlse) <= ((2 * (d + 8) * a + w + n + 8) + 4 * np.abs(rlse)) * EPS * (rlse != 0))
    want = mo.cache_after(host(kc), host(vc), host(s["k"]), host(s["v"]), w, n, host(s["lengths"]), positions)
    assert all(np.array_equal(host(x), z, equal_nan=True) for x, z in zip(got, want))


@pytest.mark.parametrize("h,kv,d,dtype", [(4, 2, 64, "f32"), (6, 1, 128, "bf16"), (40, 1, 32, "f32"), (2, 2, 128, "f32")])
@pytest.mark.parametrize("w,n", [(1, 0), (5, 2), (33, 4), (300, 0), (16, 40)])
def test_steps(h, kv, d, dtype, w, n):
    b = 4
    positions = [0, n, w + n + 3, -1]
    s = inputs(b, 3, h, kv, d, dtype, "sliced", None, w + n, positions, seed=1)
    kc, vc = s["kc"].clone(), s["vc"].clone()
    for i, p in enumerate(positions):
        kc[i, :, max(p, 0):] = float("nan")
        vc[i, :, max(p, 0):] = float("nan")
    at = s["positions"].clone()
    e, _ = spread(s, d ** -0.5, w, n, d)
    r = ROUND[dtype]
    for t in range(3):
        q, k, v = (s[x][:, t] for x in "qkv")
        before = host(kc), host(vc)
        y = ssd.window_attention_step(q, k, v, kc, vc, at, w, n)
        torch.cuda.synchronize()
        ref, _, mag = mo.attention(host(q)[:3, None], host(k)[:3, None], host(v)[:3, None], w, n, positions=host(at)[:3],
                                   kc=np.nan_to_num(before[0])[:3], vc=np.nan_to_num(before[1])[:3])
        assert np.all(np.abs(host(y)[:3] - ref[:, 0]) <= (e + r) * mag[:, 0] + r * np.abs(ref[:, 0]))
        assert not bool(y[3].any())  # an empty place of the batch
        want = mo.cache_after(*[x[:3] for x in before], host(k)[:3, None], host(v)[:3, None], w, n, None, host(at)[:3])
        for x, z, old in zip((kc, vc), want, before):
            assert np.array_equal(host(x)[:3], z, equal_nan=True) and np.array_equal(host(x)[3], old[3], equal_nan=True)
        at += 1
        at[3] = -1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("b,h,kv,d,w,n", [(1, 8, 2, 64, 1500, 4), (1, 8, 2, 64, 4000, 4), (3, 4, 4, 128, 1700, 0), (2, 70, 2, 32, 2900, 130)])
def test_steps_over_split_caches(b, h, kv, d, w, n, dtype):
    # few sequences: their slots are split over blocks.  Against the prompts' kernel
    s = inputs(b, 2, h, kv, d, dtype, "dense", None, w + n, [w + n + 5 + i for i in range(b)], seed=2)
    kc, vc, kc2, vc2 = (s[x].clone() for x in ("kc", "vc", "kc", "vc"))
    want = ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n, positions=s["positions"], k_cache=kc2, v_cache=vc2)
    e, _ = spread(s, d ** -0.5, w, n, d)
    for t in range(2):
        y = ssd.window_attention_step(s["q"][:, t], s["k"][:, t], s["v"][:, t], kc, vc, s["positions"] + t, w, n)
        # two calculations, each within its bound; sum p |v| is below max |v|
        most = float(s["vc"].abs().max())
        assert float((y.double() - want[:, t].double()).abs().max()) <= 2 * (e + 2 * ROUND[dtype]) * max(most, 1)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_a_prompt_in_pieces_is_the_prompt():
    b, L, h, kv, d, w, n = 2, 300, 4, 2, 64, 50, 6
    s = inputs(b, L, h, kv, d, "f32", seed=5)
    kc, vc, kw, vw = (torch.zeros((b, kv, w + n, d), device="cuda") for _ in range(4))
    want = ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n, k_cache=kw, v_cache=vw)
    alone = ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n)
    assert torch.equal(alone, want)
    parts, at = [], torch.zeros(b, dtype=torch.int32, device="cuda")
    for t0, t1 in ((0, 1), (1, 4), (4, 130), (130, 131), (131, 299)):
        parts.append(ssd.window_attention_fwd(s["q"][:, t0:t1], s["k"][:, t0:t1], s["v"][:, t0:t1], w, n, positions=at,
                                              k_cache=kc, v_cache=vc))
        at += t1 - t0
    parts.append(ssd.window_attention_step(s["q"][:, 299], s["k"][:, 299], s["v"][:, 299], kc, vc, at, w, n)[:, None])
    e, _ = spread(s, d ** -0.5, w, n, d)
    most = max(1.0, float(s["v"].abs().max()))
    assert float((torch.cat(parts, 1) - want).abs().max()) <= 2 * e * most
    assert torch.equal(kc, kw) and torch.equal(vc, vw)


def test_rows_behind_the_end_are_not_read():
    s = inputs(4, 150, 4, 2, 64, "bf16", "dense", [150, 70, 1, 0], seed=6)
    w, n = 40, 3
    y, lse = ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n, lengths=s["lengths"], return_lse=True)
    g = ssd.window_attention_bwd(s["q"], s["k"], s["v"], y, lse, s["dy"], w, n, lengths=s["lengths"])
    bad = {k: s[k].clone() for k in ("q", "k", "v", "dy")}
    y2, lse2 = y.clone(), lse.clone()
    for i, end in enumerate(s["lengths"].tolist()):
        for k, x in bad.items():
            x[i, end:] = float("nan")
        assert not bool(y[i, end:].any()) and not bool(lse[i, :, end:].any())
        assert all(not bool(g[k][i, end:].any()) for k in g)
        y2[i, end:] = float("inf")
        lse2[i, :, end:] = float("nan")
    got = ssd.window_attention_fwd(bad["q"], bad["k"], bad["v"], w, n, lengths=s["lengths"], return_lse=True)
    ggot = ssd.window_attention_bwd(bad["q"], bad["k"], bad["v"], y2, lse2, bad["dy"], w, n, lengths=s["lengths"])
    assert torch.equal(got[0], y) and torch.equal(got[1], lse)
    assert all(torch.equal(ggot[k], g[k]) for k in g)
    wild = torch.tensor([1 << 30, -5, 150, 151], dtype=torch.int32, device="cuda")
    tame = torch.tensor([150, 0, 150, 150], dtype=torch.int32, device="cuda")
    assert torch.equal(ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n, lengths=wild),
                       ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n, lengths=tame))


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128), ("bf16", 32)])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan"), "largest"])
@pytest.mark.parametrize("which", ["k", "v", "q", "dy"])
@pytest.mark.parametrize("b", [1, 34])  # the kernels for few blocks, and the others
def test_values_not_finite_reach_only_who_sees_them(b, dtype, d, value, which):
    # one token of the sequence holds them; rows that do not see it (and keys that it does not see) are as if it did not
    L, h, kv, w, n, at = 300, 4, 2, 20, 3, 150
    s = inputs(b, L, h, kv, d, dtype, seed=8)
    value = torch.finfo(TYPES[dtype]).max if value == "largest" else value
    clean = {}
    y0, lse0 = ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n, return_lse=True)
    clean = ssd.window_attention_bwd(s["q"], s["k"], s["v"], y0, lse0, s["dy"], w, n)
    s[which][:, at, :, ::3] = value
    y, lse = ssd.window_attention_fwd(s["q"], s["k"], s["v"], w, n, return_lse=True)
    g = ssd.window_attention_bwd(s["q"], s["k"], s["v"], y, lse, s["dy"], w, n)
    t = torch.arange(L, device="cuda")
    rows = (t >= at) & (t - at < w) if which in "kv" else t == at  # queries that the value reaches
    off = (t < at - w + 1) | (t > at)
    keys = (off & (t >= n)) if which in ("q", "dy") else (t < at - 2 * w) & (t >= n) | (t > at + 2 * w)
    e, _ = spread({"q": s["q"].nan_to_num(0, 0, 0).clamp(-9, 9), "k": s["k"].nan_to_num(0, 0, 0).clamp(-9, 9)}, d ** -0.5, w, n, d)
    tol = 8 * (e + ROUND[dtype])
    def near(a, b, sel):
        return bool(((a - b).double().abs() <= tol * (1 + b.double().abs().amax()))[:, sel].all())
    if which != "dy":
        assert near(y, y0, ~rows) and near(lse.transpose(1, 2), lse0.transpose(1, 2), ~rows)
    assert near(g["dq"], clean["dq"], ~rows)
    assert near(g["dk"], clean["dk"], keys) and near(g["dv"], clean["dv"], keys)


def test_large_scores_and_rescaling():
    # scores that rise by hundreds from tile to tile, and fall: the running maximum's reference moves, or stays
    b, L, h, kv, d, w, n = 1, 400, 2, 1, 64, 300, 2
    s = inputs(b, L, h, kv, d, "f32", seed=9)
    for shape in (torch.linspace(0.1, 40, L), torch.linspace(40, 0.1, L), 20 + 20 * torch.sin(torch.arange(L) / 9.0)):
        k = s["k"] * shape.cuda()[None, :, None, None]
        y, lse = ssd.window_attention_fwd(s["q"], k, s["v"], w, n, return_lse=True)
        ref, rlse, mag = dense([s["q"].double(), k.double(), s["v"].double()], w, n, d ** -0.5)
        e, a = spread({"q": s["q"], "k": k}, d ** -0.5, w, n, d)
        assert bool(((y.double() - ref).abs() <= e * mag).all())
        assert bool(((lse.double() - rlse).abs() <= (2 * (d + 8) * a + L + 8 + 4 * rlse.abs()) * EPS).all())


def test_arguments_that_are_no_tensors():
    s = inputs(1, 4, 2, 1, 32)
    for args in ((3.0, s["k"], s["v"]), (s["q"], None, s["v"]), (s["q"], s["k"], 3.0)):
        with pytest.raises(TypeError):
            ssd.window_attention_fwd(*args, 2)
    with pytest.raises(TypeError):
        ssd.window_attention_bwd(s["q"], s["k"], s["v"], None, None, s["dy"], 2)


def test_refusals_leave_the_outputs():
    s = inputs(2, 8, 4, 2, 32, cache=10, positions=[0, 3])
    out = torch.full((2, 8, 4, 32), 7.0, device="cuda")
    call = lambda *a, **k: ssd.window_attention_fwd(*a, out=out, **k)  # noqa: E731
    with pytest.raises(ValueError, match="cache"):
        call(s["q"], s["k"], s["v"], None, 2, k_cache=s["kc"], v_cache=s["vc"])
    with pytest.raises(TypeError):
        call(s["q"], s["k"], s["v"], 8, 2, positions=s["positions"])
    with pytest.raises(ValueError, match="shape"):
        call(s["q"], s["k"], s["v"], 9, 2, k_cache=s["kc"], v_cache=s["vc"])
    for kw in (dict(window=0), dict(window=3, sinks=-1), dict(window=3, scale=0.0), dict(window=3, scale=float("nan"))):
        with pytest.raises(ssd.SSDError, match="INVALID"):
            call(s["q"], s["k"], s["v"], **kw)
    with pytest.raises(ssd.SSDError, match="UNSUPPORTED"):
        ssd.window_attention_fwd(*(torch.zeros((1, 4, 2, 48), device="cuda") for _ in range(3)), 2)
    with pytest.raises(ssd.SSDError, match="INVALID"):
        ssd.window_attention_fwd(s["q"][:, :, :3].contiguous(), s["k"], s["v"], 2)
    with pytest.raises(ssd.SSDError, match="INVALID"):
        ssd.window_attention_fwd(s["q"], s["k"], s["v"], 3, out=s["q"])
    odd = torch.zeros((2, 8, 2 * 32 + 1), device="cuda")[..., 1:].unflatten(-1, (2, 32))
    with pytest.raises(ssd.SSDError, match="MISALIGNED"):
        call(s["q"], odd, s["v"], 3)
    with pytest.raises(TypeError):
        call(s["q"].half(), s["k"], s["v"], 3)
    with pytest.raises(ValueError, match="contiguous"):
        call(s["q"], s["k"], torch.zeros((2, 8, 32, 2), device="cuda").transpose(2, 3), 3)
    with pytest.raises(ssd.SSDError, match="WORKSPACE"):
        ssd.window_attention_bwd(s["q"], s["k"], s["v"], out, torch.zeros((2, 4, 8), device="cuda"), s["dy"], 3, 1,
                                 workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        ssd.window_attention_step(s["q"][:, 0], s["k"][:, 0], s["v"][:, 0], s["kc"], s["vc"], s["positions"], 7, 2)
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())


def test_captured_calls_replay():
    b, L, h, kv, d, w, n = 2, 70, 4, 2, 64, 600, 2
    s = inputs(b, L, h, kv, d, "bf16", "dense", [70, 31], w + n, [0, 900], seed=10)
    held = {k: s[k].clone() for k in ("q", "k", "v", "kc", "vc", "positions")}

    def calls(z):
        y, lse = ssd.window_attention_fwd(z["q"], z["k"], z["v"], 20, n, lengths=s["lengths"], return_lse=True)
        g = ssd.window_attention_bwd(z["q"], z["k"], z["v"], y, lse, s["dy"], 20, n, lengths=s["lengths"])
        p = ssd.window_attention_fwd(z["q"], z["k"], z["v"], w, n, lengths=s["lengths"], positions=z["positions"],
                                     k_cache=z["kc"], v_cache=z["vc"])
        z["positions"] += s["lengths"]
        step = ssd.window_attention_step(z["q"][:, 0], z["k"][:, 0], z["v"][:, 0], z["kc"], z["vc"], z["positions"], w, n)
        return [y, lse, *g.values(), p, step]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls({k: v.clone() for k, v in held.items()})
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(held)
    for k in range(3):
        new = inputs(b, L, h, kv, d, "bf16", cache=w + n, positions=[k, 900], seed=20 + k)
        for name, x in held.items():
            x.copy_(new[name])
        graph.replay()
        torch.cuda.synchronize()
        want = calls(new)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert torch.equal(held["kc"], new["kc"]) and torch.equal(held["positions"], new["positions"])


def test_streams():
    cases = [inputs(2, 300, 4, 2, 64, "bf16", seed=70 + k) for k in range(2)]

    def call(s, **kw):
        y, lse = ssd.window_attention_fwd(s["q"], s["k"], s["v"], 50, 2, return_lse=True, **kw)
        return [y, lse, *ssd.window_attention_bwd(s["q"], s["k"], s["v"], y, lse, s["dy"], 50, 2, **kw).values()]

    want = [call(s) for s in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for k, (s, at) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(at):
                got[k] = call(s)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for g, z in zip(got, want) for p, q in zip(g, z))
    given = call(cases[0], stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(given, want[0]))


def test_offsets_beyond_32_bits():
    # 2.2e9 elements of q, k and v: the last rows against a call on them and the window before them
    L, h, d, w = 540_000, 32, 128, 64
    piece = torch.randn((1, 1000, h, d), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").bfloat16()
    x = piece.repeat(1, L // 1000, 1, 1)
    y, lse = ssd.window_attention_fwd(x, x, x, w, return_lse=True)
    tail = 128 * 8 + L % 128
    cut = x[:, -tail - 128:]
    y1, lse1 = ssd.window_attention_fwd(cut, cut, cut, w, return_lse=True)
    assert torch.equal(y[:, -tail:], y1[:, -tail:])
    g = ssd.window_attention_bwd(x, x, x, y, lse, x, w)
    g1 = ssd.window_attention_bwd(cut, cut, cut, y1, lse1, cut, w)
    assert all(torch.equal(g[k][:, -tail:], g1[k][:, -tail:]) for k in g)


def test_a_long_cache():
    # a cache of 2.2e9 elements: the last sequence's and head's slots lie beyond 32-bit offsets
    b, kv, d, w, n = 3, 4, 128, 1_400_000, 8
    s = inputs(b, 1, 4, kv, d, "bf16", seed=11)
    kc, vc = (torch.zeros((b, kv, w + n, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(1)
    few = 3000
    kc[:, :, :few] = torch.randn((b, kv, few, d), generator=gen, device="cuda").bfloat16()
    vc[:, :, :few] = torch.randn((b, kv, few, d), generator=gen, device="cuda").bfloat16()
    at = torch.tensor([10, 2000, few], dtype=torch.int32, device="cuda")
    small_k, small_v = kc[:, :, :few + 8].clone(), vc[:, :, :few + 8].clone()
    y = ssd.window_attention_step(s["q"][:, 0], s["k"][:, 0], s["v"][:, 0], kc, vc, at, w, n)
    want = ssd.window_attention_step(s["q"][:, 0], s["k"][:, 0], s["v"][:, 0], small_k, small_v, at, few, n)
    assert float((y.float() - want.float()).abs().max()) <= 4 * 2.0 ** -8 * float(vc[:, :, :few].abs().max())
    assert torch.equal(kc[:, :, :few + 8], small_k) and torch.equal(vc[:, :, :few + 8], small_v)
    # the ring's last slot
    at.fill_(w + n - 1)
    ssd.window_attention_step(s["q"][:, 0], s["k"][:, 0], s["v"][:, 0], kc, vc, at, w, n)
    assert torch.equal(kc[:, :, -1], s["k"][:, 0]) and torch.equal(vc[:, :, -1], s["v"][:, 0])
