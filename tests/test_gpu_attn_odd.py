"""Sliding-window attention over values that are not finite: each element of a
result has what its row sees and nothing else, and a step that has diverged
takes some times a sound one's time.

The reference is in fp64: sums over the finite values, and beside them what of
infinities and NaN a row sees.  Weights of seen tokens are above 0 there (scores
are of order 1).  Bounds as in test_gpu_attn.py.
"""
from __future__ import annotations

import math
import statistics

import pytest
import torch

import mamba_chunked_ssd_amd as ssd

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f32": 0.0}
INF, NAN = math.inf, math.nan


def inputs(b, L, h, kv, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * L + d)
    return [torch.randn((b, L, n, d), generator=g).to(TYPES[dtype]).cuda() for n in (h, kv, kv, h)]


def seen_by(first, L, w, n):
    """(query, token) of a sequence with `first` tokens behind it."""
    t = first + torch.arange(L, device="cuda")[:, None]
    j = torch.arange(first + L, device="cuda")[None]
    return (j <= t) & ((t - j < w) | (j < n))


def spread(q, k, scale, tokens):
    """E of test_gpu_attn.py."""
    d = q.shape[-1]
    q, k = (x.double().nan_to_num(0, 0, 0).abs().flatten(0, -2).amax(0) for x in (q, k))
    return (2 * (d + 8) * scale * float(q @ k) + 2 * tokens + 32) * EPS


def apart(p, x):
    """p @ x where x may hold anything: p above 0 where it counts."""
    plus, minus, none = (x == INF).double(), (x == -INF).double(), x.isnan().double()
    on = (p > 0).double()
    plus, minus, none = ((on @ z) > 0 for z in (plus, minus, none))
    y = p @ x.nan_to_num(0, 0, 0)
    y = torch.where(plus, INF, y)
    y = torch.where(minus, -INF, y)
    return torch.where(none | (plus & minus), NAN, y)


def same(got, want, bound):
    got = got.double()
    odd = ~want.isfinite()
    return torch.equal(got.isnan(), want.isnan()) and torch.equal(got == INF, want == INF) and \
        torch.equal(got == -INF, want == -INF) and bool(((got - want).abs() <= bound)[~odd].all())


# one block of queries and many; sequences whose windows end inside tiles
@pytest.mark.parametrize("b", [1, 34])
@pytest.mark.parametrize("d,dtype", [(32, "bf16"), (64, "bf16"), (128, "bf16"), (32, "f32"), (64, "f32"), (128, "f32")])
@pytest.mark.parametrize("w,n", [(20, 3), (75, 0), (1000, 0), (33, 40)])
def test_forward_has_what_it_sees(b, d, dtype, w, n):
    L, h, kv = 260, 4, 2
    q, k, v, _ = inputs(b, L, h, kv, d, dtype)
    for at, kind in ((1, INF), (34, -INF), (100, NAN), (130, INF), (131, -INF), (200, INF), (259, NAN)):
        v[:, at, :, at % 7::5] = kind
    y = ssd.window_attention_fwd(q, k, v, w, n)
    on = seen_by(0, L, w, n)
    kk, vv = (x.double().repeat_interleave(h // kv, 2).transpose(1, 2) for x in (k, v))
    z = (q.double().transpose(1, 2) @ kk.transpose(2, 3).contiguous() * d ** -0.5).masked_fill(~on, -INF)
    p = torch.softmax(z, -1)
    want, mag = apart(p, vv), p @ vv.nan_to_num(0, 0, 0).abs()
    e, r = spread(q, k, d ** -0.5, min(w, L) + n), ROUND[dtype]
    assert same(y.transpose(1, 2), want, (e + r) * mag + r * want.abs())


@pytest.mark.parametrize("b", [3, 48])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "f32")])
@pytest.mark.parametrize("w,n", [(20, 3), (75, 0), (33, 40)])
def test_forward_from_a_cache(b, d, dtype, w, n):
    first, L, h, kv = 150, 150, 4, 2
    q, k, v, _ = inputs(b, first + L, h, kv, d, dtype, 1)
    for at, kind in ((2, INF), (30, NAN), (120, -INF), (149, NAN), (151, INF), (152, -INF), (290, INF)):
        v[:, at, :, at % 7::5] = kind
    kc, vc = (torch.zeros((b, kv, w + n, d), dtype=TYPES[dtype], device="cuda") for _ in range(2))
    ssd.window_attention_fwd(q[:, :first], k[:, :first], v[:, :first], w, n, k_cache=kc, v_cache=vc)
    at = torch.full((b,), first, dtype=torch.int32, device="cuda")
    y = ssd.window_attention_fwd(q[:, first:], k[:, first:], v[:, first:], w, n, positions=at, k_cache=kc, v_cache=vc)
    on = seen_by(first, L, w, n)
    kk, vv = (x.double().repeat_interleave(h // kv, 2).transpose(1, 2) for x in (k, v))
    z = (q[:, first:].double().transpose(1, 2) @ kk.transpose(2, 3).contiguous() * d ** -0.5).masked_fill(~on, -INF)
    p = torch.softmax(z, -1)
    want, mag = apart(p, vv), p @ vv.nan_to_num(0, 0, 0).abs()
    e, r = spread(q, k, d ** -0.5, w + n), ROUND[dtype]
    assert same(y.transpose(1, 2), want, (e + r) * mag + r * want.abs())


# one block for a cache and several; several tokens, so that the cache's own odd values and new ones are met
@pytest.mark.parametrize("b,h,kv,d,dtype,w,n", [(3, 4, 2, 64, "bf16", 40, 3), (2, 8, 8, 128, "bf16", 300, 0), (4, 40, 1, 32, "bf16", 90, 2),
                                                (1, 8, 2, 64, "bf16", 6000, 4), (3, 6, 2, 64, "f32", 50, 3), (1, 4, 2, 128, "f32", 3000, 4)])
def test_step_has_what_it_sees(b, h, kv, d, dtype, w, n):
    q, k, v, _ = inputs(b, w + n + 4, h, kv, d, dtype, 3)
    for at, kind in ((0, INF), (1, -INF), (w // 2, NAN), (w // 2 + 1, INF), (w + n - 1, -INF), (w + n + 1, INF), (w + n + 2, NAN)):
        v[:, at, :, at % 7::9] = kind
    kc, vc = (torch.zeros((b, kv, w + n, d), dtype=TYPES[dtype], device="cuda") for _ in range(2))
    ssd.window_attention_fwd(q[:, :-4], k[:, :-4], v[:, :-4], w, n, k_cache=kc, v_cache=vc)
    pos = torch.full((b,), w + n, dtype=torch.int32, device="cuda")
    e, r = spread(q, k, d ** -0.5, w + n), ROUND[dtype]
    for t in range(w + n, w + n + 4):
        y = ssd.window_attention_step(q[:, t], k[:, t], v[:, t], kc, vc, pos, w, n)
        pos += 1
        kk, vv = (x.double().repeat_interleave(h // kv, 1) for x in (kc, vc))
        p = torch.softmax((kk * q[:, t].double()[:, :, None]).sum(-1) * d ** -0.5, -1)[:, :, None]
        want, mag = apart(p, vv)[:, :, 0], (p @ vv.nan_to_num(0, 0, 0).abs())[:, :, 0]
        assert same(y, want, (e + r) * mag + r * want.abs())


def took(call):
    for _ in range(2):
        call()
    times = []
    for _ in range(3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return statistics.median(times)


# everything is not finite, or one sink that every query sees
ODD = [("all", slice(None), NAN), ("all", slice(None), INF), ("sink", slice(1, 2), NAN), ("sink", slice(1, 2), INF)]


@pytest.mark.parametrize("L,h,kv,d,dtype", [(4096, 32, 8, 64, "bf16"), (8192, 16, 4, 128, "bf16"), (4096, 16, 8, 64, "f32")])
@pytest.mark.parametrize("where", ODD, ids=lambda o: "%s_%s" % (o[0], o[2]))
def test_a_diverged_forward_takes_some_times_a_sound_one(L, h, kv, d, dtype, where):
    q, k, v, _ = inputs(1, L, h, kv, d, dtype)
    sound = took(lambda: ssd.window_attention_fwd(q, k, v, 512, 4))
    v[:, where[1]] = where[2]
    assert took(lambda: ssd.window_attention_fwd(q, k, v, 512, 4)) <= 20 * sound


def terms(q, k, v, dy, on, scale, g):
    """P, and the gradients with their terms' magnitudes, in fp64; heads first.  What is not finite in dy, v counts as 0."""
    q, dy = (x.double().transpose(1, 2) for x in (q, dy.nan_to_num(0, 0, 0)))
    k, v = (x.double().repeat_interleave(g, 2).transpose(1, 2) for x in (k, v.nan_to_num(0, 0, 0)))
    across = lambda x: x.transpose(2, 3).contiguous()  # noqa: E731
    p = torch.softmax((q @ across(k) * scale).masked_fill(~on, -INF), -1)
    dp, part = dy @ across(v), dy.abs() @ across(v.abs())
    ds = scale * p * (dp - (p * dp).sum(-1, keepdim=True))
    dsm = scale * p * (part + (p * part).sum(-1, keepdim=True))
    share = lambda x: x.unflatten(1, (-1, g)).sum(2)  # noqa: E731
    return p, dict(dq=ds @ k, dk=share(across(ds) @ q), dv=share(across(p) @ dy)), \
        dict(dq=dsm @ k.abs(), dk=share(across(dsm) @ q.abs()), dv=share(across(p) @ dy.abs()))


KINDS = ((1, INF), (34, -INF), (100, NAN), (130, INF), (131, -INF), (200, INF), (259, NAN))


# few blocks and many
@pytest.mark.parametrize("b", [1, 34])
@pytest.mark.parametrize("d,dtype", [(32, "bf16"), (64, "bf16"), (128, "bf16"), (32, "f32"), (64, "f32"), (128, "f32")])
@pytest.mark.parametrize("w,n", [(20, 3), (75, 0), (33, 40)])
@pytest.mark.parametrize("which", ["dy", "v", "k", "q"])
def test_backward_has_what_it_sees(which, b, d, dtype, w, n):
    L, h, kv = 260, 4, 2
    z = dict(zip(("q", "k", "v", "dy"), inputs(b, L, h, kv, d, dtype, 2)))
    clean = {x: t.clone() for x, t in z.items()}
    for at, kind in KINDS[3:] if which in "kq" else KINDS:
        z[which][:, at, :, at % 7::5] = kind
    y, lse = ssd.window_attention_fwd(z["q"], z["k"], z["v"], w, n, return_lse=True)
    got = ssd.window_attention_bwd(z["q"], z["k"], z["v"], y, lse, z["dy"], w, n)
    on = seen_by(0, L, w, n)
    held = clean if which in "kq" else z
    p, ref, mag = terms(held["q"], held["k"], held["v"], held["dy"], on, d ** -0.5, h // kv)
    odd = torch.zeros(L, dtype=torch.bool, device="cuda")
    odd[[at for at, _ in (KINDS[3:] if which in "kq" else KINDS)]] = True
    rows = (on & odd).any(1) if which in "kv" else odd  # queries whose weights or dP are not finite
    keys = (on & rows[:, None]).any(0)  # keys that such a query sees
    e, r = spread(clean["q"], clean["k"], d ** -0.5, min(w, L) + n), ROUND[dtype]
    for name in ref:
        out = got[name].transpose(1, 2).double()
        m = 1 if name == "dv" else 4
        bound = m * (e + r) * mag[name] + (r + EPS) * ref[name].abs()
        if name == "dv" and which in ("dy", "v"):
            # P is sound: each element has the kinds that its key sees, and no others
            want = ref[name]
            if which == "dy":
                both = apart(p.transpose(2, 3).contiguous(), z["dy"].double().transpose(1, 2)).unflatten(1, (kv, -1)).sum(2)
                want = torch.where(both.isfinite(), want, both)
            assert same(out, want, bound)
            continue
        sel = ~(rows if name == "dq" else keys)
        assert bool(sel.any()) or name != "dq"
        assert bool(((out - ref[name]).abs() <= bound)[:, :, sel].all()), name
        # and the others are as far from sound as the input is
        assert not bool(out[:, :, ~sel].isfinite().all()), name


@pytest.mark.parametrize("L,h,kv,d,dtype", [(4096, 32, 8, 64, "bf16"), (4096, 16, 4, 128, "bf16"), (2048, 16, 8, 64, "f32"), (1024, 4, 1, 128, "bf16")])
@pytest.mark.parametrize("which", ["q", "k", "v", "dy"])
@pytest.mark.parametrize("where", [ODD[0], ODD[3]], ids=lambda o: "%s_%s" % (o[0], o[2]))
def test_a_diverged_backward_takes_some_times_a_sound_one(L, h, kv, d, dtype, which, where):
    z = dict(zip(("q", "k", "v", "dy"), inputs(1, L, h, kv, d, dtype)))

    def time():
        y, lse = ssd.window_attention_fwd(z["q"], z["k"], z["v"], 512, 4, return_lse=True)
        return took(lambda: ssd.window_attention_bwd(z["q"], z["k"], z["v"], y, lse, z["dy"], 512, 4))

    sound = time()
    z[which][:, where[1]] = where[2]
    assert time() <= 40 * sound
