"""Parity of the short causal convolution (ssd_causal_conv_fwd, _bwd, _step)
against the fp64 oracle.

Bounds.  Inputs are exact in fp64.  A sum of W + 1 terms in fp32 is off by at
most (W + 1) 2^-24 S, S the sum of the terms' magnitudes (>= |p|).  The
logistic function takes an exponent rounded to |p| 2^-23 (log2(e) p; two
roundings) and three instructions of one ulp: y is off by less than
(p^2 s (1 - s) 2 + 6 |y|) 2^-24 <= (1 + 6 S) 2^-24 more, and silu's slope is
at most 1.1, so 2^-24 (1.1 (W + 1) S + 6 S + 1) < 2^-24 * 16 (S + 1) for
W <= 4.  A bf16 result adds half a step, 2^-8 |y|.  The gradients go through
silu' (bounded by 1.1, its own slope by 0.5) likewise, then at most W more
terms; the sums over tokens add up to (tokens of a strip + its block's)
roundings, below 400 here: both are held to 2^-24 times the sum of the terms'
magnitudes, itself times 400.
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import mamba_chunked_ssd_amd as ssd
from oracle import layer_ops as lo

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(b, L, c, W, dtype, sliced=False, state=True, ragged=False, seed=0):
    g = torch.Generator().manual_seed(1000 * seed + 7 * L + c + W)
    t = TYPES[dtype]

    def rows(*shape):
        if not sliced:
            return torch.randn(shape, generator=g).to(t).cuda()
        wide = torch.randn(shape[:-1] + (shape[-1] + 24,), generator=g).to(t).cuda()
        return wide[..., 8:8 + shape[-1]]

    d = dict(x=rows(b, L, c), weight=torch.randn((c, W), generator=g).cuda(), bias=torch.randn(c, generator=g).cuda())
    d["init"] = torch.randn((b, W - 1, c), generator=g).to(t).cuda() if state else None
    d["lengths"] = None
    if ragged:
        d["lengths"] = torch.randint(0, L + 1, (b,), generator=g, dtype=torch.int32).cuda()
        d["lengths"][-1] = 0
        if b > 1:
            d["lengths"][0] = L
    d["dy"] = torch.randn((b, L, c), generator=g).cuda()
    d["dfinal"] = torch.randn((b, W - 1, c), generator=g).cuda() if state else None
    return d


def host(t):
    return None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def half_step(dtype, ref):
    return 2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0


# (b, L, c, W, dtype, out, act, sliced, state, ragged): lengths around the taps, the tokens of a thread (16) and its
# strip of the backward pass; channel counts of one, odd, one vector and several blocks
CASES = [
    (1, 1, 1, 4, "f32", "f32", "silu", False, False, False),
    (2, 2, 5, 4, "bf16", "bf16", "silu", False, True, False),
    (1, 3, 8, 4, "bf16", "f32", None, False, True, False),
    (3, 15, 64, 2, "bf16", "bf16", "silu", True, True, True),
    (2, 16, 264, 3, "f32", "f32", "silu", False, True, False),
    (4, 17, 72, 4, "f32", "f32", None, True, False, True),
    (2, 33, 771, 4, "bf16", "bf16", "silu", False, True, True),
    (2, 129, 40, 2, "bf16", "f32", "silu", True, True, False),
    (5, 150, 520, 4, "bf16", "bf16", "silu", True, True, True),
    (1, 300, 12, 3, "f32", "f32", "silu", False, False, False),
    (3, 0, 16, 4, "bf16", "bf16", "silu", False, True, False),
]


def ids(c):
    return "b%d_L%d_c%d_w%d_%s_%s_%s%s%s%s" % (c[:7] + ("_sliced" * c[7], "_state" * c[8], "_ragged" * c[9]))


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward(case):
    b, L, c, W, dtype, out, act, sliced, state, ragged = case
    d = inputs(b, L, c, W, dtype, sliced, state, ragged)
    y, fin = ssd.causal_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], True, activation=act,
                                 lengths=d["lengths"], y_dtype=TYPES[out])
    torch.cuda.synchronize()
    args = [host(d[k]) for k in ("x", "weight", "bias", "init", "lengths")]
    ref, rfin = lo.conv(*args, act=act is not None)
    mag = lo.conv_magnitude(*args)
    assert np.all(np.abs(host(y) - ref) <= 16 * EPS * (mag + 1) * (ref != 0) + half_step(out, ref))
    assert np.array_equal(host(fin), rfin)  # copies


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_backward(case):
    b, L, c, W, dtype, out, act, sliced, state, ragged = case
    d = inputs(b, L, c, W, dtype, sliced, state, ragged)
    dy = d["dy"].to(TYPES[out])
    dx_dtype = "f32" if out == "f32" else dtype
    got = ssd.causal_conv_bwd(d["x"], d["weight"], d["bias"], dy, d["init"], d["dfinal"], activation=act,
                              lengths=d["lengths"], dx_dtype=TYPES[dx_dtype])
    torch.cuda.synchronize()
    args = [host(d[k]) for k in ("x", "weight", "bias")] + [host(dy)] + [host(d[k]) for k in ("init", "dfinal", "lengths")]
    ref = lo.conv_bwd(*args, act=act is not None)
    # magnitudes: every factor by its absolute value, silu' by what bounds it and its argument's error
    mag = lo.conv_bwd(*[None if a is None else np.abs(a) for a in args], act=False)
    scale = 1 + max(1.0, float(np.max(np.abs(args[0]), initial=0)) * float(np.max(np.abs(args[1]).sum(1))))
    for k, r in ref.items():
        bound = 400 * EPS * scale * mag[k] + half_step(dx_dtype if k == "dx" else "f32", r)
        assert np.all(np.abs(host(got[k]) - r) <= bound), k
    if d["lengths"] is not None:
        for i, end in enumerate(host(d["lengths"])):
            assert not got["dx"][i, end:].any()


@pytest.mark.parametrize("c", [1, 6, 64, 771, 1028])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("W", [2, 4])
def test_steps_are_the_forward_pass(c, dtype, out, W):
    d = inputs(3, 6, c, W, dtype, sliced=True)
    want, wfin = ssd.causal_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], True, y_dtype=TYPES[out])
    state = d["init"].clone()
    for t in range(6):
        y = ssd.causal_conv_step(d["x"][:, t], d["weight"], d["bias"], state, y_dtype=TYPES[out])
        # the same sums in the same order
        assert torch.equal(y, want[:, t])
    assert torch.equal(state, wfin)


def test_prompt_in_pieces_with_the_state_in_place():
    d = inputs(2, 40, 72, 4, "bf16")
    want, wfin = ssd.causal_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], True)
    state = d["init"].clone()
    parts = []
    for t0, t1 in ((0, 1), (1, 3), (3, 20), (20, 40)):
        parts.append(ssd.causal_conv_fwd(d["x"][:, t0:t1], d["weight"], d["bias"], state, final_out=state))
    assert torch.equal(torch.cat(parts, 1), want) and torch.equal(state, wfin)


def test_rows_behind_the_end_are_not_read():
    d = inputs(4, 50, 24, 4, "f32", ragged=True, seed=2)
    clean = ssd.causal_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], True, lengths=d["lengths"])
    gclean = ssd.causal_conv_bwd(d["x"], d["weight"], d["bias"], d["dy"], d["init"], d["dfinal"], lengths=d["lengths"])
    x, dy = d["x"].clone(), d["dy"].clone()
    for i, end in enumerate(d["lengths"].tolist()):
        x[i, end:] = float("nan")
        dy[i, end:] = float("inf")
    got = ssd.causal_conv_fwd(x, d["weight"], d["bias"], d["init"], True, lengths=d["lengths"])
    ggot = ssd.causal_conv_bwd(x, d["weight"], d["bias"], dy, d["init"], d["dfinal"], lengths=d["lengths"])
    assert all(torch.equal(p, q) for p, q in zip(got, clean))
    assert all(torch.equal(ggot[k], gclean[k]) for k in gclean)
    # lengths outside [0, seqlen] are taken as the nearest within
    wild = torch.tensor([1 << 30, -5, 50, 51], dtype=torch.int32, device="cuda")
    tame = torch.tensor([50, 0, 50, 50], dtype=torch.int32, device="cuda")
    a = ssd.causal_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], True, lengths=wild)
    b = ssd.causal_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], True, lengths=tame)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_interleaved_and_broadcast_rows():
    # (seqlen, batch, channels) storage, and one sequence read by the whole batch
    d = inputs(3, 21, 16, 4, "f32", state=False)
    want = ssd.causal_conv_fwd(d["x"], d["weight"], d["bias"])
    turned = d["x"].transpose(0, 1).contiguous().transpose(0, 1)
    assert not turned.is_contiguous()
    assert torch.equal(ssd.causal_conv_fwd(turned, d["weight"], d["bias"]), want)
    one = d["x"][:1].expand(3, 21, 16)
    got = ssd.causal_conv_fwd(one, d["weight"], d["bias"])
    assert all(torch.equal(got[i], want[0]) for i in range(3))


def test_arguments_that_are_no_tensors():
    d = inputs(2, 8, 16, 4, "f32")
    for x, weight, bias in ((3.0, d["weight"], d["bias"]), (d["x"], None, d["bias"]), (d["x"], d["weight"], 3.0)):
        with pytest.raises(TypeError):
            ssd.causal_conv_fwd(x, weight, bias)
    with pytest.raises(TypeError):
        ssd.causal_conv_bwd(d["x"], d["weight"], d["bias"], None)


def test_refusals_leave_the_outputs():
    d = inputs(2, 8, 16, 4, "f32")
    y = torch.full((2, 8, 16), 7.0, device="cuda")
    with pytest.raises(ValueError, match="activation"):
        ssd.causal_conv_fwd(d["x"], d["weight"], d["bias"], activation="relu", out=y)
    with pytest.raises(ssd.SSDError, match="UNSUPPORTED"):
        ssd.causal_conv_fwd(d["x"], torch.randn(16, 5, device="cuda"), out=y)
    with pytest.raises(TypeError):
        ssd.causal_conv_fwd(d["x"].half(), d["weight"], out=y)
    with pytest.raises(ValueError, match="row must be contiguous"):
        ssd.causal_conv_fwd(torch.randn(2, 16, 8, device="cuda").transpose(1, 2), d["weight"], out=y)
    with pytest.raises(ValueError, match="overlap"):
        ssd.causal_conv_fwd(d["x"][:, :1].expand(2, 8, 16), d["weight"], out=y)
    with pytest.raises(ssd.SSDError, match="INVALID"):
        ssd.causal_conv_fwd(d["x"], d["weight"], out=d["x"])
    with pytest.raises(ssd.SSDError, match="INVALID"):
        ssd.causal_conv_step(d["x"][:, 0], d["weight"], None, d["init"], out=d["init"].view(-1)[:32].view(2, 16))
    with pytest.raises(ssd.SSDError, match="WORKSPACE"):
        ssd.causal_conv_bwd(d["x"], d["weight"], d["bias"], d["dy"],
                            workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert bool((y == 7.0).all())


def test_captured_call_replays():
    d = inputs(2, 37, 48, 4, "bf16", ragged=True)
    x = d["x"].clone()
    state = d["init"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        ssd.causal_conv_fwd(x, d["weight"], d["bias"], d["init"])  # loads the kernels
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = ssd.causal_conv_fwd(x, d["weight"], d["bias"], d["init"], lengths=d["lengths"])
        g = ssd.causal_conv_bwd(x, d["weight"], d["bias"], d["dy"], d["init"], d["dfinal"], lengths=d["lengths"])
        ys = ssd.causal_conv_step(x[:, 0], d["weight"], d["bias"], state)
    for k in range(3):
        new = inputs(2, 37, 48, 4, "bf16", seed=20 + k)["x"]
        x.copy_(new)
        state.copy_(d["init"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ssd.causal_conv_fwd(new, d["weight"], d["bias"], d["init"], lengths=d["lengths"]))
        e = ssd.causal_conv_bwd(new, d["weight"], d["bias"], d["dy"], d["init"], d["dfinal"], lengths=d["lengths"])
        assert all(torch.equal(g[n], e[n]) for n in e)
        s2 = d["init"].clone()
        assert torch.equal(ys, ssd.causal_conv_step(new[:, 0], d["weight"], d["bias"], s2))
        assert torch.equal(state, s2)


def test_a_given_stream_runs_the_call():
    d = inputs(2, 64, 64, 4, "f32")
    want = ssd.causal_conv_bwd(d["x"], d["weight"], d["bias"], d["dy"], d["init"], d["dfinal"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ssd.causal_conv_bwd(d["x"], d["weight"], d["bias"], d["dy"], d["init"], d["dfinal"],
                              stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_c_abi_events_free_call():
    # the plain C call with dense strides given as {0, 0}
    d = inputs(1, 4, 8, 2, "f32", state=False)
    lib = ssd.load_library()
    shape = ssd.ConvShape(1, 4, 8, 2, ssd.SSD_ACT_NONE, ssd.SSD_DTYPE_F32, ssd.SSD_DTYPE_F32, 0, 0)
    y = torch.empty((1, 4, 8), device="cuda")
    st = lib.ssd_causal_conv_fwd(ctypes.byref(shape), d["x"].data_ptr(), d["weight"].data_ptr(), None, None, None,
                                 y.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(y, ssd.causal_conv_fwd(d["x"], d["weight"], activation=None))


def test_two_streams_at_once():
    cases = [inputs(2, 300, 128, 4, "bf16", seed=70 + k) for k in range(2)]
    call = lambda d: ssd.causal_conv_bwd(d["x"], d["weight"], d["bias"], d["dy"], d["init"], d["dfinal"])  # noqa: E731
    want = [call(d) for d in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for k, (d, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[k] = call(d)
    torch.cuda.synchronize()
    assert all(torch.equal(g[k], w[k]) for g, w in zip(got, want) for k in w)


@pytest.mark.parametrize("c", [4096, 4099])
def test_offsets_beyond_32_bits(c):
    # 2.2e9 elements: the last rows against a call on them alone, continued from the inputs before them
    L, tail = 540_000, 1000
    gen = torch.Generator(device="cuda").manual_seed(4)
    piece = torch.randn((1000, c), generator=gen, device="cuda").bfloat16()
    x = piece.repeat(L // 1000, 1)[None]
    w, bias = torch.randn((c, 4), generator=gen, device="cuda"), torch.randn(c, generator=gen, device="cuda")
    y, fin = ssd.causal_conv_fwd(x, w, bias, None, True, y_dtype=torch.bfloat16)
    before = x[:, L - tail - 3:L - tail].contiguous()
    y1, fin1 = ssd.causal_conv_fwd(x[:, -tail:], w, bias, before, True, y_dtype=torch.bfloat16)
    assert torch.equal(y[:, -tail:], y1) and torch.equal(fin, fin1)
    g = ssd.causal_conv_bwd(x, w, bias, y, dx_dtype=torch.bfloat16)
    g1 = ssd.causal_conv_bwd(x[:, -tail:], w, bias, y[:, -tail:], before, dx_dtype=torch.bfloat16)
    assert torch.equal(g["dx"][:, -tail:], g1["dx"])
    # the sums: all pieces of 1000 rows but the first are alike
    mid = ssd.causal_conv_bwd(x[:, 1000:2000], w, bias, y[:, 1000:2000], x[:, 997:1000].contiguous())
    want = mid["dweight"].double() * (L // 1000 - 1)
    first = ssd.causal_conv_bwd(x[:, :1000], w, bias, y[:, :1000])["dweight"].double()
    assert float((g["dweight"].double() - want - first).norm() / want.norm()) < 1e-5


@pytest.mark.parametrize("c", [24, 512])  # one channel a lane, and four
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_last_inputs_not_finite_leave_the_rows_behind_them_zero(c, value):
    # the first W - 1 rows behind an end have the last inputs in their windows
    L, W = 40, 4
    d = inputs(4, L, c, W, "f32", seed=6)
    d["lengths"] = torch.tensor([L, 18, 2, 0], dtype=torch.int32, device="cuda")
    for i, end in enumerate(d["lengths"].tolist()):
        if end > 0:
            d["x"][i, end - 1, ::2] = value
        else:
            d["init"][i, -1, ::2] = value
    d["weight"][5, 1] = value
    g = ssd.causal_conv_bwd(d["x"], d["weight"], d["bias"], d["dy"], d["init"], d["dfinal"], lengths=d["lengths"])
    y = ssd.causal_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], lengths=d["lengths"])
    for i, end in enumerate(d["lengths"].tolist()):
        assert bool((g["dx"][i, end:] == 0).all()) and bool((y[i, end:] == 0).all())


@pytest.mark.parametrize("c", [24, 512])
def test_rows_behind_the_end_add_nothing_to_the_sums(c):
    # a filter whose oldest tap overflows on the last input: no live row meets the two, a padded one does
    d = inputs(2, 30, c, 4, "f32", state=False, seed=7)
    end = 18
    d["lengths"] = torch.full((2,), end, dtype=torch.int32, device="cuda")
    d["x"][:, end - 1] = 1e30
    d["weight"][:, 0] = 1e30
    d["weight"][:, 3] = 1e-30
    d["x"][:, :end - 1] *= 1e-30
    got = ssd.causal_conv_bwd(d["x"], d["weight"], d["bias"], d["dy"], lengths=d["lengths"])
    cut = ssd.causal_conv_bwd(d["x"][:, :end].contiguous(), d["weight"], d["bias"], d["dy"][:, :end].contiguous())
    assert all(bool(torch.isfinite(v).all()) for v in cut.values())
    assert torch.equal(got["dx"][:, :end], cut["dx"])
    assert all(torch.equal(got[k], cut[k]) for k in ("dweight", "dbias"))


@pytest.mark.parametrize("kind", ["random", "drift"])
@pytest.mark.parametrize("b,L,c,W,dtype", [(2, 3001, 24, 4, "f32"), (1, 5000, 512, 3, "f32"), (3, 2048, 771, 2, "bf16"),
                                           (1, 300_000, 40, 4, "f32")])
def test_sums_over_tokens_are_held_in_64_bits(b, L, c, W, dtype, kind):
    # Without an activation the terms of dweight and dbias are products of two inputs, and inputs, exact in 64 bits.
    # They are rounded to fp32, by half a step of 2^-24, as the sums of strips of a multiple of 16 tokens, as those
    # of blocks of four strips and at the end; before that (terms + 4) roundings of 2^-53 of the terms' magnitudes.
    # "drift": terms of 1 + 2^-18 + 2^-23, each just above half a step of a sum between 64 and 128, so that a sum
    # in fp32 runs away from 128 of them by 2^-19.
    d = inputs(b, L, c, W, dtype, ragged=b > 1, seed=13)
    if kind == "drift":
        d["dy"][:] = 1 + 2.0 ** -18 + 2.0 ** -23
        d["x"][:] = 1.0
        d["init"][:] = 1.0
    got = ssd.causal_conv_bwd(d["x"], d["weight"], d["bias"], d["dy"], d["init"], activation=None, lengths=d["lengths"])
    x = torch.cat([d["init"].double(), d["x"].double()], 1)
    dy = d["dy"].double()
    if d["lengths"] is not None:
        dy = dy * (torch.arange(L, device="cuda")[None, :] < d["lengths"][:, None])[..., None]
    pad = (0, 0, 0, -L % 16)
    for k in range(W + 1):
        terms = dy * x[:, k:k + L] if k < W else dy
        have = got["dweight"][:, k] if k < W else got["dbias"]
        want = terms.sum((0, 1))
        pieces = torch.nn.functional.pad(terms, pad).view(b, -1, 16, c).sum(2).abs().sum((0, 1))
        bound = 2.0 ** -24 * (want.abs() + 2.001 * pieces) + 2 * (b * L + 4) * 2.0 ** -53 * terms.abs().sum((0, 1))
        assert bool(((have.double() - want).abs() <= bound).all()), k


# Four channels a lane, which take rows of whole aligned pieces that fill three quarters of their waves (192, 256,
# 512, 1028 channels), and the same sizes where one operand lies an element off.  b, L, c, W, x, dy, dx (and y), act,
# layout, state; lengths of L, 0, 1, 2 and what is left of the taps; one of several strips of 32 tokens
WIDE = [
    (5, 50, 192, 2, "f32", "f32", "f32", "silu", "dense", True),
    (5, 33, 256, 3, "f32", "f32", "f32", "silu", "sliced", True),
    (4, 17, 512, 4, "f32", "f32", "f32", None, "dense", True),
    (2, 7000, 1028, 4, "f32", "f32", "f32", "silu", "dense", True),
    (5, 47, 1028, 4, "bf16", "bf16", "bf16", "silu", "sliced", True),
    (4, 64, 256, 4, "bf16", "f32", "bf16", "silu", "dense", True),
    (3, 30, 512, 3, "bf16", "bf16", "f32", "silu", "sliced", False),
    (5, 21, 192, 2, "bf16", "f32", "f32", None, "sliced", True),
    (5, 50, 192, 4, "f32", "f32", "f32", "silu", "odd", True),
    (4, 40, 512, 4, "bf16", "f32", "bf16", "silu", "odd", True),
]


def wide_inputs(case):
    b, L, c, W, x, dy, _, _, layout, state = case
    d = inputs(b, L, c, W, x, layout == "sliced", state, seed=17)
    d["lengths"] = torch.tensor([L, 0, 1, 2, L - W + 1][:b], dtype=torch.int32, device="cuda")
    d["dy"] = d["dy"].to(TYPES[dy])
    if layout != "dense":
        off = 8 if layout == "sliced" else 1
        for k in ("x", "dy"):
            wide = torch.zeros((b, L, c + 24), dtype=d[k].dtype, device="cuda")
            wide[..., off:off + c] = d[k]
            d[k] = wide[..., off:off + c]
    return d


@pytest.mark.parametrize("case", WIDE, ids=lambda c: "b%d_L%d_c%d_w%d_%s_%s_%s_%s_%s%s" % (c[:9] + ("_state" * c[9],)))
def test_four_channels_a_lane(case):
    b, L, c, W, dtype, dyt, dxt, act, layout, state = case
    d = wide_inputs(case)
    got = ssd.causal_conv_bwd(d["x"], d["weight"], d["bias"], d["dy"], d["init"], d["dfinal"], activation=act,
                              lengths=d["lengths"], dx_dtype=TYPES[dxt])
    y, fin = ssd.causal_conv_fwd(d["x"], d["weight"], d["bias"], d["init"], True, activation=act,
                                 lengths=d["lengths"], y_dtype=TYPES[dxt])
    fargs = [host(d[k]) for k in ("x", "weight", "bias", "init", "lengths")]
    ref, rfin = lo.conv(*fargs, act=act is not None)
    mag = lo.conv_magnitude(*fargs)
    assert np.all(np.abs(host(y) - ref) <= 16 * EPS * (mag + 1) * (ref != 0) + half_step(dxt, ref))
    assert np.array_equal(host(fin), rfin)
    args = [host(d[k]) for k in ("x", "weight", "bias", "dy", "init", "dfinal", "lengths")]
    ref = lo.conv_bwd(*args, act=act is not None)
    mag = lo.conv_bwd(*[None if a is None else np.abs(a) for a in args], act=False)
    scale = 1 + max(1.0, float(np.max(np.abs(args[0]))) * float(np.max(np.abs(args[1]).sum(1))))
    assert set(got) == set(ref)
    for k, r in ref.items():
        bound = 400 * EPS * scale * mag[k] + half_step(dxt if k == "dx" else "f32", r)
        assert np.all(np.abs(host(got[k]) - r) <= bound), k
    for i, end in enumerate(host(d["lengths"])):
        assert not got["dx"][i, end:].any() and not y[i, end:].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_four_channels_a_lane_agree_with_one(dtype):
    # the same numbers an element off, one channel a lane: every result is made of the same sums in the same order
    b, L, c, W = 3, 100, 512, 4
    d = inputs(b, L, c, W, dtype, ragged=True, seed=18)
    odd = dict(d)
    wide = torch.zeros((b, L, c + 1), dtype=TYPES[dtype], device="cuda")
    wide[..., 1:] = d["x"]
    odd["x"] = wide[..., 1:]
    results = []
    for q in (d, odd):
        g = ssd.causal_conv_bwd(q["x"], q["weight"], q["bias"], q["dy"], q["init"], q["dfinal"], lengths=q["lengths"])
        y, fin = ssd.causal_conv_fwd(q["x"], q["weight"], q["bias"], q["init"], True, lengths=q["lengths"])
        results.append(dict(g, y=y, fin=fin))
    assert all(torch.equal(results[0][k], results[1][k]) for k in results[0])


@pytest.mark.parametrize("L", [30, 64])
@pytest.mark.parametrize("c", [24, 512])
def test_last_inputs_not_finite_enter_only_their_own_taps(c, L):
    # no live row meets the last input with another tap than the newest: those gradients of the filter stay finite,
    # also where a sequence fills its rows but not the kernel's groups of tokens
    d = inputs(3, L, c, 4, "f32", seed=23)
    d["lengths"] = torch.tensor([L, 18, 1], dtype=torch.int32, device="cuda")
    ends = d["lengths"].tolist()
    args = {k: host(d[k]) for k in ("x", "weight", "bias", "dy", "init", "dfinal", "lengths")}
    for i, end in enumerate(ends):
        d["x"][i, end - 1] = float("inf")
        args["x"][i, end - 1] = 0.0
    got = ssd.causal_conv_bwd(d["x"], d["weight"], d["bias"], d["dy"], d["init"], d["dfinal"], activation=None,
                              lengths=d["lengths"])
    ref = lo.conv_bwd(*args.values(), act=False)
    mag = lo.conv_bwd(*[np.abs(a) for a in args.values()], act=False)
    for k in ("dx", "dbias", "d_initial_states"):
        assert np.all(np.abs(host(got[k]) - ref[k]) <= 8 * EPS * mag[k]), k
    assert np.all(np.abs(host(got["dweight"][:, :3]) - ref["dweight"][:, :3]) <= 8 * EPS * mag["dweight"][:, :3])
    assert not bool(torch.isfinite(got["dweight"][:, 3]).any())
