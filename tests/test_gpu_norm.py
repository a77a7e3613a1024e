"""Parity of the RMS norm (ssd_rms_norm_fwd, _bwd) against the fp64 oracle.

Bounds, in units of EPS = 2^-24 (half a step of fp32, relative).  u = x +
residual is one rounding, EPS |u|.  Sums over a row: a lane adds at most 64
values in fp32 (64-bit beyond 16 384 channels), lanes and waves add 8 more
levels, and each square carries 3 EPS from u: mean(u^2) is off by less than 80
EPS of itself, r by 40 EPS and 4 for the square root, quotient and eps: 44.
y = u r w: 44 + 3 more, below 64 EPS |y|.  Stored in bf16 another 2^-8 |y|
at most (half a step is 2^-9 of the binade's top, 2^-8 of its bottom).
residual_out is u with the same.  8 bits: the scale is off by 64 EPS of itself
(and nothing where it is the least one); a code is y / scale rounded to nearest: half a step of
e4m3 is 2^-4 of the value, 2^-10 below 2^-6 (subnormal codes step by 2^-9),
plus 130 EPS for y's and the scale's own errors.  du: the magnitudes of its terms times (3 r's
and the product's roundings) 3 * 44 + 80 + 8 < 256 EPS; dweight adds 64
roundings of a lane over rows (256 at most; 4 waves) and one at the end: below
512 EPS of the sum of magnitudes.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mamba_chunked_ssd_amd as ssd
from oracle import mixer_ops as mo

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def host(t):
    return None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def half_step(dtype, ref):
    return 2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0


def inputs(b, L, c, x="bf16", stream="f32", out="bf16", layout="dense", ragged=False, seed=0):
    g = torch.Generator().manual_seed(1000 * seed + 7 * L + c)

    def rows(t):
        full = torch.randn((b, L, c), generator=g).to(TYPES[t])
        if layout == "dense":
            return full.cuda()
        off = 1 if layout == "odd" else 8
        wide = torch.full((b, L, c + 19), float("nan")).to(TYPES[t])
        wide[..., off:off + c] = full
        return wide.cuda()[..., off:off + c]

    d = dict(x=rows(x), weight=(1 + 0.3 * torch.randn(c, generator=g)).cuda())
    d["residual"] = 4 * rows(stream) if stream else None
    if stream and layout != "dense":
        keep = rows(stream)
        keep.mul_(4)
        d["residual"] = keep
    d["lengths"] = None
    if ragged:
        d["lengths"] = torch.tensor([L, 0, 1, L // 2, L - 1][:b], dtype=torch.int32).cuda()
    d["dy"] = rows("bf16" if out == "bf16" else "f32")
    d["dres"] = rows(stream) if stream else None
    return d


# (b, L, c, x, stream, out, block, layout, ragged): channels of less than a piece, odd ones, each number of pieces a
# lane, rows of a wave, of a block and of neither; more rows than waves of a block
CASES = [
    (1, 1, 1, "f32", "f32", "f32", 0, "dense", False),
    (2, 3, 5, "bf16", "", "bf16", 0, "odd", False),
    (1, 1, 2560, "bf16", "f32", "e4m3", 0, "dense", False),
    (3, 7, 8, "f32", "", "f32", 0, "dense", True),
    (5, 9, 33, "bf16", "bf16", "f32", 0, "odd", True),
    (2, 5, 512, "bf16", "f32", "bf16", 0, "sliced", False),
    (3, 17, 771, "f32", "f32", "f32", 0, "odd", True),
    (2, 3, 1030, "bf16", "bf16", "e4m3", 32, "odd", False),
    (1, 4, 1537, "f32", "bf16", "e4m3", 64, "dense", False),
    (2, 2, 2560, "bf16", "f32", "e4m3", 128, "sliced", False),
    (5, 3, 2900, "bf16", "", "e4m3", 128, "odd", True),
    (1, 3, 3333, "f32", "f32", "e4m3", 0, "dense", False),
    (2, 2, 4096, "f32", "f32", "bf16x", 0, "dense", False),
    (2, 2, 4097, "bf16", "f32", "bf16", 0, "odd", False),
    (3, 3, 6200, "bf16", "bf16", "e4m3", 64, "dense", True),
    (1, 2, 9001, "f32", "", "e4m3", 128, "odd", False),
    (1, 3, 12000, "bf16", "f32", "f32", 0, "sliced", False),
    (1, 2, 16384, "f32", "f32", "e4m3", 0, "dense", False),
    (2, 2, 16385, "bf16", "bf16", "e4m3", 32, "odd", False),
    (3, 2, 20011, "f32", "f32", "f32", 0, "odd", True),
    (2, 3, 40000, "bf16", "f32", "e4m3", 0, "dense", True),
    (3, 0, 16, "bf16", "f32", "bf16", 0, "dense", False),
]


def ids(c):
    return "b%d_L%d_c%d_x%s_r%s_y%s%d_%s%s" % (c[:8] + ("_ragged" * c[8],))


def check_out(y, ref, out):
    assert np.all(np.abs(host(y) - ref) <= 64 * EPS * np.abs(ref) + half_step(out, ref))


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward(case):
    b, L, c, x, stream, out, block, layout, ragged = case
    out = "f32" if out == "bf16x" else out
    d = inputs(b, L, c, x, stream, out, layout, ragged)
    got = ssd.rms_norm_fwd(d["x"], d["weight"], d["residual"], lengths=d["lengths"], y_dtype=TYPES[out],
                           scale_block=block, return_residual=True)
    torch.cuda.synchronize()
    u, y = mo.norm(host(d["x"]), host(d["weight"]), host(d["residual"]), lengths=host(d["lengths"]))
    kept = got[-1]
    assert kept.dtype == (TYPES[stream] if stream else torch.float32)
    assert np.all(np.abs(host(kept) - u) <= EPS * np.abs(u) + half_step(stream, u))
    if out != "e4m3":
        check_out(got[0], y, out)
        return
    if y.size == 0:
        return
    s, per = mo.scales(y, block)
    assert got[1].shape == s.shape
    assert np.all(np.abs(host(got[1]) - s) <= 64 * EPS * s * (s > 2.0 ** -126))
    q = y / per
    assert np.all(np.abs(host(got[0].float()) - q) <= 2.0 ** -4 * np.maximum(np.abs(q), 2.0 ** -6) + 130 * EPS * np.abs(q))


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_backward(case):
    b, L, c, x, stream, out, _, layout, ragged = case
    d = inputs(b, L, c, x, stream, "bf16" if out in ("bf16", "bf16x") else "f32", layout, ragged)
    u = d["residual"] if stream else d["x"]
    got = ssd.rms_norm_bwd(d["dy"], u, d["weight"], d["dres"], lengths=d["lengths"], dx_dtype=TYPES[x],
                           want_dresidual=True)
    torch.cuda.synchronize()
    du, dw, mag, wmag = mo.norm_bwd(host(d["dy"]), host(u), host(d["weight"]), host(d["dres"]), lengths=host(d["lengths"]))
    for k, t in (("dx", x), ("dresidual", stream or x)):
        assert got[k].dtype == TYPES[t]
        assert np.all(np.abs(host(got[k]) - du) <= 256 * EPS * mag + half_step(t, du)), k
    assert np.all(np.abs(host(got["dweight"]) - dw) <= 512 * EPS * wmag)
    if d["lengths"] is not None:
        for i, end in enumerate(host(d["lengths"])):
            assert not got["dx"][i, end:].any() and not got["dresidual"][i, end:].any()


@pytest.mark.parametrize("c", [7, 200, 5000, 17000])
def test_without_weight_stream_or_requests(c):
    d = inputs(2, 3, c, "f32", "f32", "f32")
    one = torch.ones(c, device="cuda")
    assert torch.equal(ssd.rms_norm_fwd(d["x"]), ssd.rms_norm_fwd(d["x"], one))
    a = ssd.rms_norm_bwd(d["dy"], d["x"], want_dweight=False)
    b = ssd.rms_norm_bwd(d["dy"], d["x"], one)
    assert set(a) == {"dx"} and torch.equal(a["dx"], b["dx"])
    # (b, c) rows are those of one-token sequences
    assert torch.equal(ssd.rms_norm_fwd(d["x"][:, 0], d["weight"], d["residual"][:, 0]),
                       ssd.rms_norm_fwd(d["x"][:, :1], d["weight"], d["residual"][:, :1])[:, 0])
    kept = ssd.rms_norm_fwd(d["x"], return_residual=True, residual_dtype=torch.bfloat16)[1]
    assert torch.equal(kept, d["x"].bfloat16())


@pytest.mark.parametrize("c", [6, 264, 2560, 4100, 16392, 20001])
@pytest.mark.parametrize("stream", ["f32", "bf16"])
def test_stream_in_place(c, stream):
    d = inputs(3, 5, c, "bf16", stream, "bf16", ragged=True)
    want = ssd.rms_norm_fwd(d["x"], d["weight"], d["residual"], lengths=d["lengths"], return_residual=True)
    held = d["residual"].clone()
    y, u = ssd.rms_norm_fwd(d["x"], d["weight"], held, lengths=d["lengths"], return_residual=True, residual_out=held)
    assert u is held and torch.equal(held, want[1]) and torch.equal(y, want[0])


@pytest.mark.parametrize("c", [40, 2560, 5000, 17000])
def test_rows_behind_the_end_are_not_read(c):
    d = inputs(5, 6, c, "f32", "f32", "f32", ragged=True)
    clean = ssd.rms_norm_fwd(d["x"], d["weight"], d["residual"], lengths=d["lengths"], return_residual=True)
    gclean = ssd.rms_norm_bwd(d["dy"], d["x"], d["weight"], d["dres"], lengths=d["lengths"], want_dresidual=True)
    e = {k: d[k].clone() for k in ("x", "residual", "dy", "dres")}
    for i, end in enumerate(d["lengths"].tolist()):
        for k in e:
            e[k][i, end:] = float("nan")
    got = ssd.rms_norm_fwd(e["x"], d["weight"], e["residual"], lengths=d["lengths"], return_residual=True)
    ggot = ssd.rms_norm_bwd(e["dy"], e["x"], d["weight"], e["dres"], lengths=d["lengths"], want_dresidual=True)
    assert all(torch.equal(p, q) for p, q in zip(got, clean))
    assert all(torch.equal(ggot[k], gclean[k]) for k in gclean)
    wild = torch.tensor([1 << 30, -5, 6, 7, 0], dtype=torch.int32, device="cuda")
    tame = torch.tensor([6, 0, 6, 6, 0], dtype=torch.int32, device="cuda")
    assert torch.equal(ssd.rms_norm_fwd(d["x"], lengths=wild), ssd.rms_norm_fwd(d["x"], lengths=tame))


@pytest.mark.parametrize("c", [100, 2560, 5000, 17000])
@pytest.mark.parametrize("block", [0, 32, 128])
def test_special_values_in_8_bits(c, block):
    x = torch.randn((6, c), device="cuda", generator=torch.Generator(device="cuda").manual_seed(c))
    x[0] = 0.0
    x[1, 3] = float("nan")
    x[2, 3] = float("inf")
    x[3] *= 1e-30
    x[4] *= 1e15
    x[5, 0] = 1e6  # all else in its scale's block rounds to few codes
    y, s = ssd.rms_norm_fwd(x, y_dtype=torch.float8_e4m3fn, scale_block=block)
    y = y.float()
    assert bool((y[0] == 0).all()) and bool((s[0] == 2.0 ** -126).all())
    assert bool(torch.isnan(s[1]).all()) and bool(torch.isnan(y[1]).all())  # r itself is NaN
    cut = c if block == 0 else min(block, c)
    assert bool(torch.isnan(y[2, :cut]).all()) and bool(torch.isnan(s[2, 0])) and bool((y[2, cut:] == 0).all())
    for row in (3, 4, 5):
        assert bool(torch.isfinite(y[row]).all()) and bool((y[row].abs() <= 448).all())
        blocks = torch.nn.functional.pad(y[row].abs(), (0, -c % (block or c))).view(-1, block or c)
        assert bool((blocks.amax(1) == 448).all())  # the largest of each is 448 scales


def test_arguments_that_are_no_tensors():
    d = inputs(2, 3, 16)
    for args in ((3.0, d["weight"], None), (d["x"], 3.0, None), (d["x"], None, 3.0)):
        with pytest.raises(TypeError):
            ssd.rms_norm_fwd(*args)
    with pytest.raises(TypeError):
        ssd.rms_norm_bwd(None, d["x"])
    with pytest.raises(TypeError):
        ssd.rms_norm_bwd(d["dy"], d["x"], d["weight"], 3.0)


def test_refusals_leave_the_outputs():
    d = inputs(2, 3, 16, "bf16", "f32")
    y = torch.full((2, 3, 16), 7.0, device="cuda")
    with pytest.raises(ValueError, match="scale_block"):
        ssd.rms_norm_fwd(d["x"], y_dtype=torch.float8_e4m3fn, scale_block=48)
    with pytest.raises(ValueError, match="8-bit"):
        ssd.rms_norm_fwd(d["x"], scale_block=32, out=y)
    with pytest.raises(TypeError):
        ssd.rms_norm_fwd(d["x"].half(), out=y)
    with pytest.raises(TypeError):
        ssd.rms_norm_fwd(d["x"], y_dtype=torch.float16, out=y)
    with pytest.raises(ValueError, match="row must be contiguous"):
        ssd.rms_norm_fwd(torch.randn(2, 16, 3, device="cuda").transpose(1, 2), out=y)
    with pytest.raises(ValueError, match="shape"):
        ssd.rms_norm_fwd(d["x"], residual=d["residual"][:1], out=y)
    with pytest.raises(ssd.SSDError, match="INVALID"):
        ssd.rms_norm_fwd(d["residual"], out=d["residual"])
    with pytest.raises(ssd.SSDError, match="INVALID"):
        ssd.rms_norm_fwd(d["x"], eps=-1.0, out=y)
    wide = torch.randn(2, 3, 20, device="cuda")
    with pytest.raises(ssd.SSDError, match="INVALID"):  # a strided stream is not written in place
        ssd.rms_norm_fwd(d["x"], residual=wide[..., :16], residual_out=wide.view(-1)[:96].view(2, 3, 16), out=y)
    with pytest.raises(ssd.SSDError, match="WORKSPACE"):
        ssd.rms_norm_bwd(d["dy"], d["x"], d["weight"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert bool((y == 7.0).all())


def test_captured_call_replays():
    d = inputs(3, 5, 2560, "bf16", "f32", "bf16", ragged=True)
    x = d["x"].clone()

    def calls(x):
        return [*ssd.rms_norm_fwd(x, d["weight"], d["residual"], lengths=d["lengths"], return_residual=True,
                                  y_dtype=torch.float8_e4m3fn, scale_block=128),
                *ssd.rms_norm_bwd(d["dy"], x, d["weight"], lengths=d["lengths"]).values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(x)
    for k in range(3):
        x.copy_(inputs(3, 5, 2560, seed=20 + k)["x"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(got, calls(x)))


def test_streams():
    cases = [inputs(2, 300, 640, "bf16", "f32", seed=70 + k) for k in range(2)]
    call = lambda d: ssd.rms_norm_bwd(d["dy"], d["residual"], d["weight"], d["dres"])  # noqa: E731
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
    given = ssd.rms_norm_bwd(cases[0]["dy"], cases[0]["residual"], cases[0]["weight"], cases[0]["dres"], stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(given[k], want[0][k]) for k in given)


def test_interleaved_and_broadcast_rows():
    d = inputs(3, 21, 72, "f32", "f32")
    want = ssd.rms_norm_fwd(d["x"], d["weight"], d["residual"])
    turned = d["x"].transpose(0, 1).contiguous().transpose(0, 1)
    assert not turned.is_contiguous()
    assert torch.equal(ssd.rms_norm_fwd(turned, d["weight"], d["residual"]), want)
    one = d["x"][:1].expand(3, 21, 72)
    got = ssd.rms_norm_fwd(one, d["weight"])
    assert all(torch.equal(got[i], got[0]) for i in range(3))


@pytest.mark.parametrize("c", [4096, 4099, 20000])
def test_offsets_beyond_32_bits(c):
    L = 2 ** 31 // c + 1000
    piece = torch.randn((1, 1000, c), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").bfloat16()
    x = piece.repeat(1, L // 1000 + 1, 1)[:, :L]
    y = ssd.rms_norm_fwd(x, y_dtype=torch.bfloat16)
    assert torch.equal(y[:, -700:], ssd.rms_norm_fwd(x[:, -700:], y_dtype=torch.bfloat16))
    g = ssd.rms_norm_bwd(y, x, dx_dtype=torch.bfloat16)
    g1 = ssd.rms_norm_bwd(y[:, -700:], x[:, -700:], dx_dtype=torch.bfloat16)
    assert torch.equal(g["dx"][:, -700:], g1["dx"])


def test_sums_over_many_rows():
    # 2^19 rows: 256 at most in 32 bits, then 64.  Terms of 1 + 2^-12 or so, all positive: sums of 2^8 of them are
    # off by 2^8 EPS at most, relatively, and r's 44 EPS
    rows = 1 << 19
    u = 1 + torch.rand((rows, 4), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    got = ssd.rms_norm_bwd(u, u)["dweight"].double()
    r = ((u.double() ** 2).mean(1, keepdim=True) + 1e-5).rsqrt()
    want = (u.double() ** 2 * r).sum(0)
    assert bool(((got - want).abs() <= (4 * 256 + 50) * EPS * want).all())
