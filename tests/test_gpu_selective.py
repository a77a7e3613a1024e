"""Parity of the selective scan (ssd_selective_scan_fwd, _bwd, _step) against
the fp64 oracle, and of the layer paths that the convolution and the scans
make together.

Bounds: max |gpu - oracle| / rms(oracle) <= 1e-4 for every fp32 result, as for
the chunked scan: a decay exp(d A) carries the relative error of its exponent,
(5 + |d A|) 2^-23 or so, and a state sums as many of them as it remembers
tokens, at most a few hundred here, so 300 * 6 * 2^-23 = 2e-4 of the largest
term if all erred alike and a tenth of that as they do not.  A bf16 y adds half
a step, 2^-8 |y|.
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import mamba_chunked_ssd_amd as ssd
from oracle import layer_ops as lo
from tests.gpu_util import nerr

pytestmark = pytest.mark.gpu

TOL = 1e-4
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "init", "lengths")


def inputs(b, L, c, n, g=1, dtype="f32", gate=True, state=True, ragged=False, sliced=False, seed=0, softplus=True):
    gen = torch.Generator().manual_seed(seed + 13 * L + 3 * c + n)
    t = TYPES[dtype]

    def rows(*shape):
        if not sliced:
            return torch.randn(shape, generator=gen).to(t).cuda()
        k = len(shape) - 2
        flat = int(np.prod(shape[2:]))
        wide = torch.randn(shape[:2] + (flat + 11,), generator=gen).to(t).cuda()
        return wide[..., 3:3 + flat].unflatten(-1, shape[2:]) if k > 1 else wide[..., 3:3 + flat]

    d = dict(x=rows(b, L, c), dt=rows(b, L, c), B=rows(b, L, g, n), C=rows(b, L, g, n))
    if softplus:
        d["dt_bias"] = (torch.randn(c, generator=gen) - 3).cuda()
    else:
        d["dt"] = (0.1 * d["dt"].float().abs()).to(t)
        d["dt_bias"] = torch.full((c,), 0.01).cuda()
    d["A"] = -(torch.arange(1, n + 1).float() * torch.exp(0.3 * torch.randn((c, n), generator=gen))).cuda()
    d["D"] = torch.randn(c, generator=gen).cuda()
    d["z"] = rows(b, L, c) if gate else None
    d["init"] = (0.5 * torch.randn((b, c, n), generator=gen)).cuda() if state else None
    d["dfinal"] = torch.randn((b, c, n), generator=gen).cuda() if state else None
    d["dy"] = torch.randn((b, L, c), generator=gen).cuda()
    d["lengths"] = None
    if ragged:
        d["lengths"] = torch.randint(0, L + 1, (b,), generator=gen, dtype=torch.int32).cuda()
        d["lengths"][-1] = 0
        if b > 1:
            d["lengths"][0] = L
    return d


def host(t):
    return None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def fwd(d, **kw):
    return ssd.selective_scan_fwd(*[d[k] for k in NAMES[:9]], True, lengths=d["lengths"], **kw)


def bwd(d, dy=None, **kw):
    return ssd.selective_scan_bwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["dy"] if dy is None else dy,
                                  d["z"], d["dt_bias"], d["init"], d["dfinal"], lengths=d["lengths"], **kw)


# b, L, c, n, g, dtype, y, gate, state, ragged, sliced, softplus: lengths around the tile of 16 and the segments,
# channels around a block (256 / lanes of a channel), every lane layout (n <= 8, 16, 32, 64) and padded states
CASES = [
    (1, 1, 1, 1, 1, "f32", "f32", False, False, False, False, True),
    (2, 5, 3, 2, 1, "bf16", "bf16", True, True, False, False, True),
    (1, 16, 64, 16, 1, "f32", "f32", True, True, False, False, True),
    (3, 17, 65, 16, 1, "bf16", "f32", True, True, True, True, True),
    (2, 40, 130, 8, 2, "f32", "f32", False, True, False, True, True),
    (2, 33, 36, 32, 4, "bf16", "bf16", True, True, True, False, True),
    (1, 50, 20, 64, 2, "f32", "f32", True, True, False, False, True),
    (2, 70, 9, 23, 3, "f32", "f32", True, False, True, True, False),
    (1, 300, 70, 16, 1, "bf16", "bf16", True, True, False, True, True),
    (4, 200, 24, 12, 2, "f32", "f32", True, True, True, False, True),
    (2, 0, 8, 16, 1, "f32", "f32", True, True, False, False, True),
    (1, 257, 40, 45, 1, "bf16", "f32", False, True, False, False, False),
]


def ids(c):
    return "b%d_L%d_c%d_n%d_g%d_%s_%s%s%s%s%s%s" % (c[:7] + ("_gate" * c[7], "_state" * c[8], "_ragged" * c[9],
                                                         "_sliced" * c[10], "_softplus" * c[11]))


def make(case):
    b, L, c, n, g, dtype, _, gate, state, ragged, sliced, softplus = case
    return inputs(b, L, c, n, g, dtype, gate, state, ragged, sliced, softplus=softplus)


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward(case):
    d = make(case)
    y, fin = fwd(d, y_dtype=TYPES[case[6]], dt_softplus=case[11])
    torch.cuda.synchronize()
    ref, rfin = lo.scan(*[host(d[k]) for k in NAMES], use_softplus=case[11])
    rms = np.sqrt(np.mean(ref ** 2)) if ref.size else 0.0
    assert np.all(np.abs(host(y) - ref) <= TOL * rms * (ref != 0) + (2.0 ** -8 * np.abs(ref) if case[6] == "bf16" else 0))
    assert nerr(host(fin), rfin) <= TOL


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_backward(case):
    d = make(case)
    dy = d["dy"].to(TYPES[case[6]])
    got = bwd(d, dy, dt_softplus=case[11])
    torch.cuda.synchronize()
    a = {k: host(d[k]) for k in NAMES}
    ref = lo.scan_bwd(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], host(dy), a["z"], a["dt_bias"], a["init"],
                      host(d["dfinal"]), a["lengths"], use_softplus=case[11])
    assert set(got) == set(ref)
    errs = {k: nerr(host(got[k]), r) for k, r in ref.items()}
    print(errs)
    assert all(e <= TOL for e in errs.values()), errs
    if d["lengths"] is not None:
        for i, end in enumerate(host(d["lengths"])):
            assert not any(bool(got[k][i, end:].any()) for k in ("dx", "ddt", "dB", "dC"))


@pytest.mark.parametrize("c,n,g", [(1, 1, 1), (70, 16, 1), (36, 8, 2), (20, 32, 4), (9, 64, 3), (33, 21, 1)])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_steps_follow_the_forward_pass(c, n, g, dtype, out):
    d = inputs(3, 7, c, n, g, dtype, sliced=True)
    ref, rfin = lo.scan(*[host(d[k]) for k in NAMES])
    state = d["init"].clone()
    rms = np.sqrt(np.mean(ref ** 2))
    for t in range(7):
        y = ssd.selective_scan_step(d["x"][:, t], d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t], d["D"], state,
                                    d["z"][:, t], d["dt_bias"], y_dtype=TYPES[out])
        r = ref[:, t]
        assert np.all(np.abs(host(y) - r) <= TOL * rms + (2.0 ** -8 * np.abs(r) if out == "bf16" else 0))
    assert nerr(host(state), rfin) <= TOL


def test_long_sequence_of_few_channels():
    # many segments: the states carried across them against the oracle
    d = inputs(1, 3000, 5, 16, gate=False)
    y, fin = fwd(d)
    ref, rfin = lo.scan(*[host(d[k]) for k in NAMES])
    assert nerr(host(y), ref) <= TOL and nerr(host(fin), rfin) <= TOL
    got = bwd(d)
    a = {k: host(d[k]) for k in NAMES}
    r = lo.scan_bwd(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], host(d["dy"]), a["z"], a["dt_bias"], a["init"],
                    host(d["dfinal"]))
    assert all(nerr(host(got[k]), v) <= TOL for k, v in r.items())


def test_rows_behind_the_end_are_not_read():
    d = inputs(4, 90, 24, 16, ragged=True, seed=3)
    clean, gclean = fwd(d), bwd(d)
    bad = dict(d)
    for k in ("x", "dt", "z", "B", "C", "dy"):
        bad[k] = d[k].clone()
        for i, end in enumerate(d["lengths"].tolist()):
            bad[k][i, end:] = float("nan")
    got, ggot = fwd(bad), bwd(bad)
    assert all(torch.equal(p, q) for p, q in zip(got, clean))
    assert all(torch.equal(ggot[k], gclean[k]) for k in gclean)


def test_extreme_steps():
    # steps from 1e-12 to 60: decays of exactly 1 and 0, no NaN
    d = inputs(1, 48, 8, 16, gate=False)
    d["dt"] = torch.linspace(-30, 60, 48, device="cuda")[None, :, None].expand(1, 48, 8).contiguous()
    y, fin = fwd(d)
    ref, rfin = lo.scan(*[host(d[k]) for k in NAMES])
    assert nerr(host(y), ref) <= TOL and nerr(host(fin), rfin) <= TOL
    got = bwd(d)
    assert all(bool(torch.isfinite(v).all()) for v in got.values())


@pytest.mark.parametrize("b,L,c,n", [(2, 5, 8, 16), (1, 301, 40, 16), (2, 37, 12, 6), (1, 20, 9, 40)])
def test_states_that_keep_nothing(b, L, c, n):
    # A of -infinity: exp(d A) = 0 at every token, also where tiles and segments end in rows that take no step
    d = inputs(b, L, c, n, ragged=b > 1, seed=5)
    d["A"][:, ::3] = -float("inf")
    d["A"][0] = -float("inf")
    a = {k: host(d[k]) for k in NAMES}
    a["A"] = np.maximum(a["A"], -1e30)  # as good as infinite, and 0 times it is 0
    y, fin = fwd(d)
    ref, rfin = lo.scan(*[a[k] for k in NAMES])
    assert nerr(host(y), ref) <= TOL and nerr(host(fin), rfin) <= TOL
    got = bwd(d)
    want = lo.scan_bwd(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], host(d["dy"]), a["z"], a["dt_bias"], a["init"],
                       host(d["dfinal"]), a["lengths"])
    errs = {k: nerr(host(got[k]), r) for k, r in want.items()}
    assert all(e <= TOL for e in errs.values()), errs
    state = d["init"].clone()
    row = {k: d[k][:, 0].contiguous() for k in ("x", "dt", "B", "C", "z")}
    y1 = ssd.selective_scan_step(row["x"], row["dt"], d["A"], row["B"], row["C"], d["D"], state, row["z"], d["dt_bias"])
    a1 = dict(a, **{k: a[k][:, :1] for k in ("x", "dt", "B", "C", "z")}, lengths=None)
    ref, rfin = lo.scan(*[a1[k] for k in NAMES])
    assert nerr(host(y1), ref[:, 0]) <= TOL and nerr(host(state), rfin) <= TOL


def test_prompt_in_pieces_with_the_state_in_place():
    d = inputs(2, 400, 24, 16, dtype="bf16")
    want, wfin = fwd(d)
    state = d["init"].clone()
    parts = []
    for t0, t1 in ((0, 1), (1, 18), (18, 200), (200, 400)):
        p = {k: (d[k][:, t0:t1] if k in ("x", "dt", "B", "C", "z") else d[k]) for k in NAMES}
        parts.append(ssd.selective_scan_fwd(p["x"], p["dt"], p["A"], p["B"], p["C"], p["D"], p["z"], p["dt_bias"],
                                            state, final_out=state))
    assert nerr(host(torch.cat(parts, 1)), host(want)) <= TOL and nerr(host(state), host(wfin)) <= TOL


def test_same_call_same_bits():
    d = inputs(2, 300, 70, 16, ragged=True)
    first, again = bwd(d), bwd(d)
    assert all(torch.equal(first[k], again[k]) for k in first)
    assert all(torch.equal(p, q) for p, q in zip(fwd(d), fwd(d)))


def test_optional_inputs_left_out():
    d = inputs(2, 30, 12, 16)
    y = ssd.selective_scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"])
    ref, _ = lo.scan(*[host(d[k]) for k in ("x", "dt", "A", "B", "C")])
    assert nerr(host(y), ref) <= TOL
    got = ssd.selective_scan_bwd(d["x"], d["dt"], d["A"], d["B"], d["C"], None, d["dy"], want_d_initial=False)
    r = lo.scan_bwd(*[host(d[k]) for k in ("x", "dt", "A", "B", "C")], None, host(d["dy"]))
    assert "d_initial_states" not in got and "dz" not in got
    assert all(nerr(host(v), r[k]) <= TOL for k, v in got.items())


def test_refusals_leave_the_outputs():
    d = inputs(2, 8, 12, 16)
    y = torch.full((2, 8, 12), 7.0, device="cuda")
    with pytest.raises(ssd.SSDError, match="UNSUPPORTED"):
        ssd.selective_scan_fwd(d["x"], d["dt"], -torch.ones(12, 65, device="cuda"), torch.ones(2, 8, 1, 65, device="cuda"),
                               torch.ones(2, 8, 1, 65, device="cuda"), out=y)
    with pytest.raises(ssd.SSDError, match="INVALID"):  # 12 channels in 5 groups
        ssd.selective_scan_fwd(d["x"], d["dt"], d["A"], torch.ones(2, 8, 5, 16, device="cuda"),
                               torch.ones(2, 8, 5, 16, device="cuda"), out=y)
    with pytest.raises(ValueError, match="shape"):
        ssd.selective_scan_fwd(d["x"], d["dt"][:, :7], d["A"], d["B"], d["C"], out=y)
    with pytest.raises(TypeError):
        ssd.selective_scan_fwd(d["x"], d["dt"].bfloat16(), d["A"], d["B"], d["C"], out=y)
    with pytest.raises(ssd.SSDError, match="INVALID"):
        ssd.selective_scan_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], out=d["dt"])
    with pytest.raises(ssd.SSDError, match="WORKSPACE"):
        bwd(d, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert bool((y == 7.0).all())


def test_arguments_that_are_no_tensors():
    d = inputs(1, 4, 8, 16)
    for k in ("x", "dt", "A", "B", "C", "z", "dt_bias", "init", "lengths"):
        with pytest.raises(TypeError):
            fwd(dict(d, **{k: 3.0}))
    with pytest.raises(TypeError):
        bwd(d, dy=3.0)


def test_captured_call_replays():
    d = inputs(2, 150, 20, 16, dtype="bf16", ragged=True)
    fwd(d), bwd(d)
    torch.cuda.synchronize()
    state = d["init"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, fin = fwd(d)
        g = bwd(d)
        ys = ssd.selective_scan_step(d["x"][:, 0], d["dt"][:, 0], d["A"], d["B"][:, 0], d["C"][:, 0], d["D"], state,
                                     d["z"][:, 0], d["dt_bias"])
    for k in range(3):
        new = inputs(2, 150, 20, 16, dtype="bf16", seed=50 + k)
        for n in ("x", "dt", "B", "C", "z"):
            d[n].copy_(new[n])
        state.copy_(d["init"])
        graph.replay()
        torch.cuda.synchronize()
        ey, efin = fwd(d)
        e = bwd(d)
        assert torch.equal(y, ey) and torch.equal(fin, efin)
        assert all(torch.equal(g[n], e[n]) for n in e)
        s2 = d["init"].clone()
        want = ssd.selective_scan_step(d["x"][:, 0], d["dt"][:, 0], d["A"], d["B"][:, 0], d["C"][:, 0], d["D"], s2,
                                       d["z"][:, 0], d["dt_bias"])
        assert torch.equal(ys, want) and torch.equal(state, s2)


def test_a_given_stream_runs_the_call():
    d = inputs(2, 300, 30, 16)
    want = bwd(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bwd(d, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_layer_path_prompt_then_tokens():
    # convolution and scan over a ragged prompt, then token by token from their states, against the oracle over
    # prompt and tokens together
    b, L, T, c, n = 3, 37, 5, 48, 16
    d = inputs(b, L + T, c, n, ragged=False, state=False)
    gen = torch.Generator().manual_seed(5)
    w, bias = torch.randn((c, 4), generator=gen).cuda(), torch.randn(c, generator=gen).cuda()
    lengths = torch.tensor([37, 9, 0], dtype=torch.int32, device="cuda")
    cut = {k: d[k][:, :L].contiguous() for k in ("x", "dt", "B", "C", "z")}
    u, cs = ssd.causal_conv_fwd(cut["x"], w, bias, return_final_states=True, lengths=lengths)
    y, hs = ssd.selective_scan_fwd(u, cut["dt"], d["A"], cut["B"], cut["C"], d["D"], cut["z"], d["dt_bias"], None, True,
                                   lengths=lengths)
    outs = []
    for t in range(L, L + T):
        ut = ssd.causal_conv_step(d["x"][:, t], w, bias, cs)
        outs.append(ssd.selective_scan_step(ut, d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t], d["D"], hs,
                                            d["z"][:, t], d["dt_bias"]))
    got = torch.stack(outs, 1)
    for i, end in enumerate([37, 9, 0]):
        pick = list(range(end)) + list(range(L, L + T))
        xi, dti, Bi, Ci, zi = (host(d[k][i:i + 1][:, pick]) for k in ("x", "dt", "B", "C", "z"))
        ui, _ = lo.conv(xi, host(w), host(bias))
        ref, rfin = lo.scan(ui, dti, host(d["A"]), Bi, Ci, host(d["D"]), zi, host(d["dt_bias"]))
        assert nerr(host(got[i]), ref[0, end:]) <= TOL
        assert nerr(host(y[i, :end]), ref[0, :end]) <= TOL
        assert nerr(host(hs[i]), rfin[0]) <= TOL


def test_convolution_before_the_chunked_scan():
    # x, B and C cut from one projection, each through the convolution, then the chunked scan and its backward, the
    # convolution's gradient taking the chunked scan's fp32 one
    b, L, nh, p, g, n = 2, 100, 2, 32, 1, 16
    gen = torch.Generator().manual_seed(8)
    proj = torch.randn((b, L, nh * p + 2 * g * n + nh), generator=gen).cuda()
    cuts = {"x": (0, nh * p), "B": (nh * p, nh * p + g * n), "C": (nh * p + g * n, nh * p + 2 * g * n)}
    w = (0.5 * torch.randn((nh * p + 2 * g * n, 4), generator=gen)).cuda()
    v = {k: ssd.causal_conv_fwd(proj[..., a:z], w[a:z]) for k, (a, z) in cuts.items()}
    dt = torch.nn.functional.softplus(proj[..., -nh:]).contiguous()
    A = -torch.exp(torch.randn(nh, generator=gen)).cuda()
    x4, B4, C4 = v["x"].view(b, L, nh, p), v["B"].view(b, L, g, n), v["C"].view(b, L, g, n)
    y, fin = ssd.chunk_scan_fwd(x4, dt, A, B4, C4, None, chunk_size=64, return_final_states=True)
    ref = {k: lo.conv(host(proj[..., a:z]), host(w[a:z]))[0] for k, (a, z) in cuts.items()}
    import oracle
    yr, fr, _ = oracle.scan(ref["x"].reshape(b, L, nh, p), host(dt), host(A), ref["B"].reshape(b, L, g, n),
                            ref["C"].reshape(b, L, g, n), None, None)
    assert nerr(host(y), yr) <= TOL and nerr(host(fin), fr) <= TOL
    dy = torch.randn((b, L, nh, p), generator=gen).cuda()
    grads = ssd.chunk_scan_bwd(x4, dt, A, B4, C4, None, dy, chunk_size=64)
    for k, name in (("x", "dx"), ("B", "dB"), ("C", "dC")):
        a, z = cuts[k]
        up = grads[name].view(b, L, z - a)
        got = ssd.causal_conv_bwd(proj[..., a:z], w[a:z], None, up)
        want = lo.conv_bwd(host(proj[..., a:z]), host(w[a:z]), None, host(up))
        assert all(nerr(host(got[q]), want[q]) <= TOL for q in want)


def test_interleaved_and_broadcast_rows():
    # (seqlen, batch, channels) storage; B and C of one sequence read by the whole batch; one tensor as two inputs
    d = inputs(3, 45, 20, 16, g=2)
    want, gwant = fwd(d), bwd(d)
    turned = dict(d)
    for k in ("x", "dt", "z", "B", "C", "dy"):
        turned[k] = d[k].transpose(0, 1).contiguous().transpose(0, 1)
        assert not turned[k].is_contiguous()
    got, ggot = fwd(turned), bwd(turned)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert all(torch.equal(ggot[k], gwant[k]) for k in gwant)
    one = dict(d)
    one["B"] = one["C"] = d["B"][:1].expand(3, 45, 2, 16)
    plain = dict(d)
    plain["B"] = plain["C"] = one["B"].contiguous()
    assert all(torch.equal(p, q) for p, q in zip(fwd(one), fwd(plain)))
    g1, g2 = bwd(one), bwd(plain)
    assert all(torch.equal(g1[k], g2[k]) for k in g1)


def test_two_streams_at_once():
    cases = [inputs(2, 500, 64, 16, seed=60 + k) for k in range(2)]
    want = [(fwd(d), bwd(d)) for d in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for k, (d, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[k] = (fwd(d), bwd(d))
    torch.cuda.synchronize()
    for (f, g), (wf, wg) in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(f, wf)) and all(torch.equal(g[k], wg[k]) for k in wg)


def test_offsets_beyond_32_bits():
    # two sequences of 1.15e9 elements each: the second one's results against a call on it alone
    b, L, c, n = 2, 140_000, 8192, 16
    gen = torch.Generator(device="cuda").manual_seed(3)

    def rows(width):
        t = torch.empty((b, L, width), dtype=torch.bfloat16, device="cuda")
        piece = torch.randn((b, 1000, width), generator=gen, device="cuda").bfloat16()
        for t0 in range(0, L, 1000):
            t[:, t0:t0 + 1000] = piece[:, :L - t0]
        return t

    x, dt = rows(c), rows(c)
    B, C = rows(n)[:, :, None], rows(n)[:, :, None]
    A = -torch.arange(1, n + 1, device="cuda").float().expand(c, n).contiguous()
    bias = torch.full((c,), -3.0, device="cuda")
    kw = dict(y_dtype=torch.bfloat16)
    y, fin = ssd.selective_scan_fwd(x, dt, A, B, C, None, None, bias, None, True, **kw)
    y1, fin1 = ssd.selective_scan_fwd(x[1:], dt[1:], A, B[1:], C[1:], None, None, bias, None, True, **kw)
    assert float((y[1:, -4096:].float() - y1[:, -4096:].float()).abs().max()) <= 2.0 ** -7 * float(y1.abs().max())
    assert float((fin[1:] - fin1).norm() / fin1.norm()) < TOL
    del y1
    g = ssd.selective_scan_bwd(x, dt, A, B, C, None, y, None, bias, want_d_initial=True)
    g1 = ssd.selective_scan_bwd(x[1:], dt[1:], A, B[1:], C[1:], None, y[1:], None, bias, want_d_initial=True)
    for k in ("dx", "ddt", "dB", "dC"):
        a, r = g[k][1:, -4096:], g1[k][:, -4096:]
        assert float((a - r).norm() / r.norm()) < TOL, k
    assert float((g["d_initial_states"][1:] - g1["d_initial_states"]).norm() / g1["d_initial_states"].norm()) < TOL


@pytest.mark.parametrize("c,n", [(24, 16), (9, 30), (5, 64)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_last_state_not_finite_leaves_the_rows_behind_it_zero(c, n, value):
    # an overflow at a sequence's last token, or in its final state's gradient
    d = inputs(4, 45, c, n, seed=9)
    d["lengths"] = torch.tensor([45, 19, 3, 0], dtype=torch.int32, device="cuda")
    for i, end in enumerate(d["lengths"].tolist()):
        if end > 0:
            d["x"][i, end - 1, ::2] = value
    d["dfinal"][:, 1::2] = value
    y, got = fwd(d)[0], bwd(d)
    for i, end in enumerate(d["lengths"].tolist()):
        assert bool((y[i, end:] == 0).all())
        assert all(bool((got[k][i, end:] == 0).all()) for k in ("dx", "ddt", "dz", "dB", "dC"))


@pytest.mark.parametrize("c,n", [(24, 16), (9, 30), (5, 64)])
def test_rows_behind_the_end_add_nothing_to_the_sums(c, n):
    # the last token's input overflows the last state, which no gradient of A or of an earlier token contains
    d = inputs(2, 45, c, n, gate=False, seed=10)
    end = 19
    d["dfinal"] = None
    d["x"][:, end - 1] = float("inf")
    d["lengths"] = torch.full((2,), end, dtype=torch.int32, device="cuda")
    got = bwd(d)
    a = {k: host(d[k]) for k in NAMES}
    a["x"][:, end - 1] = 0.0
    want = lo.scan_bwd(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], host(d["dy"]), a["z"], a["dt_bias"], a["init"],
                       None, a["lengths"])
    assert nerr(host(got["dA"]), want["dA"]) <= TOL
    for k in ("dx", "ddt", "dB"):
        assert nerr(host(got[k][:, :end - 1]), want[k][:, :end - 1]) <= TOL, k
    assert nerr(host(got["d_initial_states"]), want["d_initial_states"]) <= TOL


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("b,L,c,n", [(2, 5, 8, 16), (1, 301, 40, 16), (2, 37, 12, 6), (1, 20, 9, 40), (2, 19, 20, 8)])
def test_tokens_without_a_step(b, L, c, n, softplus):
    # d_t = 0, by a dt so low that softplus is 0 or by dt = 0 without it: finite rates keep their state, infinite ones
    # keep nothing, in the prompt, the gradients and the one-token step alike
    d = inputs(b, L, c, n, ragged=b > 1, seed=11, softplus=softplus)
    d["A"][:, ::3] = -float("inf")
    d["A"][0] = -float("inf")
    d["dt_bias"] = None
    none = torch.zeros(L, dtype=torch.bool, device="cuda")
    none[1::3] = none[-1] = True
    low = torch.where(torch.arange(c, device="cuda") % 2 == 0, -200.0, -float("inf")) if softplus else torch.zeros(c, device="cuda")
    d["dt"] = torch.where(none[:, None], low, d["dt"] - 2 if softplus else d["dt"])
    a = {k: host(d[k]) for k in NAMES}
    # the definition's limit: a step too small for anything but an infinite rate
    a["A"] = np.maximum(a["A"], -1e300)
    a["dt"] = np.where(host(none)[:, None], -100.0 if softplus else 1e-60, a["dt"])
    y, fin = fwd(d, dt_softplus=softplus)
    ref, rfin = lo.scan(*[a[k] for k in NAMES], use_softplus=softplus)
    assert nerr(host(y), ref) <= TOL and nerr(host(fin), rfin) <= TOL
    got = bwd(d, dt_softplus=softplus)
    want = lo.scan_bwd(a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], host(d["dy"]), a["z"], a["dt_bias"], a["init"],
                       host(d["dfinal"]), a["lengths"], use_softplus=softplus)
    errs = {k: nerr(host(got[k]), r) for k, r in want.items()}
    assert all(e <= TOL for e in errs.values()), errs
    state = d["init"].clone()
    every, _ = lo.scan(*[a[k] for k in NAMES[:9]], use_softplus=softplus)
    rms = np.sqrt(np.mean(every ** 2))
    for t in range(min(L, 20)):
        yt = ssd.selective_scan_step(d["x"][:, t], d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t], d["D"], state,
                                     d["z"][:, t], None, dt_softplus=softplus)
        assert float(np.max(np.abs(host(yt) - every[:, t]))) <= TOL * rms
    assert bool(torch.isfinite(state).all())


def test_more_gradient_rows_than_a_launch_has_threads():
    # dB and dC of 2^28 numbers each, 17 channels on two blocks: the last sequence against a call on it alone
    b, L, c, n = 64, 65536, 17, 64
    gen = torch.Generator(device="cuda").manual_seed(12)

    def rows(width):
        return torch.randn((b, L, width), generator=gen, device="cuda").bfloat16()

    x, dt, dy = rows(c), rows(c), rows(c)
    B, C = rows(n)[:, :, None], rows(n)[:, :, None]
    A = -torch.arange(1, n + 1, device="cuda").float().expand(c, n).contiguous()
    bias = torch.full((c,), -3.0, device="cuda")
    g = ssd.selective_scan_bwd(x, dt, A, B, C, None, dy, None, bias)
    one = [t[-1:] for t in (x, dt, B, C, dy)]
    g1 = ssd.selective_scan_bwd(one[0], one[1], A, one[2], one[3], None, one[4], None, bias)
    for k in ("dx", "ddt", "dB", "dC"):
        assert float((g[k][-1:] - g1[k]).norm() / g1[k].norm()) < TOL, k
    # dD is a plain sum: over all sequences in 64 bits
    want = (dy.double() * x.double()).sum((0, 1))
    assert float((g["dD"].double() - want).norm() / want.norm()) < TOL


@pytest.mark.parametrize("b,L,c,n", [(1024, 4096, 16, 64), (256, 4096, 260, 16)])
def test_sums_over_long_sequences_do_not_run_off(b, L, c, n):
    # Sequences walked whole, with q = 1 and d constant: dA sums L of 1 + 2^-14 - 2^-20 a sequence, each just below
    # half a step of a sum between 1024 and 2048, and dD as many of 1 + 2^-16 - 2^-22, over the lanes of a channel.
    # A sum in fp32 may take 256 tokens: 256 roundings, by half a step of 2^-24; two a lane step and one at the end.
    one = lambda *shape: torch.ones(shape, device="cuda")  # noqa: E731
    step, grad = 1 + 2.0 ** -14 - 2.0 ** -20, 1 + 2.0 ** -16 - 2.0 ** -22
    none = torch.zeros((1, L, 1, n), device="cuda").expand(b, L, 1, n)
    got = ssd.selective_scan_bwd(one(b, L, c), one(b, L, c) * step, torch.zeros((c, n), device="cuda"), none, none,
                                 None, one(b, L, c) * grad, None, None, one(b, c, n), one(b, c, n), dt_softplus=False)
    for k, want, roundings in (("dA", b * L * step, 256), ("dD", b * L * grad, 256 // (n // 8) + 4)):
        bound = (roundings + 1) * 2.0 ** -24 * want
        assert float((got[k].double() - want).abs().max()) <= bound, k
    assert torch.equal(got["d_initial_states"], one(b, c, n))


def test_softplus_keeps_its_relative_accuracy():
    # one token from a zero state, x = B = C = 1: y is the step size itself.  Roundings of 2^-24: two each for the
    # instructions of the exponential and the logarithm, one each for the exponential's correction, the product with
    # log(2), the bits added back (to first order) and the sum; and 0.05 |v| for log(2) rounded in the correction
    c = 50_000
    dt = torch.linspace(-60, 60, c, device="cuda").view(1, 1, c)
    one, A = torch.ones((1, 1, c), device="cuda"), -torch.ones((c, 1), device="cuda")
    B = torch.ones((1, 1, 1, 1), device="cuda")
    v = dt.double()
    want = v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))
    bound = (8 + 0.05 * v.abs()) * 2.0 ** -24 * want
    y = ssd.selective_scan_fwd(one, dt, A, B, B)
    assert bool(((y.double() - want).abs() <= bound).all())
    state = torch.zeros((1, c, 1), device="cuda")
    y = ssd.selective_scan_step(one[0], dt[0], A, B[0], B[0], None, state)
    assert bool(((y.double() - want[0]).abs() <= bound[0]).all())


def test_softplus_of_numbers_far_out():
    far = torch.tensor([float("inf"), 1e30, -200.0, -1e30, -float("inf"), float("nan")], device="cuda").view(1, 1, 6)
    one, A = torch.ones((1, 1, 6), device="cuda"), -torch.ones((6, 8), device="cuda")
    B = torch.ones((1, 1, 1, 8), device="cuda")
    for y in (ssd.selective_scan_fwd(one, far, A, B, B)[0, 0],
              ssd.selective_scan_step(one[0], far[0], A, B[0], B[0], None, torch.zeros((1, 6, 8), device="cuda"))[0]):
        y = (y / 8).tolist()  # of eight equal states
        assert y[:5] == [float("inf"), far[0, 0, 1].item(), 0.0, 0.0, 0.0] and np.isnan(y[5])


def in_64_bits(d, softplus=True, dy=None):
    """y, the final state and every gradient: the definition in 64 bits, a token of all sequences at a time, and
    differentiated by torch."""
    v = {k: None if d[k] is None else d[k].double().requires_grad_() for k in NAMES[:9]}
    b, L, c = v["x"].shape
    per = c // v["B"].shape[2]
    h = v["init"] if v["init"] is not None else torch.zeros((b, c, v["A"].shape[1]), dtype=torch.float64, device="cuda")
    raw = v["dt"] if v["dt_bias"] is None else v["dt"] + v["dt_bias"]
    step = raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs())) if softplus else raw
    live = torch.ones((b, L, 1), dtype=torch.float64, device="cuda")
    if d["lengths"] is not None:
        live = (torch.arange(L, device="cuda")[None, :] < d["lengths"][:, None]).double()[..., None]
    step = step * live
    ys = []
    for t in range(L):
        dt = step[:, t, :, None]
        h = torch.exp(dt * v["A"]) * h + dt * v["x"][:, t, :, None] * v["B"][:, t].repeat_interleave(per, 1)
        ys.append((v["C"][:, t].repeat_interleave(per, 1) * h).sum(2))
    y = torch.stack(ys, 1) + (0 if v["D"] is None else v["D"] * v["x"])
    if v["z"] is not None:
        y = y * v["z"] * torch.sigmoid(v["z"])
    y = y * live
    loss = (y * (d["dy"] if dy is None else dy).double()).sum()
    if d["dfinal"] is not None:
        loss = loss + (h * d["dfinal"].double()).sum()
    loss.backward()
    names = {"init": "d_initial_states", "dt": "ddt", "dt_bias": "ddt_bias"}
    return y.detach(), h.detach(), {names.get(k, "d" + k): t.grad for k, t in v.items() if t is not None}


# b, L, c, n, g, dtype: batch and channels enough for the waves of the uncut passes (forward from about 1800, backward
# from 4096; batch x blocks of 1024 / (padded states) channels x 4), in every lane layout, with a last block that is
# not full, several tiles, and more tokens than one sum in fp32 takes
UNCUT = [
    (1024, 300, 16, 64, 1, "f32"),
    (64, 100, 1040, 16, 1, "bf16"),
    (64, 41, 1040, 14, 1, "f32"),
    (128, 70, 520, 30, 2, "f32"),
    (64, 50, 2052, 8, 1, "f32"),
]


@pytest.mark.parametrize("case", UNCUT, ids=lambda c: "b%d_L%d_c%d_n%d_g%d_%s" % c)
@pytest.mark.parametrize("full", [True, False])
def test_sequences_walked_whole(case, full):
    b, L, c, n, g, dtype = case
    d = inputs(b, L, c, n, g, dtype, gate=full, state=full, ragged=full, seed=21)
    shape = ssd.SelectiveShape(b, L, c, n, g, ssd.SSD_DTYPE_F32, 0, 1)
    lib = ssd.load_library()
    assert lib.ssd_selective_scan_fwd_workspace_size(ctypes.byref(shape)) == 0  # no segments
    y, fin = fwd(d)
    got = bwd(d)
    ref, rfin, want = in_64_bits(d)

    def err(a, r):
        assert bool(torch.isfinite(a).all())
        rms = r.square().mean().sqrt()
        return float((a.double() - r).abs().max() / rms) if float(rms) > 0 else float(a.abs().max())

    assert err(y, ref) <= TOL and err(fin, rfin) <= TOL
    errs = {k: err(got[k], r) for k, r in want.items()}
    assert all(e <= TOL for e in errs.values()), errs


@pytest.mark.parametrize("b,c,n,g,off", [(3, 130, 21, 2, 0), (2, 96, 35, 3, 0), (2, 70, 61, 2, 0), (3, 12, 7, 4, 0),
                                         (2, 260, 5, 65, 0), (2, 70, 16, 1, 1), (2, 35, 64, 5, 1), (2, 40, 44, 2, 3)])
def test_one_token_of_any_number_of_states(b, c, n, g, off):
    # state counts that are no multiple of four, or states that lie off a 16-byte boundary; groups that end between
    # the channels of one thread
    d = inputs(b, 4, c, n, g, "bf16" if n % 2 else "f32", seed=22)
    room = torch.empty(b * c * n + off, device="cuda")
    state = room[off:].view(b, c, n)
    state.copy_(d["init"])
    ref, rfin = lo.scan(*[host(d[k]) for k in NAMES])
    rms = np.sqrt(np.mean(ref ** 2))
    for t in range(4):
        y = ssd.selective_scan_step(d["x"][:, t], d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t], d["D"], state,
                                    d["z"][:, t], d["dt_bias"])
        assert float(np.max(np.abs(host(y) - ref[:, t]))) <= TOL * rms
    assert nerr(host(state), rfin) <= TOL
