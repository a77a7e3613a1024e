"""The measured calls of two operator families: the short causal convolution
and the selective scan with a decay per channel and state, each over prompts,
backwards, and for a single token.

``run`` computes a case in its plain form (elementary torch operations in 32
bits) or, where ``own`` is true, through the library's entry points; ``exact``
computes it from the definition in 64 bits, gradients by differentiating that
definition.

A case's keys:
  op        conv_fwd, conv_bwd, conv_step, scan_fwd, scan_bwd, scan_step
  batch, seqlen, channels; width (conv); dstate, ngroups (scan)
  dtype     "bf16" or "f32": x and what is stored like it
  out       type of y and dy, and of the convolution's dx
  silu      convolution: SiLU after the sum
  gate      scan: y is multiplied by SiLU(z)
  ragged    sequences of different lengths, padded to seqlen
  carry     an initial state is given and the final state returned (backwards:
            its gradient is given and the initial state's returned)
  sliced    inputs are column slices of wider projections, as a layer has them
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _conv(op, batch, seqlen, channels, width=4, dtype="bf16", out="bf16", silu=True, ragged=False, carry=False,
          sliced=False):
    return dict(op=op, batch=batch, seqlen=seqlen, channels=channels, width=width, dtype=dtype, out=out, silu=silu,
                ragged=ragged, carry=carry, sliced=sliced)


def _scan(op, batch, seqlen, channels, dstate=16, ngroups=1, dtype="bf16", out="bf16", gate=True, ragged=False,
          carry=False, sliced=False):
    return dict(op=op, batch=batch, seqlen=seqlen, channels=channels, dstate=dstate, ngroups=ngroups, dtype=dtype,
                out=out, gate=gate, ragged=ragged, carry=carry, sliced=sliced)


def listed():
    return [
        # x, B and C of the throughput layer (80 heads of 64, one group of state 128: 5376 channels), 8 x 4096
        # tokens, a slice of the layer's input projection
        dict(_conv("conv_fwd", 8, 4096, 5376, sliced=True), name="conv_fwd_throughput"),
        # ragged prompts continued from earlier states, fp32, an odd channel count, no activation
        dict(_conv("conv_fwd", 3, 517, 771, 3, "f32", "f32", silu=False, ragged=True, carry=True),
             name="conv_fwd_ragged_f32"),
        # training of the 2.7B-shaped layer: dy in fp32 as the chunked scan's backward gives it, dx for the
        # projection's backward in bf16
        dict(_conv("conv_bwd", 2, 2048, 5376, sliced=True), name="conv_bwd_layer"),
        # a small fp32 training step over padded sequences, truncated in time (states and their gradients)
        dict(_conv("conv_bwd", 3, 1021, 264, 4, "f32", "f32", ragged=True, carry=True), name="conv_bwd_ragged_f32"),
        # one token of one sequence: latency alone
        dict(_conv("conv_step", 1, 1, 5376), name="conv_step_one"),
        # one token of 128 sequences, the serving batch
        dict(_conv("conv_step", 128, 1, 5376), name="conv_step_batch"),
        # a prompt or training forward of a layer of 5120 channels, gated, B, C and z as slices of projections
        dict(_scan("scan_fwd", 2, 2048, 5120, sliced=True), name="scan_fwd_layer"),
        # one long document with few channels: the work lies along the time axis
        dict(_scan("scan_fwd", 1, 8191, 771, 16, 1, "f32", "f32", gate=False, carry=True), name="scan_fwd_long_f32"),
        # training of the layer of 5120 channels
        dict(_scan("scan_bwd", 2, 2048, 5120, sliced=True), name="scan_bwd_layer"),
        # padded sequences, grouped B and C, a state of another size, fp32
        dict(_scan("scan_bwd", 3, 333, 264, 24, 2, "f32", "f32", ragged=True, carry=True), name="scan_bwd_ragged_f32"),
        # one token of one sequence
        dict(_scan("scan_step", 1, 1, 5120), name="scan_step_one"),
        # one token of 128 sequences: the state streams through memory once
        dict(_scan("scan_step", 128, 1, 5120), name="scan_step_batch"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Batches 1..8 (1..256 for one token), lengths 1..8192 (4096 backwards), 1..8192 channels, widths 2..4, states
    of 1..64, both types, every switch; bounded by the elements of the largest listed case of its kind."""
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd", "scan_step"])
    dtype = rng.choice(["bf16", "f32"])
    out = dtype if rng.random() < 0.6 else "f32"
    channels = _log(rng, 1, 8192)
    if rng.random() < 0.5:  # a model's channel counts are mostly multiples of 64
        channels = max(64, channels // 64 * 64)
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op.endswith("step"):
        batch, seqlen = _log(rng, 1, 256), 1
        if op == "scan_step":
            batch = min(batch, max(1, (128 * 5120) // channels))
    else:
        batch = rng.randint(1, 8)
        seqlen = _log(rng, 1, 4096 if op.endswith("bwd") else 8192)
        most = {"conv_fwd": 4 * 4096 * 5376, "conv_bwd": 2 * 2048 * 5376, "scan_fwd": 2 * 2048 * 5120,
                "scan_bwd": 2 * 2048 * 5120 // 2}[op]
        channels = max(1, min(channels, most // (batch * seqlen)))
    if op.startswith("conv"):
        return _conv(op, batch, seqlen, channels, rng.randint(2, 4), dtype, out, flip(), flip() and seqlen > 1, flip(),
                     flip())
    ngroups = rng.choice([g for g in (1, 1, 2, 4) if channels % g == 0])
    dstate = 16 if flip() else rng.randint(1, 64)
    room = 2 * 2048 * 5120 * 16 // 2
    if op != "scan_step" and batch * seqlen * channels * dstate > room:
        dstate = max(1, room // (batch * seqlen * channels))
    return _scan(op, batch, seqlen, channels, dstate, ngroups, dtype, out, flip(), flip() and seqlen > 1, flip(),
                 flip())


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rows(gen, shape, dtype, sliced, off):
    """N(0, 1) rows; where sliced, columns off.. of a wider projection (as an input projection's output is cut)."""
    if not sliced:
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)
    wide = list(shape)
    wide[-1] = off + shape[-1] + 64
    return torch.randn(wide, generator=gen, device="cuda").to(dtype)[..., off:off + shape[-1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    b, L, c = case["batch"], case["seqlen"], case["channels"]
    dt_in, dt_out = TYPES[case["dtype"]], TYPES[case["out"]]
    step = case["op"].endswith("step")
    lead = (b,) if step else (b, L)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = {"case": case, "lengths": None}
    if case["ragged"]:
        lengths = torch.randint(0, L + 1, (b,), generator=gen, device="cuda", dtype=torch.int32)
        lengths[0] = L
        if b > 2:
            lengths[b - 1] = 0  # a slot of the batch that holds no prompt
        s["lengths"] = lengths
    s["x"] = _rows(gen, lead + (c,), dt_in, case["sliced"], 64)
    if case["op"].startswith("conv"):
        w = case["width"]
        s["weight"] = randn(c, w) / math.sqrt(w)
        s["bias"] = 0.1 * randn(c)
        if step or case["carry"]:
            s["init"] = randn(b, w - 1, c).to(dt_in)
        else:
            s["init"] = None
        if case["op"] == "conv_bwd":
            # dy of the case in fp32 where the scan's backward gives it, dx in the projection's type
            s["dy"] = randn(b, L, c) if case["sliced"] else randn(b, L, c).to(dt_out)
            s["dfinal"] = randn(b, w - 1, c) if case["carry"] else None
        return s
    n, g = case["dstate"], case["ngroups"]
    s["dt"] = (0.5 * randn(*lead, c)).to(dt_in)
    s["A"] = -torch.arange(1, n + 1, device="cuda", dtype=torch.float32) * torch.exp(0.1 * randn(c, n))
    if case["sliced"]:
        # one projection gives the step size's factors, B and C side by side
        proj = randn(*lead, 32 + 2 * g * n).to(dt_in)
        s["B"] = proj[..., 32:32 + g * n].unflatten(-1, (g, n))
        s["C"] = proj[..., 32 + g * n:].unflatten(-1, (g, n))
    else:
        s["B"], s["C"] = randn(*lead, g, n).to(dt_in), randn(*lead, g, n).to(dt_in)
    s["D"] = randn(c)
    s["z"] = _rows(gen, lead + (c,), dt_in, case["sliced"], 128) if case["gate"] else None
    # softplus of the bias is log-uniform in [0.001, 0.1]
    steps = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand((c,), generator=gen, device="cuda"))
    s["dt_bias"] = steps + torch.log(-torch.expm1(-steps))
    s["init"] = 0.5 * randn(b, c, n) if step or case["carry"] else None
    if case["op"] == "scan_bwd":
        s["dy"] = randn(b, L, c).to(dt_out)
        s["dfinal"] = randn(b, c, n) if case["carry"] else None
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _live(s):
    """(b, L, 1) truth of the tokens that belong to a sequence, or None where all do."""
    if s["lengths"] is None:
        return None
    t = torch.arange(s["case"]["seqlen"], device="cuda")
    return (t[None, :] < s["lengths"][:, None])[..., None]


def _window(s):
    """Initial state and x in one row of time, fp32: row width - 1 + t is x_t."""
    c, x = s["case"], s["x"].float()
    if s["init"] is None:
        head = x.new_zeros((c["batch"], c["width"] - 1, c["channels"]))
    else:
        head = s["init"].float()
    return torch.cat([head, x], 1)


def _state_rows(s):
    """Indexes (b, width - 1) into the window of each sequence's last inputs."""
    c = s["case"]
    k = torch.arange(c["width"] - 1, device="cuda")
    ends = s["lengths"].long() if s["lengths"] is not None else torch.full((c["batch"],), c["seqlen"], device="cuda")
    return ends[:, None] + k[None, :]


def _presum(s, win):
    c = s["case"]
    pre = s["bias"].expand(c["batch"], c["seqlen"], c["channels"])
    for k in range(c["width"]):
        pre = pre + s["weight"][:, k] * win[:, k:k + c["seqlen"]]
    return pre


def _plain_conv_fwd(s):
    c = s["case"]
    win = _window(s)
    y = _presum(s, win)
    if c["silu"]:
        y = y / (1 + torch.exp(-y))
    live = _live(s)
    if live is not None:
        y = torch.where(live, y, 0.0)
    y = y.to(TYPES[c["out"]])
    if not c["carry"]:
        return [y]
    rows = torch.arange(c["batch"], device="cuda")[:, None]
    return [y, win[rows, _state_rows(s)].to(TYPES[c["dtype"]])]


def _plain_conv_bwd(s):
    c = s["case"]
    L, w = c["seqlen"], c["width"]
    win = _window(s)
    dpre = s["dy"].float()
    if c["silu"]:
        pre = _presum(s, win)
        sig = 1 / (1 + torch.exp(-pre))
        dpre = dpre * sig * (1 + pre * (1 - sig))
    live = _live(s)
    if live is not None:
        dpre = torch.where(live, dpre, 0.0)
    dwin = torch.zeros_like(win)
    for k in range(w):
        dwin[:, k:k + L] += s["weight"][:, k] * dpre
    if s["dfinal"] is not None:
        rows = torch.arange(c["batch"], device="cuda")[:, None]
        at = _state_rows(s)
        dwin[rows, at] = dwin[rows, at] + s["dfinal"]
    # long sums in 64 bits
    dweight = torch.stack([(dpre * win[:, k:k + L]).sum((0, 1), dtype=torch.float64) for k in range(w)], 1).float()
    dbias = dpre.sum((0, 1), dtype=torch.float64).float()
    got = [dwin[:, w - 1:].to(TYPES[c["out"]]), dweight, dbias]
    return got + [dwin[:, :w - 1].clone()] if c["carry"] else got


def _plain_conv_step(s):
    c = s["case"]
    win = torch.cat([s["init"].float(), s["x"].float()[:, None]], 1)
    y = s["bias"].expand(c["batch"], c["channels"])
    for k in range(c["width"]):
        y = y + s["weight"][:, k] * win[:, k]
    if c["silu"]:
        y = y / (1 + torch.exp(-y))
    s["init"].copy_(win[:, 1:])
    return [y.to(TYPES[c["out"]]), s["init"]]


def _steps(s):
    """Step sizes after bias and softplus; 0 behind a sequence's end, where the state stays as it is."""
    raw = s["dt"].float() + s["dt_bias"]
    d = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw)))
    live = None if s["case"]["op"] == "scan_step" else _live(s)
    return raw, d if live is None else torch.where(live, d, 0.0)


def _grouped(s, v):
    """(b, L, channels) as (b, L, groups, channels of a group, 1), beside B and C as (b, L, groups, 1, states)."""
    return v.unflatten(2, (s["case"]["ngroups"], -1))[..., None]


def _recur(decay, put, first):
    """h_t = decay_t h_{t-1} + put_t along dim 1 from h = first, for all t at once: runs of about sqrt(L) tokens beside
    each other, then the runs one after the other.  Overwrites both; returns every state."""
    L = put.shape[1]
    run = max(1, math.isqrt(L))
    cuts = range(run, L, run)
    for k in range(1, run):
        put[:, k::run] += decay[:, k::run] * put[:, k - 1::run][:, :put[:, k::run].shape[1]]
        decay[:, k::run] *= decay[:, k - 1::run][:, :decay[:, k::run].shape[1]]
    h = first
    for t in (0, *cuts):
        put[:, t:t + run] += decay[:, t:t + run] * h[:, None]
        h = put[:, min(t + run, L) - 1]
    return put


def _plain_states(s):
    """Step sizes, x, the initial state and every state h_t, (b, L, groups, channels of a group, states)."""
    c = s["case"]
    b, d, n, g = c["batch"], c["channels"], c["dstate"], c["ngroups"]
    _, step = _steps(s)
    x = s["x"].float()
    first = s["init"].unflatten(1, (g, -1)) if s["init"] is not None else x.new_zeros((b, g, d // g, n))
    decay = torch.exp(_grouped(s, step) * s["A"].unflatten(0, (g, -1)))
    return step, x, first, _recur(decay, _grouped(s, step * x) * s["B"].float()[:, :, :, None], first)


def _readout(s, hs):
    return (hs * s["C"].float()[:, :, :, None]).sum(-1).flatten(2)


def _plain_scan_fwd(s):
    c = s["case"]
    _, x, _, hs = _plain_states(s)
    y = _readout(s, hs) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z / (1 + torch.exp(-z))
    live = _live(s)
    if live is not None:
        y = torch.where(live, y, 0.0)
    y = y.to(TYPES[c["out"]])
    return [y, hs[:, -1].flatten(1, 2)] if c["carry"] else [y]


def _plain_scan_bwd(s):
    c = s["case"]
    g = c["ngroups"]
    step, x, first, hs = _plain_states(s)
    dy = s["dy"].float()
    live = _live(s)
    if live is not None:
        dy = torch.where(live, dy, 0.0)
    got = {}
    if s["z"] is not None:
        z = s["z"].float()
        sig = 1 / (1 + torch.exp(-z))
        got["dz"] = dy * (_readout(s, hs) + s["D"] * x) * sig * (1 + z * (1 - sig))
        dy = dy * z * sig
    A = s["A"].unflatten(0, (g, -1))
    decay = torch.exp(_grouped(s, step) * A)
    # the state's gradient runs backwards: G_t = C_t dy_t + decay_{t+1} G_{t+1}
    last = s["dfinal"].unflatten(1, (g, -1)) if s["dfinal"] is not None else torch.zeros_like(first)
    after = torch.cat([torch.ones_like(decay[:, :1]), decay.flip(1)[:, :-1]], 1)
    G = _recur(after, (_grouped(s, dy) * s["C"].float()[:, :, :, None]).flip(1), last).flip(1)
    got["dC"] = (hs * _grouped(s, dy)).sum(3)
    got["dB"] = (G * _grouped(s, step * x)).sum(3)
    gB = (G * s["B"].float()[:, :, :, None]).sum(-1).flatten(2)
    got["dx"] = gB * step + s["D"] * dy
    G *= decay
    if c["carry"]:
        got["d_initial_states"] = G[:, 0].flatten(1, 2).clone()
    # times the state before each token: the gradient of decay_t, as one of the exponent
    G[:, 1:] *= hs[:, :-1]
    G[:, 0] *= first
    raw, _ = _steps(s)
    ddt = ((G * A).sum(-1).flatten(2) + gB * x) / (1 + torch.exp(-raw))
    got["ddt"] = ddt if live is None else torch.where(live, ddt, 0.0)
    got["dA"] = (G * _grouped(s, step)).sum((0, 1), dtype=torch.float64).flatten(0, 1).float()
    got["dD"] = (dy * x).sum((0, 1), dtype=torch.float64).float()
    got["ddt_bias"] = got["ddt"].sum((0, 1), dtype=torch.float64).float()
    return got


def _plain_scan_step(s):
    c = s["case"]
    g = c["ngroups"]
    _, step = _steps(s)
    x = s["x"].float()
    decay = torch.exp(step[..., None] * s["A"]).unflatten(1, (g, -1))
    put = (step * x).unflatten(1, (g, -1))[..., None] * s["B"].float()[:, :, None]
    h = decay * s["init"].unflatten(1, (g, -1)) + put
    y = (h * s["C"].float()[:, :, None]).sum(-1).flatten(1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z / (1 + torch.exp(-z))
    s["init"].copy_(h.flatten(1, 2))
    return [y.to(TYPES[c["out"]]), s["init"]]


_PLAIN = {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step,
          "scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step}


def _lib():
    import mamba_chunked_ssd_amd as ssd
    return ssd


def _act(c):
    return "silu" if c["silu"] else None


def _own_conv_fwd(s):
    c = s["case"]
    got = _lib().causal_conv_fwd(s["x"], s["weight"], s["bias"], s["init"], c["carry"], activation=_act(c),
                                 lengths=s["lengths"], y_dtype=TYPES[c["out"]])
    return list(got) if c["carry"] else [got]


def _own_conv_bwd(s):
    c = s["case"]
    g = _lib().causal_conv_bwd(s["x"], s["weight"], s["bias"], s["dy"], s["init"], s["dfinal"], activation=_act(c),
                               lengths=s["lengths"], dx_dtype=TYPES[c["out"]], want_d_initial=c["carry"])
    got = [g["dx"], g["dweight"], g["dbias"]]
    return got + [g["d_initial_states"]] if c["carry"] else got


def _own_conv_step(s):
    c = s["case"]
    y = _lib().causal_conv_step(s["x"], s["weight"], s["bias"], s["init"], activation=_act(c),
                                y_dtype=TYPES[c["out"]])
    return [y, s["init"]]


def _own_scan_fwd(s):
    c = s["case"]
    got = _lib().selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["init"],
                                    c["carry"], dt_softplus=True, lengths=s["lengths"], y_dtype=TYPES[c["out"]])
    return list(got) if c["carry"] else [got]


def _own_scan_bwd(s):
    c = s["case"]
    return _lib().selective_scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dy"], s["z"], s["dt_bias"],
                                     s["init"], s["dfinal"], dt_softplus=True, lengths=s["lengths"],
                                     want_d_initial=c["carry"])


def _own_scan_step(s):
    c = s["case"]
    y = _lib().selective_scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["init"], s["z"], s["dt_bias"],
                                   dt_softplus=True, y_dtype=TYPES[c["out"]])
    return [y, s["init"]]


_OWN = {"conv_fwd": _own_conv_fwd, "conv_bwd": _own_conv_bwd, "conv_step": _own_conv_step,
        "scan_fwd": _own_scan_fwd, "scan_bwd": _own_scan_bwd, "scan_step": _own_scan_step}


# ---------------------------------------------------------------------------
# What a pass cannot do without, and its exact outputs
# ---------------------------------------------------------------------------

def work(case):
    b, L, c = case["batch"], case["seqlen"], case["channels"]
    i, o = (2 if case["dtype"] == "bf16" else 4), (2 if case["out"] == "bf16" else 4)
    t = b * L * c
    op = case["op"]
    if op.startswith("conv"):
        w = case["width"]
        held = b * (w - 1) * c
        params = 4 * c * (w + 1)
        sums = 2 * w + (4 if case["silu"] else 0)
        if op == "conv_step":
            return {"bytes": t * (i + o) + 2 * held * i + params, "flops": t * sums}
        if op == "conv_fwd":
            return {"bytes": t * (i + o) + (2 * held * i if case["carry"] else 0) + params, "flops": t * sums}
        dy = 4 if case["sliced"] else o
        return {"bytes": t * (i + dy + o) + (held * (i + 8) if case["carry"] else 0) + 2 * params,
                "flops": t * (6 * w + 1 + (9 if case["silu"] else 0))}
    n, g = case["dstate"], case["ngroups"]
    rows = t * i * (3 if case["gate"] else 2) + 2 * b * L * g * n * i
    held = 4 * b * c * n
    params = 4 * c * (n + 2)
    # per state: the decay's product and exponential, the input's product, the update, the readout
    if op == "scan_step":
        return {"bytes": rows + t * o + 2 * held + params, "flops": 7 * t * n}
    if op == "scan_fwd":
        return {"bytes": rows + t * o + (2 * held if case["carry"] else 0) + params, "flops": 7 * t * n}
    grads = t * 4 * (3 if case["gate"] else 2) + 2 * b * L * g * n * 4
    # the states again (5), then the adjoint, the five sums it enters and the decay's gradient (14)
    return {"bytes": rows + t * o + grads + (3 * held if case["carry"] else 0) + 2 * params, "flops": 19 * t * n}


def _exact_conv(x, weight, bias, init, ends, silu):
    """Every output and the final state by the definition, one tap and one sequence at a time."""
    b, L, c = x.shape
    w = weight.shape[1]
    ys, finals = [], []
    for i in range(b):
        end = ends[i]
        line = torch.cat([init[i], x[i, :end]]) if init is not None else torch.nn.functional.pad(
            x[i, :end], (0, 0, w - 1, 0))
        acc = torch.zeros((end, c), dtype=torch.float64, device=x.device)
        for k in range(w):
            acc = acc + line[k:k + end] * weight[:, k]
        acc = acc + bias
        if silu:
            acc = acc * torch.sigmoid(acc)
        ys.append(torch.nn.functional.pad(acc, (0, 0, 0, L - end)))
        finals.append(line[end:])
    return torch.stack(ys), torch.stack(finals)


def _exact_scan(x, dt, A, B, C, D, z, bias, init, ends):
    """The recurrence as it is defined, a token of all sequences at a time; a sequence past its end stays."""
    b, L, c = x.shape
    per = c // B.shape[2]
    h = init if init is not None else torch.zeros((b, c, A.shape[1]), dtype=torch.float64, device=x.device)
    last = torch.tensor(ends, device=x.device)
    ragged = any(e < L for e in ends)
    ys = []
    for t in range(L):
        on = (t < last)[:, None]
        d = torch.nn.functional.softplus(dt[:, t] + bias, threshold=50)
        if ragged:
            d = d * on
        Bt, Ct = (m[:, t].repeat_interleave(per, 1) for m in (B, C))
        h = torch.exp(d[:, :, None] * A) * h + (d * x[:, t])[:, :, None] * Bt
        y = (Ct * h).sum(2) + D * x[:, t]
        if z is not None:
            y = y * z[:, t] * torch.sigmoid(z[:, t])
        ys.append(y * on if ragged else y)
    return torch.stack(ys, 1), h


def exact(case, seed):
    s = prepare(case, seed)
    op, step = case["op"], case["op"].endswith("step")
    backwards = op.endswith("bwd")
    if op == "scan_bwd" and case["batch"] * case["seqlen"] * case["channels"] * case["dstate"] > 1.4e9:
        return None  # the graph of that many states in 64 bits is too large
    ends = [case["seqlen"]] * case["batch"] if s["lengths"] is None else s["lengths"].tolist()
    names = ["x", "weight", "bias", "init"] if op.startswith("conv") else [
        "x", "dt", "A", "B", "C", "D", "z", "dt_bias", "init"]
    v = {k: None if s[k] is None else s[k].double().clone().requires_grad_(backwards) for k in names}
    seq = dict(v)
    if step:
        for k in ("x", "dt", "B", "C", "z"):
            if seq.get(k) is not None:
                seq[k] = seq[k][:, None]
    if op.startswith("conv"):
        y, final = _exact_conv(*[seq[k] for k in names], ends, case["silu"])
    else:
        y, final = _exact_scan(*[seq[k] for k in names], ends)
    if not backwards:
        y, final = y.detach(), final.detach()
        if step:
            return [y[:, 0], final]
        return [y, final] if case["carry"] else [y]
    loss = (y * s["dy"].double()).sum()
    if s["dfinal"] is not None:
        loss = loss + (final * s["dfinal"].double()).sum()
    loss.backward()
    if op == "conv_bwd":
        got = [v["x"].grad, v["weight"].grad, v["bias"].grad]
        return got + [v["init"].grad] if case["carry"] else got
    got = {"dx": v["x"].grad, "ddt": v["dt"].grad, "dA": v["A"].grad, "dB": v["B"].grad, "dC": v["C"].grad,
           "dD": v["D"].grad, "ddt_bias": v["dt_bias"].grad}
    if case["gate"]:
        got["dz"] = v["z"].grad
    if case["carry"]:
        got["d_initial_states"] = v["init"].grad
    return got
