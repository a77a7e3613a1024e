"""The measured calls of two more operator families: sliding-window attention
with sinks (over prompts, backwards, and for a single token) and the
root-mean-square norm with the residual's addition (forward, also with 8-bit
outputs and scales, and backwards).

``run`` computes a case in its plain form (elementary torch operations in 32
bits) or, where ``own`` is true, through the library's entry points; ``exact``
computes it from the definition in 64 bits, gradients by differentiating that
definition.

A case's keys:
  op        norm_fwd, norm_bwd, attn_fwd, attn_bwd, attn_step
  batch, seqlen
  dtype     "bf16" or "f32": x of the norm, everything of the attention
  ragged    sequences of different lengths, padded to seqlen
  sliced    inputs are column slices of wider projections, as a layer has them
norm:
  channels
  stream    type of the residual stream, "" for none
  out       type of y (dy backwards), or "e4m3"
  block     columns that share a scale of an e4m3 output, 0 for the whole row
attention:
  heads, kvheads, headdim, window, sinks
  carry     prompts: the cache of earlier tokens is read and brought up to date
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
EPS = 1e-5
E4M3_MAX = 448.0


def _norm(op, batch, seqlen, channels, dtype="bf16", stream="f32", out="bf16", block=0, ragged=False, sliced=False):
    return dict(op=op, batch=batch, seqlen=seqlen, channels=channels, dtype=dtype, stream=stream, out=out, block=block,
                ragged=ragged, sliced=sliced)


def _attn(op, batch, seqlen, heads, kvheads, headdim, window, sinks, dtype="bf16", ragged=False, sliced=False,
          carry=False):
    return dict(op=op, batch=batch, seqlen=seqlen, heads=heads, kvheads=kvheads, headdim=headdim, window=window,
                sinks=sinks, dtype=dtype, ragged=ragged, sliced=sliced, carry=carry)


def listed():
    return [
        # before the input projection of the 2.7B-shaped layer, 8 x 4096 tokens, activations in 8 bits for that product
        dict(_norm("norm_fwd", 8, 4096, 2560, out="e4m3", block=128), name="norm_fwd_throughput_8bit"),
        # padded fp32 sequences without a residual, an odd channel count
        dict(_norm("norm_fwd", 3, 517, 771, "f32", "", "f32", ragged=True, sliced=True), name="norm_fwd_ragged_f32"),
        # one token of one sequence, a scale for the row: latency alone
        dict(_norm("norm_fwd", 1, 1, 2560, out="e4m3"), name="norm_fwd_one_8bit"),
        # training of the 2.7B-shaped layer with its residual stream in fp32
        dict(_norm("norm_bwd", 2, 2048, 2560), name="norm_bwd_layer"),
        # a small fp32 training step over padded sequences
        dict(_norm("norm_bwd", 3, 1021, 264, "f32", "f32", "f32", ragged=True), name="norm_bwd_ragged_f32"),
        # a prompt or training forward of a layer of 2560 channels: 40 heads of 64, 8 of them for keys and values,
        # cut out of one projection
        dict(_attn("attn_fwd", 2, 2048, 40, 8, 64, 512, 4, sliced=True), name="attn_fwd_layer"),
        # one long document with wide heads
        dict(_attn("attn_fwd", 1, 16384, 8, 2, 128, 2048, 16), name="attn_fwd_long"),
        # padded fp32 pieces of prompts whose earlier tokens lie in the cache
        dict(_attn("attn_fwd", 3, 333, 6, 2, 64, 100, 3, "f32", ragged=True, carry=True), name="attn_fwd_carry_f32"),
        # training of the layer of 40 heads
        dict(_attn("attn_bwd", 2, 2048, 40, 8, 64, 512, 4, sliced=True), name="attn_bwd_layer"),
        # padded fp32 sequences, one head of keys for all, a window that is no multiple of anything
        dict(_attn("attn_bwd", 3, 257, 4, 1, 32, 75, 5, "f32", ragged=True), name="attn_bwd_ragged_f32"),
        # one token of one sequence, whose cache is the only work
        dict(_attn("attn_step", 1, 1, 40, 8, 64, 2048, 4), name="attn_step_one"),
        # one token of 128 sequences, the serving batch: the caches stream through memory once
        dict(_attn("attn_step", 128, 1, 40, 8, 64, 2048, 4), name="attn_step_batch"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Norms of 1..8 x 1..8192 rows of 1..16384 channels, every pair of types; attention of 1..8 x 1..8192 tokens (4096
    backwards) and of 1..256 single tokens, 1..48 heads in groups of 1..12, windows of 1..8192 (4096 for one token),
    0..128 sinks; bounded by the work of the largest listed case of its kind."""
    flip = lambda p=0.5: rng.random() < p  # noqa: E731
    op = rng.choice(["norm_fwd", "norm_bwd", "attn_fwd", "attn_bwd", "attn_step"])
    dtype = rng.choice(["bf16", "f32"])
    if op.startswith("norm"):
        batch, seqlen, channels = rng.randint(1, 8), _log(rng, 1, 8192), _log(rng, 1, 16384)
        if flip():  # a model's channel counts are mostly multiples of 64
            channels = max(64, channels // 64 * 64)
        most = 8 * 4096 * 2560 if op == "norm_fwd" else 2 * 2048 * 2560
        seqlen = max(1, min(seqlen, most // (batch * channels)))
        stream = rng.choice(["", dtype, "f32"])
        out = rng.choice([dtype, "f32", "e4m3", "e4m3"] if op == "norm_fwd" else [dtype, "f32"])
        block = rng.choice([0, 32, 64, 128]) if out == "e4m3" else 0
        return _norm(op, batch, seqlen, channels, dtype, stream, out, block, flip() and seqlen > 1, flip())
    headdim = rng.choice([32, 64, 128])
    kvheads = rng.randint(1, 8)
    heads = kvheads * rng.choice([1, 1, 2, 3, 4, 5, 8, 12])
    heads = heads if heads <= 48 else kvheads * 4
    sinks = rng.choice([0, 1, 4, rng.randint(0, 128)])
    if op == "attn_step":
        window = _log(rng, 1, 4096)
        room = 128 * 8 * 64 * 2052 * (2 if dtype == "bf16" else 1) // 2
        batch = max(1, min(_log(rng, 1, 256), room // (kvheads * headdim * (window + sinks))))
        return _attn(op, batch, 1, heads, kvheads, headdim, window, sinks, dtype, sliced=flip())
    batch = rng.randint(1, 8)
    seqlen = _log(rng, 1, 8192 if op == "attn_fwd" else 4096)
    most = (8 * 16384 * 2048 * 128 if op == "attn_fwd" else 2 * 40 * 2048 * 512 * 64) // (1 if dtype == "bf16" else 8)
    # the plain form holds every pair of tokens of every head
    pairs = 8 * 16384 ** 2 if op == "attn_fwd" else 2 * 40 * 2048 ** 2
    while seqlen > 1 and (batch * heads * seqlen ** 2 > pairs or batch * heads * seqlen * headdim * min(seqlen, 256) > most):
        seqlen = seqlen * 3 // 4
    window = _log(rng, 1, max(2, min(8192, most // (batch * heads * seqlen * headdim))))
    return _attn(op, batch, seqlen, heads, kvheads, headdim, window, sinks, dtype, flip() and seqlen > 1, flip(),
                 op == "attn_fwd" and flip())


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """Tokens of each sequence: the first whole, shorter ones after it, the last slot of three or more holds none."""
    b, L = case["batch"], case["seqlen"]
    if not case["ragged"]:
        return [L] * b
    return [0 if b > 2 and i == b - 1 else L - (L * i * 3) // (b * 4) for i in range(b)]


def _positions(case):
    """Tokens that each sequence has behind it: none, less than the cache's slots, or many times as many."""
    b, slots = case["batch"], case["window"] + case["sinks"]
    if case["op"] == "attn_step":
        # a slot of the batch that holds no sequence
        return [-1 if b > 2 and i == b - 1 else (3 * slots + 1) * (i + 1) // b for i in range(b)]
    return [(5 * slots * i) // (2 * b) for i in range(b)] if case["carry"] else [0] * b


def _tokens(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    b, L, t = case["batch"], case["seqlen"], TYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = {"case": case, "lengths": _tokens(_lengths(case)) if case["ragged"] else None}
    if case["op"].startswith("norm"):
        c, stream = case["channels"], TYPES.get(case["stream"])
        # channels of different size, a few of them outliers, as a residual stream's are
        size = torch.exp(0.5 * randn(c)) * torch.where(torch.rand((c,), generator=gen, device="cuda") < 0.01, 8.0, 1.0)
        s["weight"] = 1 + 0.2 * randn(c)
        if case["op"] == "norm_fwd":
            wide = randn(b, L, c + 64 if case["sliced"] else c).to(t)
            s["x"] = wide[..., 64:] if case["sliced"] else wide
            s["residual"] = (4 * size * randn(b, L, c)).to(stream) if stream else None
        else:
            s["u"] = (4 * size * randn(b, L, c)).to(stream or t)
            wide = randn(b, L, c + 64 if case["sliced"] else c).to(TYPES[case["out"]])
            s["dy"] = wide[..., 64:] if case["sliced"] else wide
            s["dres"] = randn(b, L, c).to(stream) if stream else None
        return s
    h, kv, d = case["heads"], case["kvheads"], case["headdim"]
    lead = (b,) if case["op"] == "attn_step" else (b, L)
    if case["sliced"]:
        wide = randn(*lead, (h + 2 * kv) * d).to(t)
        q, k, v = wide.split([h * d, kv * d, kv * d], -1)
        s["q"], s["k"], s["v"] = q.unflatten(-1, (h, d)), k.unflatten(-1, (kv, d)), v.unflatten(-1, (kv, d))
    else:
        s["q"], s["k"], s["v"] = randn(*lead, h, d).to(t), randn(*lead, kv, d).to(t), randn(*lead, kv, d).to(t)
    s["positions"] = s["kc"] = s["vc"] = None
    if case["carry"] or case["op"] == "attn_step":
        s["positions"] = _tokens(_positions(case))
        s["kc"], s["vc"] = (randn(b, kv, case["window"] + case["sinks"], d).to(t) for _ in range(2))
    if case["op"] == "attn_bwd":
        s["dy"] = randn(b, L, h, d).to(t)
        # what the forward pass left
        y, lse = _attend(s, *_plain_keys(s))
        s["y"], s["lse"] = y.to(t), lse
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


def _scales(y, block):
    """(rows.., channels) as (rows.., blocks, columns of a block), and each block's scale (rows.., blocks, 1)."""
    c = y.shape[-1]
    wide = block or c
    y = torch.nn.functional.pad(y, (0, -c % wide)).unflatten(-1, (-1, wide))
    return y, (y.abs().amax(-1, keepdim=True) / E4M3_MAX).clamp_min(2.0 ** -126)


def _plain_norm_fwd(s):
    c = s["case"]
    u = s["x"].float()
    if s["residual"] is not None:
        u = u + s["residual"].float()
    y = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS) * s["weight"]
    live = _live(s)
    if live is not None:
        u, y = torch.where(live, u, 0.0), torch.where(live, y, 0.0)
    if c["out"] == "e4m3":
        y, scale = _scales(y, c["block"])
        codes = (y / scale).clamp(-E4M3_MAX, E4M3_MAX).to(TYPES["e4m3"])
        got = [codes.flatten(-2)[..., :c["channels"]].contiguous(), scale.squeeze(-1)]
    else:
        got = [y.to(TYPES[c["out"]])]
    return got + [u.to(TYPES[c["stream"]])] if c["stream"] else got


def _plain_norm_bwd(s):
    c = s["case"]
    u, dy = s["u"].float(), s["dy"].float()
    live = _live(s)
    if live is not None:
        dy = torch.where(live, dy, 0.0)
    r = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
    du = r * (s["weight"] * dy - u * (r * r) * (s["weight"] * dy * u).mean(-1, keepdim=True))
    if s["dres"] is not None:
        du = du + (s["dres"].float() if live is None else torch.where(live, s["dres"].float(), 0.0))
    got = {"dx": du.to(TYPES[c["dtype"]]), "dweight": (dy * u * r).sum((0, 1), dtype=torch.float64).float()}
    if s["dres"] is not None:
        got["dresidual"] = du.to(TYPES[c["stream"]])
    return got


def _held(s, behind):
    """The token that each slot of the cache holds once `behind` (b) tokens are past, -1 for none: (b, slots)."""
    c = s["case"]
    slot = torch.arange(c["window"] + c["sinks"], device="cuda")[None, :]
    last = behind[:, None].long() - 1
    ring = last - (last - slot) % c["window"]
    return torch.where(slot < c["sinks"], torch.where(slot <= last, slot, -1),
                       torch.where(ring >= c["sinks"], ring, -1))


def _plain_keys(s):
    """Keys and values in fp32 (b, kv, n, d) and the token that each is (b, n), -1 for none."""
    c = s["case"]
    behind = s["positions"] if s["positions"] is not None else torch.zeros(c["batch"], dtype=torch.int32, device="cuda")
    t = torch.arange(c["seqlen"], device="cuda")
    new = behind[:, None] + t
    if s["lengths"] is not None:
        new = torch.where(t < s["lengths"][:, None], new, -1)
    k, v = s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    if s["kc"] is None:
        return k, v, new
    return torch.cat([s["kc"].float(), k], 2), torch.cat([s["vc"].float(), v], 2), torch.cat([_held(s, behind), new], 1)


def _weights(s, k, tok):
    """Softmax numerators, their sums and maxima, (b, kv, g, L, n or 1), and q (b, kv, g, L, d) in fp32."""
    c = s["case"]
    b, L, kv, d = c["batch"], c["seqlen"], c["kvheads"], c["headdim"]
    q = s["q"].float().unflatten(2, (kv, -1)).permute(0, 2, 3, 1, 4)
    score = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (-1, L)) * d ** -0.5
    t = torch.arange(L, device="cuda")
    t = t + s["positions"][:, None] if s["positions"] is not None else t.expand(b, L)
    t, j = t[:, :, None], tok[:, None, :]
    seen = (j >= 0) & (j <= t) & ((t - j < c["window"]) | (j < c["sinks"]))
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    return p, p.sum(-1, keepdim=True), top, q


def _attend(s, k, v, tok):
    """y (b, L, h, d) and the logarithm of the softmax's sum (b, h, L); 0 behind a sequence's end."""
    p, total, top, _ = _weights(s, k, tok)
    y = (p.flatten(2, 3) @ v).unflatten(2, p.shape[2:4]) / total
    y, lse = y.permute(0, 3, 1, 2, 4).flatten(2, 3), (top + torch.log(total)).squeeze(-1).flatten(1, 2)
    live = _live(s)
    if live is None:
        return y, lse
    return torch.where(live[..., None], y, 0.0), torch.where(live.transpose(1, 2), lse, 0.0)


def _plain_attn_fwd(s):
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    y, lse = _attend(s, *_plain_keys(s))
    if not c["carry"]:
        return [y.to(t), lse]
    ends = s["lengths"] if s["lengths"] is not None else c["seqlen"]
    after = _held(s, s["positions"] + ends) - s["positions"][:, None]
    pick = after.clamp_min(0)[:, None, :, None]
    for cache, new in ((s["kc"], s["k"]), (s["vc"], s["v"])):
        new = new.transpose(1, 2)
        new = torch.gather(new, 2, pick.expand(-1, c["kvheads"], -1, c["headdim"]))
        cache.copy_(torch.where((after >= 0)[:, None, :, None], new, cache))
    return [y.to(t), s["kc"], s["vc"]]


def _plain_attn_bwd(s):
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    k, v, tok = _plain_keys(s)
    p, total, _, q = _weights(s, k, tok)
    p = p / total
    dy = s["dy"].float().unflatten(2, (c["kvheads"], -1)).permute(0, 2, 3, 1, 4)
    live = _live(s)
    if live is not None:
        p, dy = (torch.where(live[:, None, None], x, 0.0) for x in (p, dy))
    dp = (dy.flatten(2, 3) @ v.transpose(2, 3)).view_as(p)
    ds = (p * (dp - (p * dp).sum(-1, keepdim=True)) * c["headdim"] ** -0.5).flatten(2, 3)
    dq = (ds @ k).view_as(q).permute(0, 3, 1, 2, 4).flatten(2, 3)
    dk = (ds.transpose(2, 3) @ q.flatten(2, 3)).transpose(1, 2)
    dv = (p.flatten(2, 3).transpose(2, 3) @ dy.flatten(2, 3)).transpose(1, 2)
    return {"dq": dq.to(t), "dk": dk.to(t), "dv": dv.to(t)}


def _plain_attn_step(s):
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    at, w, n = s["positions"].long(), c["window"], c["sinks"]
    on = (at >= 0)[:, None, None]
    slot = torch.where(at < n, at, n + (at - n) % w).clamp_min(0)
    rows = torch.arange(c["batch"], device="cuda")
    for cache, new in ((s["kc"], s["k"]), (s["vc"], s["v"])):
        cache[rows, :, slot] = torch.where(on, new, cache[rows, :, slot])
    q = s["q"].float().unflatten(1, (c["kvheads"], -1))
    score = (q @ s["kc"].float().transpose(2, 3)) * c["headdim"] ** -0.5
    seen = torch.arange(w + n, device="cuda") <= at[:, None]
    score = torch.where(seen[:, None, None], score, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    y = (p @ s["vc"].float() / p.sum(-1, keepdim=True)).flatten(1, 2)
    return [torch.where(on, y, 0.0).to(t), s["kc"], s["vc"]]


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "attn_fwd": _plain_attn_fwd,
          "attn_bwd": _plain_attn_bwd, "attn_step": _plain_attn_step}


def _lib():
    import mamba_chunked_ssd_amd as ssd
    return ssd


def _own_norm_fwd(s):
    c = s["case"]
    got = _lib().rms_norm_fwd(s["x"], s["weight"], s["residual"], eps=EPS, lengths=s["lengths"],
                              y_dtype=TYPES[c["out"]], scale_block=c["block"], return_residual=bool(c["stream"]))
    return list(got) if isinstance(got, tuple) else [got]


def _own_norm_bwd(s):
    c = s["case"]
    return _lib().rms_norm_bwd(s["dy"], s["u"], s["weight"], s["dres"], eps=EPS, lengths=s["lengths"],
                               dx_dtype=TYPES[c["dtype"]], want_dresidual=s["dres"] is not None)


def _own_attn_fwd(s):
    c = s["case"]
    got = _lib().window_attention_fwd(s["q"], s["k"], s["v"], c["window"], c["sinks"], lengths=s["lengths"],
                                      positions=s["positions"], k_cache=s["kc"], v_cache=s["vc"],
                                      return_lse=not c["carry"])
    return [got, s["kc"], s["vc"]] if c["carry"] else list(got)


def _own_attn_bwd(s):
    c = s["case"]
    return _lib().window_attention_bwd(s["q"], s["k"], s["v"], s["y"], s["lse"], s["dy"], c["window"], c["sinks"],
                                       lengths=s["lengths"])


def _own_attn_step(s):
    c = s["case"]
    y = _lib().window_attention_step(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["positions"], c["window"], c["sinks"])
    return [y, s["kc"], s["vc"]]


_OWN = {"norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd, "attn_fwd": _own_attn_fwd, "attn_bwd": _own_attn_bwd,
        "attn_step": _own_attn_step}


# ---------------------------------------------------------------------------
# What a pass cannot do without, and its exact outputs
# ---------------------------------------------------------------------------

def _pairs(case):
    """Pairs of a query and a key that it sees, of all sequences and one head."""
    total, w, n = 0, case["window"], case["sinks"]
    for first, length in zip(_positions(case), _lengths(case)):
        t = torch.arange(first, first + length, dtype=torch.int64)
        total += int((torch.minimum(t + 1, torch.tensor(w)) + (t + 1 - w).clamp(0, n)).sum())
    return total


def work(case):
    size = {"bf16": 2, "f32": 4, "e4m3": 1, "": 0}
    i = size[case["dtype"]]
    rows = sum(_lengths(case))
    every = case["batch"] * case["seqlen"]
    if case["op"].startswith("norm"):
        c, r, o = case["channels"], size[case["stream"]], size[case["out"]]
        if case["op"] == "norm_fwd":
            scales = -(-c // (case["block"] or c)) * 4 * every if case["out"] == "e4m3" else 0
            return {"bytes": rows * c * (i + r) + every * c * (r + o) + scales + 4 * c, "flops": 5 * rows * c}
        return {"bytes": rows * c * ((r or i) + r + o) + every * c * (i + r) + 8 * c, "flops": 13 * rows * c}
    h, kv, d = case["heads"], case["kvheads"], case["headdim"]
    if case["op"] == "attn_step":
        slots = case["window"] + case["sinks"]
        keys = sum(min(t + 1, slots) for t in _positions(case))
        return {"bytes": 2 * i * kv * d * (keys + case["batch"]) + 2 * i * h * d * case["batch"], "flops": 4 * h * d * keys}
    pairs = h * _pairs(case)
    tokens = i * d * (rows * (h + 2 * kv) + every * h)
    if case["op"] == "attn_fwd":
        # earlier tokens that some new one sees are read, the cache's slots of the new ones written
        slots = case["window"] + case["sinks"]
        old = sum(min(p, slots) for p, n in zip(_positions(case), _lengths(case)) if n) if case["carry"] else 0
        put = sum(min(n, slots) for n in _lengths(case)) if case["carry"] else 0
        return {"bytes": tokens + 2 * i * kv * d * (old + put) + (0 if case["carry"] else 4 * h * every),
                "flops": 4 * d * pairs}
    return {"bytes": i * d * (rows * (3 * h + 2 * kv) + every * (h + 2 * kv)) + 4 * h * rows, "flops": 10 * d * pairs}


def _exact_norm(case, x, residual, weight, ends):
    """Row by row of the definition, the stream and the unrounded y; zeros behind an end."""
    u = x if residual is None else x + residual
    rms = (u.square().sum(-1) / case["channels"] + EPS).sqrt()
    on = torch.zeros(u.shape[:2], dtype=torch.float64, device=u.device)
    for i, end in enumerate(ends):
        on[i, :end] = 1
    return u * on[..., None], u / rms[..., None] * weight * on[..., None]


def _exact_attention(case, q, k, v, past, ends):
    """One sequence and one head at a time; past: (keys, values, their tokens) of each sequence, oldest first."""
    group = case["heads"] // case["kvheads"]
    ys, lses = [], []
    for i, end in enumerate(ends):
        behind, kp, vp, tp = past[i]
        t = torch.arange(behind, behind + end, device=q.device)
        tok = torch.cat([tp, t])
        back = t[:, None] - tok[None, :]
        hidden = (back < 0) | ((back >= case["window"]) & (tok[None, :] >= case["sinks"]))
        heads, sums = [], []
        for h in range(case["heads"]):
            keys, values = torch.cat([kp[h // group], k[i, :end, h // group]]), torch.cat([vp[h // group], v[i, :end, h // group]])
            logit = (q[i, :end, h] @ keys.T / math.sqrt(case["headdim"])).masked_fill(hidden, -math.inf)
            heads.append(torch.softmax(logit, 1) @ values)
            sums.append(torch.logsumexp(logit, 1))
        pad = case["seqlen"] - end
        ys.append(torch.nn.functional.pad(torch.stack(heads, 1), (0, 0, 0, 0, 0, pad)))
        lses.append(torch.nn.functional.pad(torch.stack(sums), (0, pad)))
    return torch.stack(ys), torch.stack(lses)


def _slot(case, token):
    return token if token < case["sinks"] else case["sinks"] + (token - case["sinks"]) % case["window"]


def exact(case, seed):
    s = prepare(case, seed)
    ends = _lengths(case)
    if case["op"] == "norm_fwd":
        u, y = _exact_norm(case, s["x"].double(), None if s["residual"] is None else s["residual"].double(),
                           s["weight"].double(), ends)
        got = [y]
        if case["out"] == "e4m3":
            parts = y.split(case["block"] or case["channels"], -1)
            scales = [p.abs().amax(-1).div(E4M3_MAX).clamp_min(2.0 ** -126) for p in parts]
            # what the codes round
            got = [torch.cat([p / q[..., None] for p, q in zip(parts, scales)], -1), torch.stack(scales, -1)]
        return got + [u] if case["stream"] else got
    if case["op"] == "norm_bwd":
        u, w = s["u"].double().requires_grad_(), s["weight"].double().requires_grad_()
        out, y = _exact_norm(case, u, None, w, ends)
        loss = (y * s["dy"].double()).sum()
        if s["dres"] is not None:
            loss = loss + (out * s["dres"].double()).sum()
        loss.backward()
        got = {"dx": u.grad, "dweight": w.grad}
        return {**got, "dresidual": u.grad} if s["dres"] is not None else got
    backwards = case["op"] == "attn_bwd"
    first, step = _positions(case), case["op"] == "attn_step"
    q, k, v = (s[n].double()[:, None] if step else s[n].double() for n in "qkv")
    q, k, v = (x.clone().requires_grad_(backwards) for x in (q, k, v))
    caches = [None if s[n] is None else s[n].double() for n in ("kc", "vc")]
    past = []
    if step:
        ends = [0 if p < 0 else 1 for p in first]
    for i, p in enumerate(first):
        kept = [j for j in range(max(p, 0)) if j < case["sinks"] or j >= p - case["window"]]
        at = torch.tensor([_slot(case, j) for j in kept], dtype=torch.int64, device="cuda")
        held = [x.new_zeros((case["kvheads"], 0, case["headdim"])) if c is None else c[i][:, at] for x, c in zip((k, v), caches)]
        past.append((max(p, 0), *held, torch.tensor(kept, dtype=torch.int64, device="cuda")))
    y, lse = _exact_attention(case, q, k, v, past, ends)
    if backwards:
        (y * s["dy"].double()).sum().backward()
        return {"dq": q.grad, "dk": k.grad, "dv": v.grad}
    if not case["carry"] and not step:
        return [y, lse]
    for cache, new in zip(caches, (k, v)):
        for i, (p, end) in enumerate(zip(first, ends)):
            fresh = [j for j in range(end) if p + j < case["sinks"] or j >= end - case["window"]]
            at = torch.tensor([_slot(case, p + j) for j in fresh], dtype=torch.int64, device="cuda")
            cache[i][:, at] = new[i, torch.tensor(fresh, dtype=torch.int64, device="cuda")].transpose(0, 1)
    return [y[:, 0] if step else y, *caches]
