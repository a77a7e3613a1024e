"""Sliding-window attention with sinks and the RMS norm in plain fp64 numpy,
one token at a time, with their gradients by the chain rule: test
infrastructure, sharing no code with the library.

Sequences may end early: ``lengths`` (batch,) or None.  Rows behind the end
are 0 in every output.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, np.float64)


def _ends(lengths, b, L):
    return [L] * b if lengths is None else [min(max(int(v), 0), L) for v in lengths]


# ---------------------------------------------------------------------------
# Attention: q (b, L, h, d), k and v (b, L, kv, d), caches (b, kv, sinks + window, d)
# ---------------------------------------------------------------------------

def slot_of(j, window, sinks):
    return j if j < sinks else sinks + (j - sinks) % window


def sees(t, j, window, sinks):
    return j <= t and (t - j < window or j < sinks)


def _tokens(k, v, i, first, end, kc, vc, window, sinks):
    """{token: (keys, values)} of sequence i: what the cache still holds of those before `first`, and its new ones."""
    held = {}
    for j in range(first):
        if j < sinks or j >= first - window:
            s = slot_of(j, window, sinks)
            held[j] = (kc[i][:, s], vc[i][:, s])
    for t in range(end):
        held[first + t] = (k[i, t], v[i, t])
    return held


def attention(q, k, v, window, sinks=0, scale=None, lengths=None, positions=None, kc=None, vc=None):
    """y, lse and the magnitudes sum_j p |v_j| that bound y's rounding."""
    q, k, v, kc, vc = map(_f64, (q, k, v, kc, vc))
    b, L, h, d = q.shape
    g = h // k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    y, lse, mag = np.zeros(q.shape), np.zeros((b, h, L)), np.zeros(q.shape)
    for i, end in enumerate(_ends(lengths, b, L)):
        first = 0 if positions is None else max(int(positions[i]), 0)
        held = _tokens(k, v, i, first, end, kc, vc, window, sinks)
        for t in range(end):
            seen = [j for j in held if sees(first + t, j, window, sinks)]
            ks = np.stack([held[j][0] for j in seen])
            vs = np.stack([held[j][1] for j in seen])
            for n in range(h):
                s = scale * ks[:, n // g] @ q[i, t, n]
                top = s.max()
                e = np.exp(s - top)
                p = e / e.sum()
                y[i, t, n] = p @ vs[:, n // g]
                mag[i, t, n] = p @ np.abs(vs[:, n // g])
                lse[i, n, t] = top + np.log(e.sum())
    return y, lse, mag


def attention_bwd(q, k, v, dy, window, sinks=0, scale=None, lengths=None):
    """Gradients, and for each the sum of its terms' magnitudes (of the parts of a term too)."""
    q, k, v, dy = map(_f64, (q, k, v, dy))
    b, L, h, d = q.shape
    g = h // k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out = {n: np.zeros(x.shape) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    mag = {n: np.zeros(x.shape) for n, x in out.items()}
    for i, end in enumerate(_ends(lengths, b, L)):
        for t in range(end):
            seen = np.array([j for j in range(t + 1) if sees(t, j, window, sinks)])
            for n in range(h):
                m = n // g
                ks, vs = k[i, seen, m], v[i, seen, m]
                s = scale * ks @ q[i, t, n]
                p = np.exp(s - s.max())
                p /= p.sum()
                dp = vs @ dy[i, t, n]
                delta = p @ dp
                ds = scale * p * (dp - delta)
                # |dy| . |v| of each key and of the row's mean bound the parts of dp - delta
                part = np.abs(vs) @ np.abs(dy[i, t, n])
                dsm = scale * p * (part + p @ part)
                out["dq"][i, t, n] = ds @ ks
                mag["dq"][i, t, n] = dsm @ np.abs(ks)
                out["dk"][i, seen, m] += np.outer(ds, q[i, t, n])
                mag["dk"][i, seen, m] += np.outer(dsm, np.abs(q[i, t, n]))
                out["dv"][i, seen, m] += np.outer(p, dy[i, t, n])
                mag["dv"][i, seen, m] += np.outer(p, np.abs(dy[i, t, n]))
    return out, mag


def cache_after(kc, vc, k, v, window, sinks=0, lengths=None, positions=None):
    """The caches once the new tokens are in, token by token."""
    kc, vc = np.array(kc), np.array(vc)
    b, L = k.shape[:2]
    for i, end in enumerate(_ends(lengths, b, L)):
        first = 0 if positions is None else max(int(positions[i]), 0)
        for t in range(end):
            s = slot_of(first + t, window, sinks)
            kc[i][:, s], vc[i][:, s] = k[i, t], v[i, t]
    return kc, vc


# ---------------------------------------------------------------------------
# RMS norm: x, residual, u, dy (b, L, c), weight (c)
# ---------------------------------------------------------------------------

def _live(shape, lengths):
    b, L = shape[:2]
    on = np.zeros((b, L, 1), bool)
    for i, end in enumerate(_ends(lengths, b, L)):
        on[i, :end] = True
    return on


def norm(x, weight=None, residual=None, eps=1e-5, lengths=None):
    """u and y."""
    x, weight, residual = map(_f64, (x, weight, residual))
    on = _live(x.shape, lengths)
    u = np.where(on, x if residual is None else x + residual, 0)
    r = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    return u, np.where(on, u * r * (1 if weight is None else weight), 0)


def scales(y, block):
    """The scale of each block of columns (of the row: block 0) of an 8-bit y, and those of every column."""
    c = y.shape[-1]
    block = block or c
    most = np.stack([np.abs(y[..., k:k + block]).max(-1) for k in range(0, c, block)], -1)
    s = np.maximum(most / 448, 2.0 ** -126)
    return s, np.repeat(s, block, -1)[..., :c]


def norm_bwd(dy, u, weight=None, dres=None, eps=1e-5, lengths=None):
    """du and dweight, and the sums of their terms' magnitudes."""
    dy, u, weight, dres = map(_f64, (dy, u, weight, dres))
    on = _live(u.shape, lengths)
    dy, u = np.where(on, dy, 0), np.where(on, u, 0)
    dres = 0 if dres is None else np.where(on, dres, 0)
    w = np.ones(u.shape[-1]) if weight is None else weight
    r = np.where(on, 1 / np.sqrt((u * u).mean(-1, keepdims=True) + np.where(on, eps, 1)), 0)
    du = r * w * dy - u * r ** 3 * (w * dy * u).mean(-1, keepdims=True) + dres
    mag = np.abs(r * w * dy) + np.abs(u) * r ** 3 * np.abs(w * dy * u).mean(-1, keepdims=True) + np.abs(dres)
    return du, (dy * u * r).sum((0, 1)), mag, np.abs(dy * u * r).sum((0, 1))
