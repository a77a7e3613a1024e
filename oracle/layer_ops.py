"""The short causal convolution and the selective scan in plain fp64 numpy, one
token at a time, with their gradients by the chain rule: test infrastructure,
sharing no code with the library.

Sequences may end early: ``lengths`` (batch,) or None.  Rows behind the end
are 0 in y and in every gradient; the final state is the one after the last
token.
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def silu(v):
    return v * sigmoid(v)


def dsilu(v):
    s = sigmoid(v)
    return s * (1 + v * (1 - s))


def _f64(a):
    return None if a is None else np.asarray(a, np.float64)


def _ends(lengths, b, L):
    return [L] * b if lengths is None else [min(max(int(v), 0), L) for v in lengths]


# ---------------------------------------------------------------------------
# Convolution: x (b, L, c), weight (c, W), bias (c), init (b, W - 1, c)
# ---------------------------------------------------------------------------

def _line(x, init, i, end, W):
    """Inputs of sequence i with the state's rows in front: row W - 1 + t is x_t."""
    head = np.zeros((W - 1, x.shape[2])) if init is None else init[i]
    return np.concatenate([head, x[i, :end]])


def conv(x, weight, bias=None, init=None, lengths=None, act=True):
    x, weight, bias, init = map(_f64, (x, weight, bias, init))
    b, L, c = x.shape
    W = weight.shape[1]
    y, final = np.zeros((b, L, c)), np.zeros((b, W - 1, c))
    for i, end in enumerate(_ends(lengths, b, L)):
        line = _line(x, init, i, end, W)
        for t in range(end):
            p = (weight.T * line[t:t + W]).sum(0) + (0 if bias is None else bias)
            y[i, t] = silu(p) if act else p
        final[i] = line[end:]
    return y, final


def conv_magnitude(x, weight, bias=None, init=None, lengths=None):
    """sum_k |w_k x| + |bias| of each output: what its rounding errors scale with."""
    return conv(np.abs(_f64(x)), np.abs(_f64(weight)), None if bias is None else np.abs(_f64(bias)),
                None if init is None else np.abs(_f64(init)), lengths, act=False)[0]


def conv_bwd(x, weight, bias, dy, init=None, dfinal=None, lengths=None, act=True):
    x, weight, bias, init, dy, dfinal = map(_f64, (x, weight, bias, init, dy, dfinal))
    b, L, c = x.shape
    W = weight.shape[1]
    g = dict(dx=np.zeros((b, L, c)), dweight=np.zeros((c, W)), dbias=np.zeros(c),
             d_initial_states=np.zeros((b, W - 1, c)))
    for i, end in enumerate(_ends(lengths, b, L)):
        line = _line(x, init, i, end, W)
        dline = np.zeros_like(line)
        for t in range(end):
            d = dy[i, t].copy()
            if act:
                d *= dsilu((weight.T * line[t:t + W]).sum(0) + (0 if bias is None else bias))
            g["dbias"] += d
            g["dweight"] += (d * line[t:t + W]).T
            dline[t:t + W] += weight.T * d
        if dfinal is not None:
            dline[end:] += dfinal[i]
        g["d_initial_states"][i] = dline[:W - 1]
        g["dx"][i, :end] = dline[W - 1:]
    return g


# ---------------------------------------------------------------------------
# Selective scan: x, dt, z (b, L, c), A (c, n), B, C (b, L, g, n), D, dt_bias (c)
# ---------------------------------------------------------------------------

def _scan_inputs(x, dt, A, B, C, D, z, dt_bias, init):
    x, dt, A, B, C, D, z, dt_bias, init = map(_f64, (x, dt, A, B, C, D, z, dt_bias, init))
    b, L, c = x.shape
    per = c // B.shape[2]
    raw = dt if dt_bias is None else dt + dt_bias
    h0 = np.zeros((b, c, A.shape[1])) if init is None else init
    return x, raw, A, np.repeat(B, per, 2), np.repeat(C, per, 2), np.zeros(c) if D is None else D, z, h0


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, init=None, lengths=None, use_softplus=True):
    x, raw, A, B, C, D, z, h0 = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, init)
    b, L, c = x.shape
    y, final = np.zeros((b, L, c)), h0.copy()
    step = softplus(raw) if use_softplus else raw
    for i, end in enumerate(_ends(lengths, b, L)):
        for t in range(end):
            d = step[i, t][:, None]
            final[i] = np.exp(d * A) * final[i] + d * x[i, t][:, None] * B[i, t]
            y[i, t] = (C[i, t] * final[i]).sum(1) + D * x[i, t]
            if z is not None:
                y[i, t] *= silu(z[i, t])
    return y, final


def scan_bwd(x, dt, A, B, C, D, dy, z=None, dt_bias=None, init=None, dfinal=None, lengths=None, use_softplus=True):
    groups = np.asarray(B).shape[2]
    x, raw, A, B, C, D, z, h0 = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, init)
    dy, dfinal = _f64(dy), _f64(dfinal)
    b, L, c = x.shape
    n = A.shape[1]
    step = softplus(raw) if use_softplus else raw
    slope = sigmoid(raw) if use_softplus else np.ones_like(raw)
    g = dict(dx=np.zeros((b, L, c)), ddt=np.zeros((b, L, c)), dA=np.zeros((c, n)), dB=np.zeros((b, L, groups, n)),
             dC=np.zeros((b, L, groups, n)), dD=np.zeros(c), ddt_bias=np.zeros(c),
             d_initial_states=np.zeros((b, c, n)))
    if z is not None:
        g["dz"] = np.zeros((b, L, c))
    for i, end in enumerate(_ends(lengths, b, L)):
        hs = [h0[i]]
        for t in range(end):
            d = step[i, t][:, None]
            hs.append(np.exp(d * A) * hs[-1] + d * x[i, t][:, None] * B[i, t])
        G = np.zeros((c, n)) if dfinal is None else dfinal[i].copy()
        for t in reversed(range(end)):
            d, xt = step[i, t][:, None], x[i, t][:, None]
            o = dy[i, t].copy()
            if z is not None:
                g["dz"][i, t] = o * ((C[i, t] * hs[t + 1]).sum(1) + D * x[i, t]) * dsilu(z[i, t])
                o *= silu(z[i, t])
            G = G + C[i, t] * o[:, None]
            e = np.exp(d * A)
            q = e * G * hs[t]
            gB = (G * B[i, t]).sum(1)
            g["dC"][i, t] = (o[:, None] * hs[t + 1]).reshape(groups, -1, n).sum(1)
            g["dB"][i, t] = (d * xt * G).reshape(groups, -1, n).sum(1)
            g["dA"] += d * q
            g["dx"][i, t] = step[i, t] * gB + D * o
            g["dD"] += o * x[i, t]
            g["ddt"][i, t] = ((A * q).sum(1) + x[i, t] * gB) * slope[i, t]
            g["ddt_bias"] += g["ddt"][i, t]
            G = e * G
        g["d_initial_states"][i] = G
    return g
