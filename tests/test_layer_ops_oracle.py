"""The oracle of the short causal convolution and the selective scan: closed
forms, and its gradients against central differences of its forward pass."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import layer_ops as lo


def _conv_case(rng, b=2, L=7, c=3, W=4):
    return dict(x=rng.normal(size=(b, L, c)), weight=rng.normal(size=(c, W)), bias=rng.normal(size=c),
                init=rng.normal(size=(b, W - 1, c)))


def _scan_case(rng, b=2, L=6, c=4, n=3, g=2):
    return dict(x=rng.normal(size=(b, L, c)), dt=rng.normal(size=(b, L, c)), A=-np.exp(rng.normal(size=(c, n))),
                B=rng.normal(size=(b, L, g, n)), C=rng.normal(size=(b, L, g, n)), D=rng.normal(size=c),
                z=rng.normal(size=(b, L, c)), dt_bias=rng.normal(size=c), init=rng.normal(size=(b, c, n)))


def _differences(f, arrays, grads, names, step=1e-6):
    """Central differences of the scalar f(**arrays): the error is O(step^2) + eps |f| / step, below 1e-8 of the
    values here (|f| is of order 10), hence the bound of 1e-6."""
    for name, grad in names.items():
        a = arrays[name]
        for idx in np.ndindex(a.shape):
            keep = a[idx]
            a[idx] = keep + step
            hi = f(**arrays)
            a[idx] = keep - step
            lo_ = f(**arrays)
            a[idx] = keep
            assert abs((hi - lo_) / (2 * step) - grads[grad][idx]) < 1e-6 * max(1.0, abs(grads[grad][idx])), (name, idx)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act", [False, True])
def test_conv_gradients_against_differences(W, act):
    rng = np.random.default_rng(W)
    arrays = _conv_case(rng, W=W)
    lengths = [7, 2]
    dy, dfin = rng.normal(size=(2, 7, 3)), rng.normal(size=(2, W - 1, 3))

    def f(**a):
        y, fin = lo.conv(**a, lengths=lengths, act=act)
        return (y * dy).sum() + (fin * dfin).sum()

    g = lo.conv_bwd(arrays["x"], arrays["weight"], arrays["bias"], dy, arrays["init"], dfin, lengths, act)
    _differences(f, arrays, g, dict(x="dx", weight="dweight", bias="dbias", init="d_initial_states"))


@pytest.mark.parametrize("use_softplus", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_scan_gradients_against_differences(use_softplus, gate):
    rng = np.random.default_rng(10 + gate)
    arrays = _scan_case(rng)
    if not use_softplus:
        arrays["dt"], arrays["dt_bias"] = np.abs(arrays["dt"]) + 0.1, np.abs(arrays["dt_bias"])
    if not gate:
        arrays["z"] = None
    lengths = [6, 3]
    dy, dfin = rng.normal(size=(2, 6, 4)), rng.normal(size=(2, 4, 3))

    def f(**a):
        y, fin = lo.scan(**a, lengths=lengths, use_softplus=use_softplus)
        return (y * dy).sum() + (fin * dfin).sum()

    g = lo.scan_bwd(dy=dy, dfinal=dfin, lengths=lengths, use_softplus=use_softplus, **arrays)
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", dt_bias="ddt_bias", init="d_initial_states")
    if gate:
        names["z"] = "dz"
    _differences(f, arrays, g, names)


def test_conv_is_numpys_convolution():
    rng = np.random.default_rng(3)
    x, w = rng.normal(size=(1, 20, 2)), rng.normal(size=(2, 4))
    y, fin = lo.conv(x, w, act=False)
    for c in range(2):
        assert np.allclose(y[0, :, c], np.convolve(x[0, :, c], w[c, ::-1])[:20], atol=1e-12)
    assert np.array_equal(fin[0], x[0, -3:])


def test_scan_of_constant_inputs_is_a_geometric_series():
    # one channel and state, d = 1, x = B = C = 1: h_t = sum_{s<=t} e^{A s}
    L, A = 9, -0.3
    one = np.ones((1, L, 1))
    y, fin = lo.scan(one, one, [[A]], one[..., None], one[..., None], use_softplus=False)
    want = np.cumsum(np.exp(A * np.arange(L)))
    assert np.allclose(y[0, :, 0], want, atol=1e-12) and np.isclose(fin[0, 0, 0], want[-1])


def test_pieces_joined_by_their_states_are_the_whole():
    rng = np.random.default_rng(4)
    a = _scan_case(rng)
    y, fin = lo.scan(**a)
    cut = {k: (v[:, :4] if k in ("x", "dt", "B", "C", "z") else v) for k, v in a.items()}
    y1, f1 = lo.scan(**cut)
    rest = {k: (v[:, 4:] if k in ("x", "dt", "B", "C", "z") else v) for k, v in a.items()}
    rest["init"] = f1
    y2, f2 = lo.scan(**rest)
    assert np.allclose(np.concatenate([y1, y2], 1), y) and np.allclose(f2, fin)
    c = _conv_case(rng)
    y, fin = lo.conv(**c)
    y1, f1 = lo.conv(c["x"][:, :2], c["weight"], c["bias"], c["init"])
    y2, f2 = lo.conv(c["x"][:, 2:], c["weight"], c["bias"], f1)
    assert np.allclose(np.concatenate([y1, y2], 1), y) and np.array_equal(f2, fin)
