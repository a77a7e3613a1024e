"""The fp64 oracle of sliding-window attention and the RMS norm against itself:
its gradients by differences, its cache token by token, closed forms."""
from __future__ import annotations

import numpy as np

from oracle import mixer_ops as mo


def test_attention_gradients_against_differences():
    # the oracle's own, in fp64: the error of central differences with h = 1e-5 is below 1e-8 here
    rng = np.random.default_rng(2)
    x = {"dq": rng.standard_normal((1, 6, 2, 4)), "dk": rng.standard_normal((1, 6, 1, 4)), "dv": rng.standard_normal((1, 6, 1, 4))}
    dy = rng.standard_normal((1, 6, 2, 4))
    ref, _ = mo.attention_bwd(x["dq"], x["dk"], x["dv"], dy, 3, 1)
    for name in x:
        for i in np.ndindex(x[name].shape):
            lo = []
            for sign in (1, -1):
                z = {k: v.copy() for k, v in x.items()}
                z[name][i] += sign * 1e-5
                lo.append((mo.attention(z["dq"], z["dk"], z["dv"], 3, 1)[0] * dy).sum())
            assert abs((lo[0] - lo[1]) / 2e-5 - ref[name][i]) < 1e-7


def test_norm_gradients_against_differences():
    # the fp64 oracle's own gradients, by central differences of its forward pass: error h^2 f''' / 6 and rounding
    # 2^-53 |f| / h, with h = 1e-5 below 1e-8 here
    rng = np.random.default_rng(1)
    x, w, dy, dres = rng.standard_normal((1, 3, 6)), rng.standard_normal(6), rng.standard_normal((1, 3, 6)), rng.standard_normal((1, 3, 6))
    du, dw, _, _ = mo.norm_bwd(dy, x, w, dres)

    def loss(x, w):
        u, y = mo.norm(x, w)
        return (y * dy).sum() + (u * dres).sum()

    h = 1e-5
    for i in np.ndindex(x.shape):
        e = np.zeros(x.shape)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - du[i]) < 1e-7
    for i in range(6):
        e = np.zeros(6)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_a_prompt_in_pieces_is_the_prompt():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((1, 40, 2, 4)), rng.standard_normal((1, 40, 1, 4)), rng.standard_normal((1, 40, 1, 4))
    for w, n in ((1, 0), (7, 3), (5, 20), (60, 2)):
        want, lse, _ = mo.attention(q, k, v, w, n)
        kc, vc = np.full((1, 1, w + n, 4), np.nan), np.full((1, 1, w + n, 4), np.nan)
        for t0, t1 in ((0, 1), (1, 6), (6, 30), (30, 31), (31, 40)):
            y, part, _ = mo.attention(q[:, t0:t1], k[:, t0:t1], v[:, t0:t1], w, n, positions=[t0], kc=kc, vc=vc)
            kc, vc = mo.cache_after(kc, vc, k[:, t0:t1], v[:, t0:t1], w, n, positions=[t0])
            assert np.allclose(y, want[:, t0:t1], atol=1e-13) and np.allclose(part, lse[:, :, t0:t1], atol=1e-13)


def test_closed_forms():
    rng = np.random.default_rng(4)
    v = rng.standard_normal((1, 9, 1, 4))
    zero = np.zeros((1, 9, 1, 4))
    # equal scores: the mean over what is seen; a window of one: the value itself
    y, lse, _ = mo.attention(zero, zero, v, 3, 1)
    seen = [[j for j in range(t + 1) if t - j < 3 or j < 1] for t in range(9)]
    assert np.allclose(y[0, :, 0], [v[0, s, 0].mean(0) for s in seen])
    assert np.allclose(lse[0, 0], np.log([len(s) for s in seen]))
    assert np.allclose(mo.attention(v, v, v, 1)[0], v)
    u, y = mo.norm(np.full((1, 2, 5), -3.0), eps=0.0)
    assert np.allclose(y, -1.0) and np.allclose(u, -3.0)
