"""Window attention and the RMS norm as a model's layers run them, beside the
convolution and the chunked scan: a training step with its gradients, a prompt
followed by single tokens, and the calls in one captured graph.

Bounds: every operator of a chain is within 2^-18 relatively in fp32 (its own
tests; 2-norms over all elements, for which rounding errors of single elements
average), products with the projections too; a chain of n of them is held to n
2^-18.
"""
from __future__ import annotations

import pytest
import torch

import mamba_chunked_ssd_amd as ssd

pytestmark = pytest.mark.gpu

B, L, C, H, KV, D, W, N = 2, 150, 128, 4, 2, 32, 40, 3


def weights(seed=0):
    g = torch.Generator().manual_seed(seed)

    def mat(i, o):
        return (torch.randn((i, o), generator=g) / i ** 0.5).cuda()

    return dict(n1=(1 + 0.2 * torch.randn(C, generator=g)).cuda(), n2=(1 + 0.2 * torch.randn(C, generator=g)).cuda(),
                qkv=mat(C, (H + 2 * KV) * D), o=mat(H * D, C), conv=torch.randn((C, 4), generator=g).cuda() / 2,
                bias=torch.randn(C, generator=g).cuda() / 4)


def heads(qkv):
    q, k, v = qkv.split([H * D, KV * D, KV * D], -1)
    return q.unflatten(-1, (H, D)), k.unflatten(-1, (KV, D)), v.unflatten(-1, (KV, D))


def near(a, b, steps):
    a, b = a.detach(), b.detach()
    return float((a.double() - b.double()).norm() / b.double().norm()) <= steps * 2.0 ** -18


def dense(q, k, v):
    k, v = (x.repeat_interleave(H // KV, 2).transpose(1, 2) for x in (k, v))
    t = torch.arange(q.shape[1], device=q.device)
    back = t[:, None] - t[None, :]
    seen = (back >= 0) & ((back < W) | (t[None, :] < N))
    p = torch.softmax((q.transpose(1, 2) @ k.transpose(2, 3) * D ** -0.5).masked_fill(~seen, float("-inf")), -1)
    return (p @ v).transpose(1, 2)


def test_training_step():
    w = weights()
    g = torch.Generator(device="cuda").manual_seed(1)
    x, g1, g2 = (torch.randn((B, L, C), generator=g, device="cuda") for _ in range(3))
    n1, u0 = ssd.rms_norm_fwd(x, w["n1"], return_residual=True)
    c = ssd.causal_conv_fwd(n1, w["conv"], w["bias"])
    q, k, v = heads(c @ w["qkv"])
    y, lse = ssd.window_attention_fwd(q, k, v, W, N, return_lse=True)
    o = y.flatten(2) @ w["o"]
    n2, u1 = ssd.rms_norm_fwd(o, w["n2"], u0, return_residual=True)
    # backwards from gradients of both outputs
    b2 = ssd.rms_norm_bwd(g1, u1, w["n2"], g2, want_dresidual=True)
    dy = (b2["dx"] @ w["o"].T).unflatten(-1, (H, D))
    ba = ssd.window_attention_bwd(q, k, v, y, lse, dy, W, N)
    dc = torch.cat([ba[i].flatten(2) for i in ("dq", "dk", "dv")], -1) @ w["qkv"].T
    bc = ssd.causal_conv_bwd(n1, w["conv"], w["bias"], dc)
    b1 = ssd.rms_norm_bwd(bc["dx"], u0, w["n1"], b2["dresidual"])
    # the same in fp64, differentiated
    z = {i: t.double().requires_grad_() for i, t in w.items()}
    zx = x.double().requires_grad_()

    def norm(u, weight):
        return u * (u.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * weight

    a = torch.nn.functional.pad(norm(zx, z["n1"]), (0, 0, 3, 0))
    p = z["bias"] + sum(a[:, i:i + L] * z["conv"][:, i] for i in range(4))
    zo = dense(*heads(p * torch.sigmoid(p) @ z["qkv"])).flatten(2) @ z["o"]
    zu = zo + zx
    zn = norm(zu, z["n2"])
    ((zn * g1).sum() + (zu * g2).sum()).backward()
    assert near(n2, zn, 6) and near(u1, zu, 6)
    assert near(b2["dweight"], z["n2"].grad, 7)
    assert near(y.flatten(2).flatten(0, 1).T @ b2["dx"].flatten(0, 1), z["o"].grad, 8)
    assert near(bc["dweight"], z["conv"].grad, 10) and near(bc["dbias"], z["bias"].grad, 10)
    assert near(b1["dweight"], z["n1"].grad, 11) and near(b1["dx"], zx.grad, 11)


def layer(x, w, attend, conv):
    n1, u = ssd.rms_norm_fwd(x, w["n1"], return_residual=True)
    o = attend(*heads(conv(n1) @ w["qkv"])).flatten(-2) @ w["o"]
    return ssd.rms_norm_fwd(o, w["n2"], u)


def test_a_prompt_and_single_tokens():
    w = weights(2)
    x = torch.randn((B, L, C), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    whole = layer(x, w, lambda q, k, v: ssd.window_attention_fwd(q, k, v, W, N),
                  lambda n: ssd.causal_conv_fwd(n, w["conv"], w["bias"]))
    kc, vc = (torch.zeros((B, KV, W + N, D), device="cuda") for _ in range(2))
    state = torch.zeros((B, 3, C), device="cuda")
    at = torch.zeros(B, dtype=torch.int32, device="cuda")
    cut = 100
    parts = [layer(x[:, :cut], w,
                   lambda q, k, v: ssd.window_attention_fwd(q, k, v, W, N, positions=at, k_cache=kc, v_cache=vc),
                   lambda n: ssd.causal_conv_fwd(n, w["conv"], w["bias"], state, True, final_out=state)[0])]
    at += cut
    for t in range(cut, L):
        y = layer(x[:, t], w, lambda q, k, v: ssd.window_attention_step(q, k, v, kc, vc, at, W, N),
                  lambda n: ssd.causal_conv_step(n, w["conv"], w["bias"], state))
        parts.append(y[:, None])
        at += 1
    assert near(torch.cat(parts, 1), whole, 6)


def test_eight_bits_before_a_product():
    # codes and scales stand for y: a product of what they stand for is within their rounding of the exact one
    w = weights(3)
    x = torch.randn((B, L, C), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    codes, scales = ssd.rms_norm_fwd(x, w["n1"], y_dtype=torch.float8_e4m3fn, scale_block=32)
    y = (codes.double().unflatten(-1, (-1, 32)) * scales.double()[..., None]).flatten(-2)
    exact = ssd.rms_norm_fwd(x, w["n1"]).double()
    # half a step of e4m3 is 2^-4 of a value at most (of 2^-6 scales below that); 2^-18 for y and the scale themselves
    least = 2.0 ** -6 * scales.double().repeat_interleave(32, -1)
    assert bool(((y - exact).abs() <= 2.0 ** -4 * torch.maximum(exact.abs(), least) + 2.0 ** -18 * exact.abs()).all())
    bound = (2.0 ** -4 * torch.maximum(exact.abs(), least) + 2.0 ** -18 * exact.abs()) @ w["qkv"].double().abs()
    assert bool(((y @ w["qkv"].double() - exact @ w["qkv"].double()).abs() <= bound).all())


def test_beside_the_chunked_scan_in_one_graph():
    # norm, scan over one group, norm, attention on the scan's output: replayed on other inputs
    w = weights(4)
    A = -torch.rand(4, device="cuda")

    def run(x, dt):
        n, u = ssd.rms_norm_fwd(x, w["n1"], return_residual=True)
        s = n.unflatten(-1, (4, 32))
        y = ssd.chunk_scan_fwd(s.contiguous(), dt, A, n[:, :, None, :16].contiguous(), n[:, :, None, 16:32].contiguous(), None, 64)
        m, u = ssd.rms_norm_fwd(y.flatten(2), w["n2"], u, return_residual=True)
        z, lse = ssd.window_attention_fwd(*heads(m @ w["qkv"]), W, N, return_lse=True)
        g = ssd.window_attention_bwd(*heads(m @ w["qkv"]), z, lse, z, W, N)
        return [u, z, *g.values()]

    gen = torch.Generator(device="cuda").manual_seed(5)
    sets = [(torch.randn((B, 128, C), generator=gen, device="cuda"), torch.rand((B, 128, 4), generator=gen, device="cuda"))
            for _ in range(4)]
    held = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(*held)
    for s in sets[1:]:
        for t, x in zip(held, s):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, run(*s)))
