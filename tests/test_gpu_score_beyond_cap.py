"""Gradients of attention whose raw scores lie far beyond the cap, on the GPU
against fp64 within bounds that are relative to each weight."""

import math

import numpy as np
import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from oracle import score as so
from test_gpu_score import cuda_ready, problem  # noqa: F401

pytestmark = pytest.mark.gpu

BF16, FP16 = so.BF16, so.FP16


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hk", [2, 1])
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("side", [1.0, -1.0])
def test_gradients_beyond_the_cap(side, slopes, Hk, d):
    """Raw scores of eight caps, of either sign: 1 - tanh^2 is 2^-21, and dQ and
    dK, which are sums of it, hold as many digits on both sides.

    An element of dx is off by its roundings to fp16 and bf16, P's and x's own
    errors, and x' 's: 2^-18 of itself (an exponential and a reciprocal of
    2^-22 each, an argument of some 30 in fp32) and twice the score's error in
    caps, which is d + 8 terms' in fp32."""
    N, H, cap = 96, 2, 1.0
    q, k, v, do, kw, _ = problem(N, d, H=H, Hk=Hk, causal=False, slopes=slopes, seed=d + Hk)
    q, k = q * 0.3, k * 0.3
    q[..., 0], k[..., 0] = side * 8.0, math.sqrt(d)
    q, k = q.to(torch.bfloat16), k.to(torch.bfloat16)
    o, lse = ab.attn_fwd_score(q, k, v, softcap=cap, **kw)
    dq, dk, _ = ab.attn_bwd_score(q, k, v, o, do, lse, softcap=cap, **kw)
    Q, K, V, O, Y, L = (so._f64(t) for t in (q, k, v, o, do, lse))
    s = kw["scale"]
    want, room = [np.zeros(Q.shape), np.zeros(K.shape)], [np.zeros(Q.shape), np.zeros(K.shape)]
    for b, h, hk, x, der, seen, mag in so._heads(Q, K, False, cap, kw["slopes"], 0, None, None, s):
        raw = s * (Q[b, h] @ K[b, hk].T) / cap
        assert raw.min() * side > 5 or raw.max() * side > 5
        p = np.exp(x - L[b, h][:, None])
        dP, D = Y[b, h] @ V[b, hk].T, np.sum(Y[b, h] * O[b, h], axis=-1, keepdims=True)
        dx = p * (dP - D) * der
        raw_err = mag * (d + 8) * 2.0 ** -23 / cap
        err = (so.score_error(mag, seen, d, cap, kw["slopes"], N) + 4 * so.FP32 * np.abs(L[b, h])
               + 2.0 ** -21)[:, None]
        edP = (np.abs(Y[b, h]) @ np.abs(V[b, hk]).T + np.sum(np.abs(Y[b, h] * O[b, h]), axis=-1,
                                                             keepdims=True)) * (d + 2) * 2.0 ** -23
        e = 1.01 * (np.abs(dx) * (FP16 + BF16 + 2 * err + 2 * raw_err + 2.0 ** -18)
                    + 2.0 ** -39 * np.abs(dP - D) + p * der * edP) + H * N * 2.0 ** -23 * np.abs(dx)
        want[0][b, h], room[0][b, h] = s * (dx @ K[b, hk]), s * (e @ np.abs(K[b, hk]))
        want[1][b, hk] += s * (dx.T @ Q[b, h])
        room[1][b, hk] += s * (e.T @ np.abs(Q[b, h]))
    for got, ref, e, n in ((dq, want[0], room[0], "dQ"), (dk, want[1], room[1], "dK")):
        off = np.abs(got.double().cpu().numpy() - ref) / (e + BF16 * np.abs(ref) + 2.0 ** -133)
        assert off.max() <= 1.0, "%s: %.3f of its bound" % (n, off.max())
