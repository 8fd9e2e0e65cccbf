"""The fp64 oracle of attention with changed scores, pinned on the CPU: against
PyTorch's fp64 autograd of the definition, by finite differences, against the
plain attention oracle where nothing is changed, and in closed forms."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import score as so

CASES = {
    "plain": dict(),
    "cap": dict(cap=2.0),
    "slopes": dict(slopes=True),
    "both_window": dict(cap=1.5, slopes=True, window=3),
    "documents": dict(cap=3.0, doc=True),
    "prefix": dict(slopes=True, prefix=True),
    "full": dict(cap=1.0, slopes=True, causal=False),
}


def problem(name, B=2, H=4, Hk=2, N=9, d=8, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    kw = dict(CASES[name])
    kw["scale"] = 0.7
    kw.setdefault("causal", True)
    if kw.pop("slopes", None):
        kw["slopes"] = torch.tensor([0.5, -0.25, 0.0, 1.0], dtype=torch.float64)
    if kw.pop("doc", None):
        kw["doc"] = torch.tensor([[0, 0, 0, 3, 3, 5, 5, 5, 5], [0, 1, 1, 1, 1, 1, 1, 7, 7]])
    if kw.pop("prefix", None):
        kw["prefix"] = torch.tensor([4, 20])
    return t(B, H, N, d), t(B, Hk, N, d), t(B, Hk, N, d), t(B, H, N, d), kw


def by_torch(q, k, v, scale, causal=True, cap=0.0, slopes=None, window=0, doc=None, prefix=None):
    """(O, L) with autograd, masked pair by pair from the definition."""
    B, H, N, _ = q.shape
    g = H // k.shape[1]
    x = scale * torch.einsum("bhid,bhjd->bhij", q, k.repeat_interleave(g, 1))
    if cap:
        x = cap * torch.tanh(x / cap)
    mask = torch.zeros((B, N, N), dtype=torch.bool)
    for b in range(B):
        for i in range(N):
            for j in range(N):
                mask[b, i, j] = not causal or (
                    (j <= i and (not window or j > i - window) and (doc is None or j >= doc[b, i]))
                    or (prefix is not None and j < prefix[b]))
    if slopes is not None:
        at = torch.arange(N, dtype=torch.float64)
        x = x - slopes[:, None, None] * (at[:, None] - at[None, :]).abs()
    x = x.masked_fill(~mask[:, None], float("-inf"))
    return torch.softmax(x, -1) @ v.repeat_interleave(g, 1), torch.logsumexp(x, -1)


@pytest.mark.parametrize("name", list(CASES))
def test_against_autograd(name):
    q, k, v, do, kw = problem(name)
    qr, kr, vr = (t.clone().requires_grad_() for t in (q, k, v))
    o, lse = by_torch(qr, kr, vr, **kw)
    f = so.forward(q, k, v, **kw)
    np.testing.assert_allclose(f["O"], o.detach().numpy(), rtol=0, atol=1e-13)
    np.testing.assert_allclose(f["L"], lse.detach().numpy(), rtol=0, atol=1e-13)
    o.backward(do)
    b = so.backward(q, k, v, f["O"], do, f["L"], **kw)
    for n, t in (("dQ", qr), ("dK", kr), ("dV", vr)):
        np.testing.assert_allclose(b[n], t.grad.numpy(), rtol=0, atol=1e-12, err_msg=n)


@pytest.mark.parametrize("name", ["cap", "both_window", "prefix"])
def test_by_finite_differences(name):
    q, k, v, do, kw = problem(name, B=1, N=5, seed=3)
    if "prefix" in kw:
        kw["prefix"] = kw["prefix"][:1]
    loss = lambda *x: float(np.sum(so.forward(*x, **kw)["O"] * do.numpy()))  # noqa: E731
    f = so.forward(q, k, v, **kw)
    b = so.backward(q, k, v, f["O"], do, f["L"], **kw)
    h = 1e-5
    rng = np.random.default_rng(0)
    for w, n in ((0, "dQ"), (1, "dK"), (2, "dV")):
        for _ in range(12):
            at = tuple(rng.integers(0, s) for s in (q, k, v)[w].shape)
            x = [t.numpy().copy() for t in (q, k, v)]
            x[w][at] += h
            up = loss(*x)
            x[w][at] -= 2 * h
            assert abs((up - loss(*x)) / (2 * h) - b[n][at]) < 1e-7


@pytest.mark.parametrize("causal", [False, True])
def test_unchanged_scores_are_plain_attention(causal):
    q, k, v, do, _ = problem("plain", H=2, Hk=2)
    f = so.forward(q, k, v, causal=causal, scale=0.6)
    ref = oracle.attention_forward(q, k, v, causal, 0.6)
    np.testing.assert_allclose(f["O"], ref[0], rtol=0, atol=1e-13)
    np.testing.assert_allclose(f["L"], ref[1], rtol=0, atol=1e-13)


def test_closed_forms():
    # one key: O = V, L = the changed score, and no gradient but dV's
    q, k, v, do, kw = problem("cap", B=1, N=1)
    f = so.forward(q, k, v, **kw)
    g = np.repeat(k.numpy(), 2, axis=1)
    u = kw["scale"] * np.sum(q.numpy() * g, axis=-1)
    np.testing.assert_allclose(f["L"], kw["cap"] * np.tanh(u / kw["cap"]), atol=1e-14)
    np.testing.assert_allclose(f["O"], np.repeat(v.numpy(), 2, axis=1), atol=1e-14)
    b = so.backward(q, k, v, f["O"], do, f["L"], **kw)
    assert np.max(np.abs(b["dQ"])) < 1e-14 and np.max(np.abs(b["dK"])) < 1e-14
    # equal products: weights fall by e^-slope a step
    z = np.zeros((1, 1, 4, 8))
    val = np.arange(4.0)[None, None, :, None] * np.ones((1, 1, 4, 8))
    f = so.forward(z, z, val, slopes=np.array([math.log(2.0)]))
    w = np.array([1, 2, 4, 8]) / 15
    np.testing.assert_allclose(f["O"][0, 0, 3], w @ np.arange(4.0), atol=1e-14)
    # a cap far below the scores leaves two weights, e^cap apart from e^-cap
    q = np.ones((1, 1, 2, 8))
    k = np.stack([np.ones(8), -np.ones(8)])[None, None]
    f = so.forward(q, k, np.stack([np.ones(8), np.zeros(8)])[None, None], causal=False, scale=100.0,
                   cap=0.5)
    np.testing.assert_allclose(f["O"], 1 / (1 + math.exp(-1.0)), atol=1e-14)


def test_sums_of_probabilities():
    q, k, v, do, kw = problem("both_window", seed=5)
    f = so.forward(q, k, v, **kw)
    b = so.backward(q, k, v, f["O"], do, f["L"], **kw)
    np.testing.assert_allclose(b["dV"].sum(2), do.numpy().reshape(2, 2, 2, 9, 8).sum((2, 3)),
                               atol=1e-12)


def test_bounds_cover_their_roundings():
    """The forward's bound holds, and not by an order of magnitude, for the
    same sums with P and O rounded to bf16."""
    q, k, v, _, kw = problem("cap", N=64, d=64, H=2, Hk=1)
    q, k, v = (t.to(torch.bfloat16).double() for t in (q, k, v))
    kw["scale"] = 0.125
    f = so.forward(q, k, v, **kw)
    x = so.change(kw["scale"] * (q @ k.repeat_interleave(2, 1).transpose(2, 3)).numpy(), kw["cap"])[0]
    x = np.where(so.visible(64, True), x, -np.inf)
    p = torch.from_numpy(np.exp(x - x.max(-1, keepdims=True)))
    o = (p.to(torch.bfloat16).double() @ v.repeat_interleave(2, 1) / p.sum(-1, keepdim=True))
    off = np.abs(o.to(torch.bfloat16).double().numpy() - f["O"]) / f["dO"]
    assert 0.1 < off.max() <= 1.0
