"""fp64 oracle of attention with changed scores (a tanh cap, a bias that falls
with distance, a prefix mask, shared key heads), forward and backward, and of
how far a kernel's rounding may take each result from it.

TEST INFRASTRUCTURE ONLY (like the rest of ``oracle/``); it shares no code with
the CUDA path.  Whole N x N matrices of one head at a time, straight from the
definitions; every function takes torch tensors or numpy arrays and works on
float64 numpy arrays.
"""

from __future__ import annotations

import numpy as np

from . import _f64

BF16, FP16, FP32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24  # half a step, relative


def visible(N: int, causal: bool, window: int = 0, doc=None, prefix=None) -> np.ndarray:
    """bool [N, N]: whether query i sees key j; doc [N], prefix a number."""
    i, j = np.arange(N)[:, None], np.arange(N)[None, :]
    if not causal:
        return np.ones((N, N), dtype=bool)
    seen = j <= i
    if window > 0:
        seen &= j > i - window
    if doc is not None:
        seen &= j >= np.asarray(doc).astype(np.int64)[:, None]
    if prefix is not None:
        seen |= j < int(prefix)
    return seen


def change(u, cap: float = 0.0, slope: float = 0.0, dist=0.0):
    """(x, dx/du) of scaled products u at distances dist."""
    u = np.asarray(u, dtype=np.float64)
    if cap:
        t = np.tanh(u / cap)
        x, der = cap * t, 1.0 - t * t
    else:
        x, der = u, np.ones_like(u)
    return x - slope * np.abs(dist), der


def _heads(q, k, causal, cap, slopes, window, doc, prefix, scale):
    """Per query head: (b, h, key head, u, x, dx/du, mask, |q| |k| scale)."""
    B, H, N, _ = q.shape
    g = H // k.shape[1]
    dist = np.arange(N)[:, None] - np.arange(N)[None, :]
    for b in range(B):
        seen = visible(N, causal, window, None if doc is None else _f64(doc)[b],
                       None if prefix is None else _f64(prefix)[b])
        for h in range(H):
            u = scale * (q[b, h] @ k[b, h // g].T)
            x, der = change(u, cap, 0.0 if slopes is None else float(_f64(slopes)[h]), dist)
            mag = scale * (np.abs(q[b, h]) @ np.abs(k[b, h // g]).T)
            yield b, h, h // g, x, der, seen, mag


def score_error(mag, seen, d, cap, slopes, N):
    """A bound on the error of a computed score, base e: the product's d terms
    added in fp32 (a tensor core truncates: 2^-23 each), the factors and the
    cap's roundings (2^-21 of the cap beyond the polynomial, fp32 steps of the
    score within it), the bias's product and sum."""
    top = np.max(np.where(seen, mag, 0.0), axis=-1, initial=0.0)
    e = top * (d + 8) * 2.0 ** -23
    if cap:
        e = e + 2.0 ** -21 * cap
    if slopes is not None:
        e = e + 2.0 ** -22 * float(np.max(np.abs(_f64(slopes)))) * N
    return e  # [N]


def forward(q, k, v, causal=True, scale=1.0, cap=0.0, slopes=None, window=0, doc=None, prefix=None):
    """dict of O [B, H, N, d], L [B, H, N] and their bounds dO, dL: P rounded
    to bf16 for its product with V, O rounded to bf16, scores off by
    score_error, sums of N terms in fp32, exponentials to 2^-21."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, H, N, d = q.shape
    out = {n: np.zeros((B, H, N, d)) for n in ("O", "dO")}
    out.update({n: np.zeros((B, H, N)) for n in ("L", "dL")})
    for b, h, hk, x, _, seen, mag in _heads(q, k, causal, cap, slopes, window, doc, prefix, scale):
        x = np.where(seen, x, -np.inf)
        m = np.max(x, axis=-1, keepdims=True)
        e = np.exp(x - m)
        z = np.sum(e, axis=-1, keepdims=True)
        p = e / z
        out["O"][b, h] = p @ v[b, hk]
        out["L"][b, h] = (m + np.log(z))[:, 0]
        err = score_error(mag, seen, d, cap, slopes, N) + 2.0 ** -21 + N * FP32
        out["dL"][b, h] = err + 4 * FP32 * np.abs(out["L"][b, h]) + 4 * FP32 * np.abs(m[:, 0])
        A = p @ np.abs(v[b, hk])
        out["dO"][b, h] = BF16 * np.abs(out["O"][b, h]) \
            + (BF16 + 2 * err[:, None] + N * 2.0 ** -23) * 1.01 * A
    return out


def backward(q, k, v, o, do, lse, causal=True, scale=1.0, cap=0.0, slopes=None, window=0, doc=None,
             prefix=None):
    """dict of dQ, dK, dV from the given o and lse, and bounds eQ, eK, eV: P
    and dx each rounded to bf16 once, P x' to fp16 (2^-39 absolute below its
    range, held times 2^14), 1 - tanh^2 off by 2^-20, sums of N (d) terms in fp32."""
    q, k, v, o, do, lse = (_f64(t) for t in (q, k, v, o, do, lse))
    B, H, N, d = q.shape
    g = H // k.shape[1]
    out = {n: np.zeros(q.shape) for n in ("dQ", "eQ")}
    out.update({n: np.zeros(k.shape) for n in ("dK", "dV", "eK", "eV")})
    for b, h, hk, x, der, seen, mag in _heads(q, k, causal, cap, slopes, window, doc, prefix, scale):
        L = lse[b, h][:, None]
        p = np.where(seen, np.exp(np.where(seen, x, 0.0) - L), 0.0)
        dP = do[b, h] @ v[b, hk].T
        D = np.sum(do[b, h] * o[b, h], axis=-1, keepdims=True)
        dx = p * (dP - D) * der
        out["dV"][b, hk] += p.T @ do[b, h]
        out["dQ"][b, h] = scale * (dx @ k[b, hk])
        out["dK"][b, hk] += scale * (dx.T @ q[b, h])
        err = (score_error(mag, seen, d, cap, slopes, N) + 4 * FP32 * np.abs(lse[b, h])
               + 2.0 ** -21)[:, None]
        eP = p * (2 * err) * 1.01
        edP = (np.abs(do[b, h]) @ np.abs(v[b, hk]).T
               + np.sum(np.abs(do[b, h] * o[b, h]), axis=-1, keepdims=True)) * (d + 2) * 2.0 ** -23
        tail = (FP16 + BF16) * np.abs(dx) + np.where(seen, 2.0 ** -39, 0.0) * np.abs(dP - D)
        edx = 1.01 * (tail + (eP * der + p * (2.0 ** -20 if cap else 0.0)) * np.abs(dP - D)
                      + p * der * edP)
        sums = N * 2.0 ** -23
        out["eV"][b, hk] += (BF16 * p + eP + sums * p).T @ np.abs(do[b, h]) * 1.01
        out["eQ"][b, h] = scale * ((edx + sums * np.abs(dx)) @ np.abs(k[b, hk]))
        out["eK"][b, hk] += scale * ((edx + g * sums * np.abs(dx)).T @ np.abs(q[b, h]))
    for n, e in (("dQ", "eQ"), ("dK", "eK"), ("dV", "eV")):
        out[e] += BF16 * np.abs(out[n]) + 2.0 ** -133  # the result's own rounding
    return out


def decode(q, kvals, vvals, page_table, seq_lens, scale, window=0, cap=0.0, slopes=None):
    """The newest token of each sequence over its pages: dict of O [B, H, d],
    L [B, H] and bounds dO, dL.  kvals, vvals: float64 [pages, Hkv, page_size,
    d].  Bounds: scores off by score_error, exponentials to 2^-21, weights of
    16 bits for V, sums of n terms in fp32, O's rounding to bf16."""
    q = _f64(q)
    B, H, d = q.shape[0], q.shape[1], q.shape[-1]
    q = q.reshape(B, H, d)
    table = np.asarray(_f64(page_table)).astype(np.int64)
    page = kvals.shape[2]
    g = H // kvals.shape[1]
    out = {"O": np.zeros((B, H, d)), "L": np.full((B, H), -np.inf), "dO": np.zeros((B, H, d)),
           "dL": np.zeros((B, H))}
    for b in range(B):
        n = int(seq_lens[b])
        at = np.arange(max(0, n - window) if window else 0, n)
        if not len(at):
            continue
        rows = table[b, at // page], at % page
        for h in range(H):
            k, v = kvals[rows[0], h // g, rows[1]], vvals[rows[0], h // g, rows[1]]
            sl = 0.0 if slopes is None else float(_f64(slopes)[h])
            x, _ = change(scale * (k @ q[b, h]), cap, sl, n - 1 - at)
            m = np.max(x)
            e = np.exp(x - m)
            p = e / np.sum(e)
            mag = scale * (np.abs(k) @ np.abs(q[b, h]))
            err = float(score_error(mag, np.ones(len(at), dtype=bool), d, cap,
                                    None if slopes is None else [sl], n))
            err += 2.0 ** -21 + len(at) * FP32
            out["O"][b, h], out["L"][b, h] = p @ v, m + np.log(np.sum(e))
            out["dL"][b, h] = err + 4 * FP32 * (abs(out["L"][b, h]) + abs(m))
            out["dO"][b, h] = BF16 * np.abs(out["O"][b, h]) \
                + (2 * err + 2.0 ** -15 + len(at) * 2.0 ** -22) * 1.01 * (p @ np.abs(v)) \
                + 2.0 ** -133  # a zero's own
    return out
