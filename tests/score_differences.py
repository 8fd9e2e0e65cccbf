"""Differences along the gradient, for tests of gradients that a wrong one cannot
pass: problems, directions and what rounding may take (oracle/score.py)."""

import math

import numpy as np
import torch

from oracle import score as so

SHARP = [dict(cap=3.0, slopes=True), dict(cap=30.0), dict(slopes=True), dict(cap=3.0, causal=False)]


def sharp(cap=0.0, slopes=False, causal=True, N=150, d=64):
    """(q, k, v, do, arguments, cap) on the host: two query heads on one key head."""
    g = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn((1, h, N, d), generator=g) for h in (2, 1, 1, 2))
    q, k, v, do = (t.to(torch.bfloat16) for t in (2 * q, k, v, do))
    kw = dict(causal=causal, scale=1 / math.sqrt(d), window=0, doc=None, prefix=None,
              slopes=torch.tensor([0.0625, 0.00390625]) if slopes else None)
    return q, k, v, do, kw, cap


def along_the_gradient(q, k, v, do, kw, cap):
    """For each of q, k, v: a direction, <dO, O>'s slope along it by central
    differences of the fp64 forward, and what rounding may take from the slope
    that a kernel's gradient gives.

    The direction is the oracle's gradient, so the slope is a sum of squares.
    The kernel's gradient differs by the bounds of so.backward, independent from
    element to element: their root of squares, three times.  Its o (off by dO)
    enters by D, the same for a row: dx_ij moves by p_ij x'_ij dD_i, the slope by
    the sum of those over the row, rows independent."""
    f = so.forward(q, k, v, cap=cap, **kw)
    b = so.backward(q, k, v, f["O"], do, f["L"], cap=cap, **kw)
    x, y = [so._f64(t) for t in (q, k, v)], so._f64(do)
    g = x[0].shape[1] // x[1].shape[1]
    out = []
    for w, n in enumerate("QKV"):
        step = b["d" + n] / np.sqrt(np.mean(b["d" + n] ** 2))
        at = lambda e: np.sum(so.forward(*[t + e * step * (i == w) for i, t in enumerate(x)],  # noqa: E731
                                         cap=cap, **kw)["O"] * y)
        slope = (at(1e-4) - at(-1e-4)) / 2e-4
        room = 3 * math.sqrt(np.sum((b["e" + n] * step) ** 2))
        if n != "V":
            moved = 0.0
            for bb, h, hk, xs, der, seen, _ in so._heads(*x[:2], kw["causal"], cap, kw["slopes"],
                                                         kw["window"], kw["doc"], kw["prefix"],
                                                         kw["scale"]):
                p = np.where(seen, np.exp(np.where(seen, xs, 0.0) - f["L"][bb, h][:, None]), 0.0)
                u = step[bb, h] @ x[1][bb, hk].T if n == "Q" else x[0][bb, h] @ step[bb, hk].T
                dD = np.sum(np.abs(y[bb, h]) * f["dO"][bb, h], axis=-1)
                moved += np.sum((kw["scale"] * np.sum(p * der * u, axis=-1) * dD) ** 2)
            room += 3 * math.sqrt(moved)
        out.append((n, step, slope, room + 1e-6 * abs(slope)))
    return out, b
