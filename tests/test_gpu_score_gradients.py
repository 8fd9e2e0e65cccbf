"""Gradients of attention with changed scores: against differences along the
gradient itself, with slopes of either sign under a cap, and whole tensors of
longer sequences."""

import numpy as np
import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from score_differences import SHARP, along_the_gradient, sharp
from test_gpu_score import check, cuda_ready, problem  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [150, 300])
@pytest.mark.parametrize("case", SHARP)
def test_differences_along_the_gradient(case, N):
    """150 keys with the maximum, 300 without it (under a cap)."""
    q, k, v, do, kw, cap = sharp(N=N, **case)
    rows, _ = along_the_gradient(q, k, v, do, kw, cap)
    q, k, v, do = (t.cuda() for t in (q, k, v, do))
    kw["slopes"] = kw["slopes"].cuda() if kw["slopes"] is not None else None
    o, lse = ab.attn_fwd_score(q, k, v, softcap=cap, **kw)
    got = ab.attn_bwd_score(q, k, v, o, do, lse, softcap=cap, **kw)
    for (n, step, slope, room), t in zip(rows, got):
        assert room < 0.05 * abs(slope), n
        mine = float(np.sum(t.double().cpu().numpy() * step))
        assert abs(mine - slope) <= room, "d%s: %.4g for %.4g, room %.2g" % (n, mine, slope, room)


@pytest.mark.parametrize("N", [200, 300])  # with the maximum, and without
@pytest.mark.parametrize("slope", [-0.05, -3.0, -200.0, 3.0, 200.0])
@pytest.mark.parametrize("more", [dict(causal=False), dict(), dict(window=270), dict(mask="doc"),
                                  dict(mask="prefix")])
def test_slopes_of_either_sign_under_a_cap(slope, more, N):
    """The largest bias of a row is at its own key or at the farthest it sees."""
    q, k, v, do, kw, cap = problem(N, 64, B=2, cap=20.0, gain=3.0, seed=N, **more)
    kw["slopes"] = torch.tensor([slope, -0.1], device="cuda")
    check(q, k, v, do, kw, cap)


@pytest.mark.parametrize("d,more", [(64, dict(cap=50.0, gain=4.0)), (128, dict(cap=50.0, gain=4.0)),
                                    (128, dict(slopes=True)),
                                    (64, dict(cap=100.0, gain=6.0, slopes=True, causal=False))])
def test_longer_sequences(d, more):
    check(*problem(2311, d, H=2, Hk=1, seed=8, **more))
