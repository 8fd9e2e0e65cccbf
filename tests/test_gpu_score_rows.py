"""Rows of the forward with changed scores that see little, and blocks that walk
many short tasks, on the GPU against the fp64 oracle (oracle/score.py)."""

import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from oracle import score as so
from test_gpu_score import cuda_ready, host, problem, within  # noqa: F401

pytestmark = pytest.mark.gpu


def starts_of_tiles(B, N):
    """Documents of one 128-row tile each."""
    return (torch.arange(N, dtype=torch.int32) // 128 * 128).expand(B, N).contiguous().cuda()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,N,documents", [
    (4, 16, 512, False),  # tasks of one query tile, the last blocks' of one key tile
    (4, 16, 512, True),   # every task of one key tile
    (4, 64, 384, True)])  # tasks of two query tiles, and of one at the end, of one key tile
@pytest.mark.parametrize("slopes", [False, True])
def test_tasks_of_one_key_tile_behind_others(B, H, N, documents, slopes, d):
    """A block's tasks follow one another through shared memory, in which the
    halves of a row exchange their sums: a task with one key tile must not be
    ahead of what the one before it still reads."""
    q, k, v, _, kw, cap = problem(N, d, B=B, H=H, Hk=H // 4, cap=50.0, gain=3.0, slopes=slopes,
                                  seed=B + d)
    if documents:
        kw["doc"] = starts_of_tiles(B, N)
    o, lse = ab.attn_fwd_score(q, k, v, softcap=cap, **kw)
    f = so.forward(q, k, v, cap=cap, **host(kw))
    within(o, f["O"], f["dO"], "O")
    within(lse, f["L"], f["dL"], "L")
    off = torch.zeros((), dtype=torch.bool, device="cuda")
    for _ in range(300):
        o2, lse2 = ab.attn_fwd_score(q, k, v, softcap=cap, **kw)
        off |= (o2 != o).any() | (lse2 != lse).any()
    assert not off


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [5.0, 30.0, 50.0])
@pytest.mark.parametrize("slopes", [False, True])
def test_a_row_that_sees_one_key_returns_its_value_under_a_cap(cap, slopes, d):
    """Its weight is 1 whatever its score, also among rows that see more: the
    first of a causal sequence, and of every document."""
    N = 600
    q, k, v, _, kw, _ = problem(N, d, H=3, Hk=3, gain=3.0, slopes=slopes, seed=d)
    starts = torch.tensor([0, 1, 2, 31, 32, 40, 127, 128, 300, 301, 599], dtype=torch.int32)
    doc = torch.zeros(N, dtype=torch.int32)
    for s in starts.tolist():
        doc[s:] = s
    at = starts.cuda()
    for more, rows in ((dict(), at[:1]), (dict(doc=doc.cuda()[None]), at),
                       (dict(doc=doc.cuda()[None], window=260), at),
                       (dict(doc=torch.arange(N, dtype=torch.int32).cuda()[None]), slice(None))):
        o, _ = ab.attn_fwd_score(q, k, v, softcap=cap, **dict(kw, **more))
        assert torch.equal(o[:, :, rows], v[:, :, rows])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [30.0, 50.0])
def test_rows_of_one_key_have_no_gradient(cap, d):
    """A row with one key weighs it by 1 whatever its score: with o = v exactly,
    dP - D is fp32 rounding, and dQ and dK are no more than the bounds around
    zero (oracle/score.py)."""
    N = 300
    q, k, v, do, kw, _ = problem(N, d, H=2, Hk=2, seed=d)
    kw["doc"] = torch.arange(N, dtype=torch.int32).cuda()[None]
    o, lse = ab.attn_fwd_score(q, k, v, softcap=cap, **kw)
    dq, dk, dv = ab.attn_bwd_score(q, k, v, o, do, lse, softcap=cap, **kw)
    b = so.backward(q, k, v, v, do, lse, cap=cap, **host(kw))
    for t, n in ((dq, "Q"), (dk, "K"), (dv, "V")):
        within(t, b["d" + n], b["e" + n], "d" + n)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("cap", [0.0, 30.0, 100.0])
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("N", [200, 400])
def test_keys_that_no_row_sees_may_hold_anything(N, slopes, cap, bad):
    """Keys behind a row, before its document or outside its window leave its
    bits as they were, in forward form with the maximum and without."""
    q, k, v, _, kw, _ = problem(N, 64, gain=3.0, slopes=slopes, seed=N)
    doc = torch.zeros(N, dtype=torch.int32)
    doc[N // 2:] = N // 2
    for more, hidden, rows in ((dict(), slice(N - 7, N), slice(0, N - 7)),
                               (dict(doc=doc.cuda()[None]), slice(0, N // 2), slice(N // 2, N)),
                               (dict(window=70), slice(0, 20), slice(100, N))):
        want = ab.attn_fwd_score(q, k, v, softcap=cap, **dict(kw, **more))
        odd = k.clone()
        odd[:, :, hidden] = bad
        got = ab.attn_fwd_score(q, odd, v, softcap=cap, **dict(kw, **more))
        for a, b in zip(got, want):
            assert torch.equal(a[:, :, rows], b[:, :, rows])
