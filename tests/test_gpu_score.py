"""Attention with changed scores on the GPU against the fp64 oracle, element by
element, within bounds that count every rounding (oracle/score.py).

Lengths around the 64- and 128-row tiles, every mask with every change of the
scores, shared key heads, strided operands, caps far below and far above the
scores, gradients against differences, and what must repeat."""

import itertools
import math

import numpy as np
import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from oracle import score as so

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_backward_pass_attn_gb300 import build as abuild

    abuild.build()
    ab.load_library()
    assert ab.attn_last_device_error() == ab.ATTN_OK
    yield
    assert ab.attn_last_device_error() == ab.ATTN_OK


def randn(shape, g, gain=1.0):
    return (torch.randn(shape, generator=g) * gain).to(torch.bfloat16).cuda()


def documents(B, N, seed):
    g = torch.Generator().manual_seed(seed)
    doc = torch.zeros((B, N), dtype=torch.int32)
    for b in range(B):
        start = 0
        for i in range(N):
            if float(torch.rand((), generator=g)) < 6 / max(N, 6):
                start = i
            doc[b, i] = start
    return doc.cuda()


def ladder(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")


def problem(N, d, H=2, Hk=1, B=1, seed=0, gain=1.0, cap=0.0, slopes=False, mask="none", window=0,
            causal=True):
    g = torch.Generator().manual_seed(seed)
    q, k, v = randn((B, H, N, d), g, gain), randn((B, Hk, N, d), g), randn((B, Hk, N, d), g)
    do = randn((B, H, N, d), g)
    kw = dict(causal=causal, scale=1 / math.sqrt(d), window=window,
              doc=documents(B, N, seed) if mask == "doc" else None, prefix=None,
              slopes=ladder(H) if slopes else None)
    if mask == "prefix":
        kw["prefix"] = torch.tensor([(N * (b + 1)) // 3 for b in range(B)], dtype=torch.int32).cuda()
    return q, k, v, do, kw, cap


def host(kw):
    return {n: t.cpu() if isinstance(t, torch.Tensor) else t for n, t in kw.items()}


def within(got, want, bound, name):
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape
    assert np.all(np.isfinite(got)), name
    off = np.abs(got - want) / bound
    assert off.max(initial=0.0) <= 1.0, "%s: %.3f of its bound at %s" % (
        name, off.max(), np.unravel_index(off.argmax(), off.shape))


def check(q, k, v, do, kw, cap, backward=True):
    o, lse = ab.attn_fwd_score(q, k, v, softcap=cap, **kw)
    f = so.forward(q, k, v, cap=cap, **host(kw))
    within(o, f["O"], f["dO"], "O")
    within(lse, f["L"], f["dL"], "L")
    if not backward:
        return
    got = ab.attn_bwd_score(q, k, v, o, do, lse, softcap=cap, **kw)
    b = so.backward(q, k, v, o, do, lse, cap=cap, **host(kw))
    for t, n in zip(got, "QKV"):
        within(t, b["d" + n], b["e" + n], "d" + n)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 384, 513])
def test_lengths(N, d):
    check(*problem(N, d, gain=4.0, cap=20.0, slopes=True, seed=N))


CHANGES = {"none": {}, "cap": dict(cap=15.0, gain=4.0), "slopes": dict(slopes=True),
           "both": dict(cap=15.0, gain=4.0, slopes=True)}
MASKS = {"full": dict(causal=False), "causal": {}, "window": dict(window=270), "narrow": dict(window=1),
         "doc": dict(mask="doc"), "doc_window": dict(mask="doc", window=33), "prefix": dict(mask="prefix")}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("change,mask", list(itertools.product(CHANGES, MASKS)))
def test_changes_and_masks(change, mask, d):
    check(*problem(333, d, B=2, seed=7, **CHANGES[change], **MASKS[mask]))


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (8, 2), (6, 6), (16, 1)])
@pytest.mark.parametrize("mask", ["full", "causal", "doc", "prefix"])
def test_shared_key_heads(H, Hk, mask):
    check(*problem(200, 64, H=H, Hk=Hk, B=2, seed=H, cap=10.0, gain=3.0, slopes=True, **MASKS[mask]))


@pytest.mark.parametrize("N", [190, 290])  # with the maximum and without
@pytest.mark.parametrize("cap", [1e-3, 0.05, 1.0, 7.0, 50.0, 1e4, 1e30])
@pytest.mark.parametrize("gain", [0.02, 1.0, 12.0])
def test_caps(cap, gain, N):
    """Every score above the cap, every score far below it, and both."""
    check(*problem(N, 128, cap=cap, gain=gain, seed=2))


def test_a_row_that_sees_one_key_returns_its_value():
    q, k, v, _, kw, _ = problem(300, 64, H=2, Hk=2)
    for more in (dict(window=1), dict(doc=torch.arange(300, dtype=torch.int32).cuda()[None])):
        o, _ = ab.attn_fwd_score(q, k, v, softcap=0.0, **dict(kw, **more))
        assert torch.equal(o, v)
    o, _ = ab.attn_fwd_score(q, k, v, softcap=30.0, **dict(kw, window=1))
    assert torch.equal(o, v)


def test_a_cap_out_of_reach_changes_little():
    q, k, v, _, kw, _ = problem(300, 64, gain=2.0)
    o, lse = ab.attn_fwd_score(q, k, v, softcap=1e6, **kw)
    _, plain = ab.attn_fwd_score(q, k, v, **kw)
    # tanh(y) = y (1 - y^2 / 3 ...), the polynomial's 6e-8 and fp32 steps
    assert float((lse - plain).abs().max()) <= 2e-6 * float(plain.abs().max() + 40)
    assert float((o.float() - ab.attn_fwd_score(q, k, v, **kw)[0].float()).abs().max()) <= 2 ** -6


@pytest.mark.parametrize("slope", [-0.05, 0.0, 3.0, 1000.0])
@pytest.mark.parametrize("causal", [False, True])
def test_slopes(slope, causal):
    """Negative ones prefer what is far; steep ones leave the row's own key."""
    q, k, v, do, kw, cap = problem(260, 64, causal=causal)
    kw["slopes"] = torch.tensor([slope, 0.1], device="cuda")
    check(q, k, v, do, kw, cap)


@pytest.mark.parametrize("prefix", [[-5, 0], [1, 128], [129, 299], [300, 301], [2 ** 31 - 1, 64]])
@pytest.mark.parametrize("d", [64, 128])
def test_prefixes(prefix, d):
    q, k, v, do, kw, cap = problem(300, d, B=2, cap=8.0, gain=3.0, slopes=True)
    kw["prefix"] = torch.tensor(prefix, dtype=torch.int32).cuda()
    check(q, k, v, do, kw, cap)


@pytest.mark.parametrize("window", [1, 2, 127, 128, 129, 499, 500, 2 ** 31 - 1, 2 ** 40])
def test_windows(window):
    q, k, v, do, kw, cap = problem(500, 64, cap=9.0, gain=2.0)
    o, lse = ab.attn_fwd_score(q, k, v, softcap=cap, **dict(kw, window=window))
    f = so.forward(q, k, v, cap=cap, **host(dict(kw, window=window)))
    within(o, f["O"], f["dO"], "O")
    got = ab.attn_bwd_score(q, k, v, o, do, lse, softcap=cap, **dict(kw, window=window))
    b = so.backward(q, k, v, o, do, lse, cap=cap, **host(dict(kw, window=window)))
    for t, n in zip(got, "QKV"):
        within(t, b["d" + n], b["e" + n], "d" + n)


def test_operands_as_a_projection_leaves_them():
    """Heads of one fused [B][N][heads][d] tensor, bit for bit the same as
    contiguous copies; and rows with room between them."""
    g = torch.Generator().manual_seed(4)
    B, N, H, Hk, d = 2, 201, 4, 2, 64
    x = randn((B, N, H + 2 * Hk, d), g)
    q, k, v = (t.transpose(1, 2) for t in x.split((H, Hk, Hk), dim=2))
    do = randn((B, H, N, d), g)
    wide = torch.zeros((B, H, N, d + 8), dtype=torch.bfloat16, device="cuda")
    wide[..., :d] = q
    kw = dict(causal=True, softcap=5.0, slopes=ladder(H))
    want = ab.attn_fwd_score(q.contiguous(), k.contiguous(), v.contiguous(), **kw)
    wantg = ab.attn_bwd_score(q.contiguous(), k.contiguous(), v.contiguous(), want[0], do, want[1], **kw)
    for qq in (q, wide[..., :d]):
        o, lse = ab.attn_fwd_score(qq, k, v, **kw)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        dq, dk, dv = ab.attn_bwd_score(qq, k, v, o, do, lse, **kw)
        assert torch.equal(dk, wantg[1]) and torch.equal(dv, wantg[2])
        assert float((dq.float() - wantg[0].float()).abs().max()) <= 2 ** -7 * float(dq.abs().max())


def test_dk_and_dv_repeat_bit_for_bit():
    q, k, v, do, kw, cap = problem(700, 128, H=8, Hk=2, cap=6.0, gain=3.0)
    o, lse = ab.attn_fwd_score(q, k, v, softcap=cap, **kw)
    first = ab.attn_bwd_score(q, k, v, o, do, lse, softcap=cap, **kw)
    for _ in range(5):
        again = ab.attn_fwd_score(q, k, v, softcap=cap, **kw)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
        got = ab.attn_bwd_score(q, k, v, o, do, lse, softcap=cap, **kw)
        assert torch.equal(got[1], first[1]) and torch.equal(got[2], first[2])
        # dQ: fp32 sums in another order, then one rounding to bf16
        assert float((got[0].float() - first[0].float()).abs().max()) <= 2 ** -7 * float(first[0].abs().max())


def test_gradients_against_differences():
    """<dO, O> along random directions: central differences of the fp64 oracle
    at steps its curvature and rounding both leave room for."""
    q, k, v, do, kw, cap = problem(150, 64, H=2, Hk=1, cap=3.0, gain=2.0, slopes=True)
    o, lse = ab.attn_fwd_score(q, k, v, softcap=cap, **kw)
    got = ab.attn_bwd_score(q, k, v, o, do, lse, softcap=cap, **kw)
    x = [t.double().cpu().numpy() for t in (q, k, v)]
    y = do.double().cpu().numpy()
    bound = so.backward(q, k, v, o, do, lse, cap=cap, **host(kw))
    rng = np.random.default_rng(1)
    for w, n in enumerate("QKV"):
        step = rng.standard_normal(x[w].shape)
        at = lambda e: np.sum(so.forward(*[t + e * step * (i == w) for i, t in enumerate(x)],  # noqa: E731
                                         cap=cap, **host(kw))["O"] * y)
        slope = (at(1e-4) - at(-1e-4)) / 2e-4
        mine = float(np.sum(got[w].double().cpu().numpy() * step))
        # the kernel's o is rounded to bf16 and enters D: 2^-8 of sum p dp x
        room = float(np.sum(bound["e" + n] * np.abs(step))) + 2 ** -8 * abs(slope) + 1e-6
        assert abs(mine - slope) <= room


@pytest.mark.parametrize("N,d,more", [
    (1100, 64, dict(cap=12.0, gain=4.0, window=300)), (390, 128, dict(cap=12.0, gain=4.0, causal=False)),
    (300, 64, dict(causal=False, slopes=True)), (390, 128, dict(slopes=True, mask="prefix")),
    (520, 128, dict(cap=100.0, gain=4.0, slopes=True))])
def test_many_heads(N, d, more):
    """More tasks and items than blocks, tasks of two query tiles, several
    rounds of each block."""
    check(*problem(N, d, H=24, Hk=8, B=3, **more))


def test_error_word_stays_clear_after_odd_document_maps():
    """Entries outside [0, i] are clamped: values of no meaning, no fault."""
    q, k, v, do, kw, _ = problem(400, 64)
    kw["doc"] = torch.randint(-1000, 1000, (1, 400), generator=torch.Generator().manual_seed(1),
                              dtype=torch.int32).cuda()
    o, lse = ab.attn_fwd_score(q, k, v, **kw)
    ab.attn_bwd_score(q, k, v, o, do, lse, **kw)
    assert ab.attn_last_device_error() == ab.ATTN_OK


@pytest.mark.parametrize("H,Hk,B,mask", [(8, 1, 1, "causal"), (8, 1, 1, "full"), (6, 1, 2, "doc_window"),
                                         (12, 2, 1, "prefix"), (12, 1, 1, "window")])
@pytest.mark.parametrize("d", [64, 128])
def test_a_key_heads_sums_in_several_blocks(H, Hk, B, mask, d):
    """Few key heads: their query heads are dealt to several blocks, whose sums
    are joined in order, the same bits every time."""
    N = 401
    assert ab.load_library().attn_bwd_score_workspace_size(B, H, Hk, N, d, 1, 0) \
        > ab.attn_bwd_workspace_size(B, H, N, d)
    p = problem(N, d, H=H, Hk=Hk, B=B, cap=9.0, gain=3.0, slopes=True, seed=4, **MASKS[mask])
    check(*p)
    q, k, v, do, kw, cap = p
    o, lse = ab.attn_fwd_score(q, k, v, softcap=cap, **kw)
    a, b = (ab.attn_bwd_score(q, k, v, o, do, lse, softcap=cap, **kw) for _ in range(2))
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,slopes", [(0.0, False), (40.0, False), (0.0, True), (40.0, True)])
def test_gradients_of_keys_that_every_row_sees_a_little_of(cap, slopes, d):
    """Keys of weights around 2^-20 to 2^-27: their own dK holds as well as any."""
    q, k, v, do, kw, _ = problem(300, d, causal=False, slopes=slopes)
    q[..., 0], k[..., 0] = 8.0, 0.0
    k[:, :, 100:, 0] = -1.25 * math.sqrt(d)  # e^-10 (capped at 40: e^-9.8) of the others
    k[:, :, 200:, 0] = -1.75 * math.sqrt(d)  # e^-14 (e^-13.5)
    check(q, k, v, do, kw, cap)
