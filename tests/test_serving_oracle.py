"""The fp64 oracle of the answering path (``oracle/serving.py``) against what
does not depend on it: finite differences, invariants, brute force over every
8-bit value, and the attention oracle.  CPU only."""

import math

import numpy as np
import pytest

import oracle
from oracle import serving
from oracle.fp8 import e4m3_to_f64

RNG = np.random.default_rng


def rope_case(seed=0, B=2, H=3, N=5, d=8, sections=(1, 3), interleaved=False):
    rng = RNG(seed)
    x = rng.standard_normal((B, H, N, d))
    pos = rng.integers(-50, 50, (len(sections), B, N))
    f = rng.uniform(0.01, 1.0, d // 2)
    return x, pos, f, sections, interleaved


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sections", [(4,), (1, 3), (2, 1, 1), (1, 1, 1, 1), (0, 4)])
def test_rope_gradient_against_differences(sections, interleaved):
    """d<g, rope(x)>/dx by central differences (exact for a linear map up to
    rounding: 1e-16 / 1e-3 of values near 1) is the inverse turn of g."""
    x, pos, f, sections, il = rope_case(1, B=1, H=1, N=3, sections=sections,
                                        interleaved=interleaved)
    g = RNG(2).standard_normal(x.shape)
    grad = serving.rope(g, pos, f, sections, il, inverse=True)
    h = 1e-3
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        num = np.sum(g * (serving.rope(x + e, pos, f, sections, il)
                          - serving.rope(x - e, pos, f, sections, il))) / (2 * h)
        assert abs(num - grad[i]) < 1e-11


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_invariants(interleaved):
    """Lengths are kept, position 0 changes nothing, the inverse undoes the
    turn, and scores depend on the difference of positions only."""
    x, pos, f, sec, il = rope_case(3, interleaved=interleaved)
    y = serving.rope(x, pos, f, sec, il)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-13)
    assert np.array_equal(serving.rope(x, pos * 0, f, sec, il), x)
    assert np.allclose(serving.rope(y, pos, f, sec, il, inverse=True), x, atol=1e-13)
    k = RNG(4).standard_normal(x.shape)
    z = serving.rope(k, pos + 7, f, sec, il)
    s1 = np.sum(y * z, -1)
    s2 = np.sum(serving.rope(x, pos + 100, f, sec, il) * serving.rope(k, pos + 107, f, sec, il), -1)
    assert np.allclose(s1, s2, atol=1e-11)


def test_rope_pairs_and_axes():
    """One pair turned by a quarter: which elements it is, and by which axis."""
    x = np.arange(8.0).reshape(1, 1, 1, 8)
    f = np.full(4, math.pi / 2)
    pos = np.array([[[0]], [[1]]])
    y = serving.rope(x, pos, f, (3, 1))
    assert np.allclose(y[0, 0, 0], [0, 1, 2, -7, 4, 5, 6, 3], atol=1e-14)
    y = serving.rope(x, pos, f, (3, 1), interleaved=True)
    assert np.allclose(y[0, 0, 0], [0, 1, 2, 3, 4, 5, -7, 6], atol=1e-14)


def test_nearest_e4m3_is_nearest():
    """Against every code by brute force, at values, ties, and between them."""
    vals = e4m3_to_f64(np.arange(256))
    pts = np.concatenate([vals[np.isfinite(vals)],
                          [(a + b) / 2 for a, b in zip(vals[:126], vals[1:127])],
                          RNG(5).uniform(-460, 460, 500), RNG(6).uniform(-0.05, 0.05, 500)])
    got = serving.nearest_e4m3(pts)
    fine = np.where(np.isfinite(vals))[0]
    for x, c in zip(pts, got):
        best = np.min(np.abs(vals[fine] - x))
        assert abs(vals[c] - x) == best, (x, c)
        ties = [int(k) for k in fine if abs(vals[k] - x) == best and (k < 128) == (c < 128)]
        assert c in ties and (len(ties) == 1 or c % 2 == 0)
    assert list(serving.nearest_e4m3([np.inf, -np.inf, np.nan, 500.0])) == [0x7E, 0xFE, 0x7F, 0x7E]


def test_row_descale():
    rows = np.array([[0, 0], [448, -1], [449, 0], [-447, 0], [1, 0.5], [np.inf, 3], [np.nan, 3],
                     [np.inf, np.nan], [1e-40, 0], [3e38, 0]])
    s = serving.row_descale(rows)
    assert list(s[:8]) == [1, 1, 2, 1, 2.0 ** -8, 2.0 ** -7, 2.0 ** -7, 1]
    assert s[8] == 2.0 ** -126 and s[9] == 2.0 ** 120
    for r, f in zip(rows[:5], s[:5]):
        assert np.max(np.abs(r)) <= 448 * f


@pytest.mark.parametrize("window", [0, 1, 5, 100])
def test_decode_is_the_last_causal_row(window):
    """Shuffled pages, shared heads: the last row of the attention oracle."""
    rng = RNG(7)
    B, Hkv, g, d, ps, n = 2, 2, 3, 4, 16, [37, 16]
    pages = 9
    K, V = (rng.standard_normal((pages, Hkv, ps, d)) for _ in range(2))
    table = rng.permutation(pages)[:6].reshape(2, 3)
    q = rng.standard_normal((B, Hkv * g, 1, d))
    r = serving.decode(q, K, V, table, n, 0.3, window)
    for b in range(B):
        k = serving.gather(K, table[b], range(n[b]))
        v = serving.gather(V, table[b], range(n[b]))
        for h in range(Hkv * g):
            qq = np.zeros((1, 1, n[b], d))
            qq[0, 0, -1] = q[b, h, 0]
            o, lse = oracle.attention_forward(qq, k[None, h // g:h // g + 1],
                                              v[None, h // g:h // g + 1], True, 0.3,
                                              window=window)
            assert np.allclose(o[0, 0, -1], r["O"][b, h], atol=1e-13)
            assert abs(lse[0, 0, -1] - r["L"][b, h]) < 1e-12


def test_decode_skips_bad_pages_and_empty_sequences():
    rng = RNG(8)
    K, V = (rng.standard_normal((4, 1, 16, 4)) for _ in range(2))
    q = rng.standard_normal((4, 1, 4))
    table = np.array([[0, 1, 2], [0, 7, 2], [-1, 9, 4], [0, 1, 2]])
    r = serving.decode(q, K, V, table, [40, 40, 40, 0], 1.0)
    assert list(r["n"]) == [40, 24, 0, 0]
    assert np.all(r["O"][2:] == 0) and np.all(np.isneginf(r["L"][2:]))
    kept = serving.decode(q[1:2], K, V, np.array([[0, 2, 3]]), [24], 1.0)
    assert np.allclose(kept["O"][0], r["O"][1])
