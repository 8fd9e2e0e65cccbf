"""NaN and infinities at visible positions of attn_decode's cache, and in its
queries, wherever a sequence is split: one unit of work, a few parts that one
block joins, and more than 32 parts, joined in two steps.

A NaN among a head's visible scores makes that head's O and L NaN; one in a
row of V makes the outputs of its column NaN and leaves L alone.  Heads and
sequences that do not use the value keep their bits.
"""

import numpy as np
import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from attention_backward_pass_attn_gb300.inputs import make_tensor
from oracle import serving
from serving_cases import filled_cache
from test_gpu_decode import cuda_ready, f64, run  # noqa: F401

pytestmark = pytest.mark.gpu

# positions at d = 64: a unit is 128 keys in bf16 and 256 in e4m3, so these are
# one unit; two or four; 71 or 36 (a block each, joined in two steps)
LENGTHS = [50, 500, 9000]
PAGE, HKV, GROUP, D = 32, 2, 2, 64


def case(n, fp8, seed=3):
    lens = [n, 40]
    c = filled_cache(lens, PAGE, HKV, D, seed, fp8)
    return lens, c, make_tensor((2, HKV * GROUP, 1, D), seed + 9)


def at(c, p, h=0, b=0):
    return int(c["table"][b, p // PAGE]), h, p % PAGE


def nan_key(c, p, fp8):
    if fp8:
        c["kc"].view(torch.uint8)[at(c, p)][5] = 0x7F
    else:
        c["kc"][at(c, p)][5] = float("nan")


def expect_nan(got, good, heads):
    o, lse = got
    rest = [h for h in range(HKV * GROUP) if h not in heads]
    assert torch.isnan(o[0, heads]).all() and torch.isnan(lse[0, heads]).all()
    for x, y in zip(got, good):
        assert torch.equal(x[0, rest], y[0, rest]) and torch.equal(x[1], y[1])
    assert torch.isfinite(good[0]).all() and torch.isfinite(good[1]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", LENGTHS)
def test_nan_in_a_query(n, fp8):
    lens, c, q = case(n, fp8)
    good = run(q, c, lens)
    q[0, 3, 0, 7] = float("nan")
    expect_nan(run(q, c, lens), good, [3])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("where", ["first", "middle", "last", "part", "all"])
def test_nan_in_keys(n, fp8, where):
    """One row, every row of one unit (a part of its own where the sequence is
    split), every row."""
    lens, c, q = case(n, fp8)
    good = run(q, c, lens)
    unit = min(n, 256)
    rows = {"first": [0], "middle": [n // 2], "last": [n - 1],
            "part": range((n // 2) // unit * unit, min(n, (n // 2) // unit * unit + unit)),
            "all": range(n)}[where]
    for p in rows:
        nan_key(c, p, fp8)
    expect_nan(run(q, c, lens), good, [0, 1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", LENGTHS[1:])
def test_nan_in_a_part_of_no_weight(n, fp8):
    """The NaN's part lies hundreds of e-folds below the others' scores, so that
    its weight is zero in 32 bits."""
    lens, c, q = case(n, fp8)
    unit = 256
    part = range((n // 2) // unit * unit, min(n, (n // 2) // unit * unit + unit))
    away = torch.from_numpy(-16 * np.sign(f64(q)[0, 0, 0]))
    q[0, 1] = q[0, 0]
    for p in part:
        if fp8:
            c["kc"].view(torch.float8_e4m3fn)[at(c, p)] = away.to(torch.float8_e4m3fn)
            c["kd"][at(c, p)] = 4.0
        else:
            c["kc"][at(c, p)] = 4 * away.to(torch.bfloat16)
    good = run(q, c, lens)
    nan_key(c, part[3], fp8)
    expect_nan(run(q, c, lens), good, [0, 1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
def test_nan_and_infinity_in_values(n, fp8, value):
    """In one element of V (in its factor, with e4m3, which has no infinity):
    the outputs that use it are not finite, everything else keeps its bits."""
    lens, c, q = case(n, fp8)
    good = run(q, c, lens)
    p = n // 2
    if fp8 and value != "nan":
        c["vd"][at(c, p)] = float(value)
        columns = torch.arange(D)
    elif fp8:
        c["vc"].view(torch.uint8)[at(c, p)][5] = 0xFF
        columns = torch.tensor([5])
    else:
        c["vc"][at(c, p)][5] = float(value)
        columns = torch.tensor([5])
    o, lse = run(q, c, lens)
    used = torch.zeros(D, dtype=torch.bool)
    used[columns] = True
    assert not torch.isfinite(o[0, :2, 0, used]).any()
    if value == "nan":
        assert torch.isnan(o[0, :2, 0, used]).all()
    assert torch.equal(o[0, :2, 0, ~used], good[0][0, :2, 0, ~used])
    assert torch.equal(o[0, 2:], good[0][0, 2:]) and torch.equal(o[1], good[0][1])
    assert torch.equal(lse, good[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", LENGTHS)
def test_infinite_scores(n, fp8):
    """Of a key that scores +inf for one head and -inf for another: NaN, and
    the answer without that key."""
    lens, c, q = case(n, fp8)
    q[0, 0, 0, 5], q[0, 1, 0, 5] = 0.5, -0.5
    p = n // 2
    if fp8:  # an infinite factor: a score of +-inf by the sign of the product
        k = torch.zeros(D)
        k[5] = 1.0
        c["kc"].view(torch.float8_e4m3fn)[at(c, p)] = k.to(torch.float8_e4m3fn)
        c["kd"][at(c, p)] = float("inf")
    else:
        c["kc"][at(c, p)][5] = float("inf")
    o, lse = run(q, c, lens)
    assert torch.isnan(o[0, 0]).all() and torch.isnan(lse[0, 0]).all()
    assert torch.isfinite(o[0, 1:]).all() and torch.isfinite(o[1]).all()
    # without the key: the oracle on two pieces, joined
    k64, v64 = serving.cache_values(c["kc"], c["kd"]), serving.cache_values(c["vc"], c["vd"])
    rows = [x for x in range(n) if x != p]
    k, v = (serving.gather(t, c["table"][0].numpy(), rows)[0] for t in (k64, v64))
    s = (k @ f64(q)[0, 1, 0]) / 8
    w = np.exp(s - s.max())
    ref, A = w @ v / w.sum(), w @ np.abs(v) / w.sum()
    L = s.max() + np.log(w.sum())
    e = ((D + 8) * 2.0 ** -23 + 2.0 ** -22) * np.max(np.abs(k) @ np.abs(f64(q)[0, 1, 0])) / 8
    chain = 64 + n // 16  # a thread's sums, at most
    assert abs(f64(lse)[0, 1, 0] - L) <= e + chain * 2.0 ** -24 + 2.0 ** -22 * (1 + abs(L))
    assert np.all(np.abs(f64(o)[0, 1, 0] - ref) <= np.abs(ref) * 2.0 ** -8
                  + (2 * e + chain * 2.0 ** -22 + 2.0 ** -16) * A * (1 + 2.0 ** -8))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", LENGTHS)
def test_all_scores_minus_infinity(n, fp8):
    """Weight 0 throughout: O = 0 and L = -inf, as if there were nothing to see."""
    lens, c, q = case(n, fp8)
    good = run(q, c, lens)
    q[0, :2, 0, 5] = -0.5
    for p in range(n):
        if fp8:
            k = torch.zeros(D)
            k[5] = 1.0
            c["kc"].view(torch.float8_e4m3fn)[at(c, p)] = k.to(torch.float8_e4m3fn)
            c["kd"][at(c, p)] = float("inf")
        else:
            c["kc"][at(c, p)][5] = float("inf")
    o, lse = run(q, c, lens)
    assert torch.all(o[0, :2] == 0) and torch.isneginf(lse[0, :2]).all()
    assert torch.equal(o[0, 2:], good[0][0, 2:]) and torch.equal(o[1], good[0][1])
