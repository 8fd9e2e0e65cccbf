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
