"""The oracle of 4-bit rows, pinned on the CPU: closed cases, brute force over
all codes, and the properties that the cache's format promises."""

import numpy as np
import pytest
import torch

from attention_backward_pass_attn_gb300.inputs import make_tensor
from oracle import int4


def bf16(x):
    return torch.tensor(x, dtype=torch.float64).to(torch.bfloat16).double().numpy()


def test_closed_cases():
    assert int4.factor(np.zeros(32)) == 1.0
    assert int4.factor([7.0] + [0.0] * 31) == 1.0
    assert int4.factor([-14.0] + [3.0] * 31) == 2.0
    assert int4.factor([1.0] + [0.0] * 31) == 18 / 128       # 1/7 = 18.29 / 128
    assert int4.factor([2.0 ** -125] * 32) == 2.0 ** -120
    assert np.isnan(int4.factor([1.0, float("nan")] + [0.0] * 30))
    assert int4.factor([float("inf"), 7.0] + [0.0] * 30) == 1.0
    # ties of the factor: 7 x 16.5 and 7 x 17.5 sixteenths, to the even one
    assert int4.factor([115.5]) == 16.0 and int4.factor([122.5]) == 18.0
    c, f = int4.quantise(np.array([7.0, 0.5, 1.5, 2.5, -0.5, -1.5, float("inf"), -float("inf")]
                                  + [0.0] * 24))
    assert f.tolist() == [1.0] and c[:8].tolist() == [7, 0, 2, 2, 0, -2, 7, -7]


@pytest.mark.parametrize("std", [1e-30, 0.01, 1.0, 300.0, 1e30])
def test_codes_are_the_nearest(std):
    x = make_tensor((6, 64), 5, std=std).double().numpy()
    c, f = int4.quantise(x)
    scale = np.repeat(f, 32, axis=-1)
    every = np.arange(-7, 8)
    best = np.min(np.abs(x[..., None] - every * scale[..., None]), axis=-1)
    assert np.all(np.abs(x - c * scale) == best)
    # the largest value of a group is not clamped, and factors have five bits
    assert np.all(np.max(np.abs(x.reshape(-1, 32)), axis=-1) < 7.5 * f.reshape(-1))
    m, _ = np.frexp(f)
    assert np.all(m * 32 == np.round(m * 32))


def test_values_are_bf16_numbers():
    x = make_tensor((16, 128), 6).double().numpy()
    c, f = int4.quantise(x)
    y = int4.values(int4.pack(c), f)
    assert np.array_equal(bf16(y), y) and np.array_equal(int4.unpack(int4.pack(c)), c)
    assert np.all(np.abs(y - x) <= np.repeat(f, 32, axis=-1) / 2)


def test_the_largest_bf16_numbers_fit():
    top = float(torch.finfo(torch.bfloat16).max)
    c, f = int4.quantise(np.array([top] * 32))
    assert np.isfinite(bf16(7 * f)).all() and np.all(c == 7)
