"""The angle of lora_rope at far positions, against turns reduced exactly (rational numbers, 1 /
2 pi to 60 digits): up to 2^31 turns of a pair the reduced angle is the exact one rounded to
fp32, so the tolerance of test_gpu_rope.py holds without a term that grows with the position:
|error| <= (|a| + |b|) 9 * 2^-24.  (The fp64 steps before it leave 2^-53 of a turn, 2^-50
radian, far inside the rounding of the last of those nine.)"""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import adapter_gemv_sgmv_b200 as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


def _turns(pos, f):
    """pos * f / (2 pi) less its nearest whole number, exact up to PI's digits, rounded once."""
    u = Fraction(int(pos)) * Fraction(float(f)) / (2 * PI)
    return float(u - round(u))


def _check(pos, freqs, interleaved=False, inverse=False):
    n, half = len(pos), len(freqs)
    g = torch.Generator(device=DEV).manual_seed(n + half)
    x = torch.randn(n, 2, 2 * half, generator=g, device=DEV)
    x[:, 0, half:] = 0
    y = torch.empty_like(x)
    L.lora_rope([x], [y], torch.tensor(pos, dtype=torch.int64, device=DEV),
                torch.tensor(freqs, dtype=torch.float64, device=DEV), interleaved=interleaved, inverse=inverse)
    turn = torch.tensor([[_turns(p, f) for f in freqs] for p in pos], dtype=torch.float64, device=DEV)[:, None]
    c, s = torch.cos(2 * math.pi * turn), torch.sin(2 * math.pi * turn) * (-1 if inverse else 1)
    pairs = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, half), slice(half, None))
    a, b = (x[..., p].double() for p in pairs)
    tol = (a.abs() + b.abs()) * 9 * 2.0 ** -24
    for p, want in zip(pairs, (a * c - b * s, b * c + a * s)):
        over = (y[..., p].double() - want).abs() - tol
        i = int(over.flatten().argmax())
        n_i, rest = divmod(i, 2 * half)
        assert float(over.max()) <= 0, f"position {pos[n_i]}, frequency {freqs[rest % half]}: {float(over.max())} past it"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_angles_up_to_two_to_the_31_turns(interleaved, inverse):
    rng = np.random.default_rng(1)
    freqs = np.r_[1.0, 6.283185307179586, 6.0, rng.uniform(0.5, 6.28, 13)]
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 1999999973, -1234567891, *map(int, rng.integers(2 ** 28, 2 ** 31, 24))]
    _check(pos, freqs, interleaved, inverse)


def test_angles_of_slow_pairs_at_positions_up_to_two_to_the_53():
    rng = np.random.default_rng(2)
    freqs = np.r_[2.0 ** -20, 1e-6, rng.uniform(2.0 ** -21, 2.0 ** -20, 6)]
    pos = [2 ** 53, -2 ** 53, 2 ** 53 - 1, 2 ** 52 + 1, *map(int, rng.integers(2 ** 50, 2 ** 53, 12))]
    _check(pos, freqs)


@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", dict(factor=4.0)),
                                        ("bands", dict(base=500000.0, factor=8.0, low=1.0, high=4.0, original=8192))])
def test_angles_of_usual_frequencies_at_far_positions(scaling, kw):
    f, _ = L.lora_rope_freqs(64, scaling=scaling, **kw)
    rng = np.random.default_rng(3)
    _check([*map(int, rng.integers(2 ** 20, 2 ** 33, 30))], f.numpy())
