"""Rotary positions as far as fa_rotary takes them, against angles in exact arithmetic.

Tolerance, from the arithmetic: the fraction of a half turn is rounded to float32 (pi 2^-25 <
1.6 2^-24 rad) and nothing before it counts; sincospi is within 4 * 2^-24, its product with
mscale, the products with x and their sum round by 2^-24 each: 9 2^-24 of m (|x1| + |x2|), at
every position.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

from exact_io_aware_64_b200 import binding

pytestmark = pytest.mark.gpu

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097493")


def angles(first, n, freq):
    """[n, len(freq)] float64 in [-pi, pi], reduced in exact arithmetic."""
    out = np.empty((n, len(freq)))
    for k, f in enumerate(freq):
        per = Fraction(float(f)) / TWO_PI
        for i in range(n):
            t = (first + i) * per
            out[i, k] = float((t - round(t)) * TWO_PI)
    return out


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("first", [0, 1 << 24, (1 << 31) - 3, -(1 << 31), 1 << 36, (1 << 40) - 9,
                                   1 << 40, -(1 << 40)])
def test_far_positions(first, interleaved):
    N, d = 9, 64
    x = torch.randn(1, 2, N, d, generator=torch.Generator().manual_seed(1))
    f, _ = binding.rotary_frequencies(d)
    f = torch.cat([f[:-2].cpu(), torch.tensor([3.0, 123.456])]).cuda()  # beyond one radian a token
    ang = angles(first, N, f.cpu().tolist())[None, None]
    a = np.arange(d // 2)
    a, b = (2 * a, 2 * a + 1) if interleaved else (a, a + d // 2)
    X = x.double().numpy()
    for sign, call in ((1.0, binding.rotary), (-1.0, binding.rotary_bwd)):
        got = call(x.cuda(), None, f, first=first, interleaved=interleaved, mscale=1.5)[0]
        got = got.double().cpu().numpy()
        c, s = 1.5 * np.cos(ang), sign * 1.5 * np.sin(ang)
        bound = 9 * 2.0 ** -24 * 1.5 * (np.abs(X[..., a]) + np.abs(X[..., b]))
        for at, want in ((a, X[..., a] * c - X[..., b] * s), (b, X[..., b] * c + X[..., a] * s)):
            over = np.abs(got[..., at] - want) - bound
            assert over.max() <= 0, f"off by {over.max():.3e} more than the bound"
