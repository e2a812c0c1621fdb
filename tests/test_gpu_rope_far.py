"""Angles of far positions and of any frequencies, against exact rational
arithmetic: what the rotation may be off by does not grow with the position.

Tolerance: as in test_gpu_rope for fp32 (4e-7 in all, 6e-7 allowed, of |x| + |y|,
then half a step), to which 2^-32 of a turn adds 1.5e-9.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

from broadcast_gemm_attention_gb300 import binding as B

pytestmark = pytest.mark.gpu

# pi to 60 decimals
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)

POSITIONS = [0, 1, -1, 999_983, 16_777_217, 2 ** 31 - 2, -2 ** 31]


def turn(f: float, pos: int) -> float:
    """pos f / 2 pi less whole turns, in radians."""
    t = Fraction(f) * pos / (2 * PI)
    return float((t - round(t)) * 2 * PI)


@pytest.mark.parametrize("freqs", [[1.0, 0.5, 1e-4, 3.1e-9], [1000.123, 3.0, 77777.77, 6.283185307179586],
                                   [-1.0, -1e-7, -3e-11, -2500.5], [1e9 + 0.3, -1.1e12, 2.0 ** 40, 4e10 / 7]])
@pytest.mark.parametrize("backward", [False, True])
def test_angles_are_exact_at_any_position(freqs, backward):
    half, L = len(freqs), 2
    n = len(POSITIONS)
    x = torch.randn(n, 2, L, 2 * half, generator=torch.Generator().manual_seed(1))
    start = torch.tensor(POSITIONS, dtype=torch.int32).cuda()
    y = torch.empty_like(x).cuda()
    with B.Plan(64, 64, 4) as p:
        call = p.rope_backward if backward else p.rope_forward
        call(B.Rope(2 * half, freqs), x.cuda(), y, start=start)
        assert p.status() == B.IKBO_OK
    angle = np.array([[[turn(f, pos + l) for f in freqs] for l in range(L)] for pos in POSITIONS])[:, None]
    c, s = np.cos(angle), np.sin(angle) * (-1 if backward else 1)
    xd = x.double().numpy()
    a, b = xd[..., :half], xd[..., half:]
    ref = np.concatenate([a * c - b * s, b * c + a * s], -1)
    size = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= (6e-7 + 1.5e-9) * size + 2.0 ** -24 * np.abs(ref)), float((err / size).max())
