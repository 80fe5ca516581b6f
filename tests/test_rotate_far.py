"""Angles of large frequencies at far positions: whole turns drop exactly there, too."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import step as oracle
from tests.test_rotate import f64, i32, normal

gpu = pytest.mark.gpu
U = 2.0 ** -8
PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679, 10 ** 100)
FREQS = [1.0, 3.25, 1000.0, 65537.0, 1234567.0, -7.7e9, 1.1e15, 3.3e38]
POSITIONS = [0, 1, -1, 4097, 123456789, 2 ** 31 - 1, -2 ** 31]


@pytest.fixture(scope="module")
def jg():
    from jagged_gdpa_gb300 import build as b
    b.build()
    import jagged_gdpa_gb300 as m
    return m


def angles():
    """pos * f less its whole turns, by rational arithmetic."""
    f = [Fraction(float(np.float32(x))) for x in FREQS]
    return np.array([[float((p * x / (2 * PI)) % 1 * 2 * PI) for x in f] for p in POSITIONS])


def test_rational_angles():
    t = angles()
    assert np.allclose(np.cos(t[:4, :4]), np.cos(np.outer(POSITIONS[:4], np.float32(FREQS[:4]).astype(float))), atol=1e-8)


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_large_frequencies(jg, interleaved):
    rng = np.random.default_rng(0)
    rows = len(POSITIONS)
    q, freq = normal(rng, rows, 3, 32), torch.tensor(FREQS, device="cuda")
    got, _ = jg.jgdpa_norm_rotate(q, None, None, None, freq, eps=None, interleaved=interleaved, q_positions=i32(POSITIONS))
    x, t = f64(q), angles()[:, None]
    a, b = oracle.pair_columns(len(FREQS), interleaved)
    want, size = x.copy(), np.abs(x)
    want[..., a], want[..., b] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t), x[..., b] * np.cos(t) + x[..., a] * np.sin(t)
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    # of each of the pair 2^-19.3 from the angle (2^-22 of a turn) and 2^-20.9 from the hardware's sine and cosine
    bad = ~(np.abs(f64(got) - want) <= U * np.abs(want) + 2.0 ** -18 * size)
    assert not bad.any(), f"{bad.sum()} of {bad.size}"
