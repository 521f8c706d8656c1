"""Rotary tables with a magnitude: rounded once, like the table without one."""
import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("magnitude", [1.0, 1.3689, 0.1 * np.log(16) + 1, 0.7, 3.0])
@pytest.mark.parametrize("P,d_rope", [(65536, 64), (40000, 6)])
def test_rope_table_rounds_once(P, d_rope, magnitude):
    tables = csa2.rope_table(P, d_rope, magnitude=float(magnitude), device="cuda")
    a = np.arange(P)[:, None] * 10000.0 ** (-2.0 * np.arange(d_rope // 2) / d_rope)[None]
    ours = rounding = 0.0
    for t, want in zip(tables, (magnitude * np.cos(a), magnitude * np.sin(a))):
        err = t.cpu().numpy().astype(np.float64) - want
        # a far angle itself is rounded in float64: 2^-53 of up to P
        assert np.abs(err).max() <= 2 * U * magnitude + P * 2.0 ** -50
        ours += np.mean(err ** 2)
        rounding += np.mean((want.astype(np.float32) - want) ** 2)
    # Before the last rounding, at most 0.31, 0.19 and 0.25 half steps below 1 (the square of the angle, the series, its
    # product) and 0.25 (the magnitude's), at the largest angle and half of them on average: as independent uniform
    # errors a root mean square of 0.15 half steps, beside 0.42 of the rounding itself: 6 % more.  Twice that is allowed
    # for, and a little; rounding twice costs 28 % or more for each of these magnitudes but 1.
    assert np.sqrt(ours) <= 1.15 * np.sqrt(rounding)


def test_rope_table_of_a_vanishing_magnitude():
    """A magnitude below float32's least value gives zeros, not NaN."""
    for t in csa2.rope_table(300, 64, magnitude=1e-50):
        assert (t == 0).all()
