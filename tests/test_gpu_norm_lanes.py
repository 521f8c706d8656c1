"""Every channel of a row is normalised by one and the same number, whichever lane holds it."""
import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2

pytestmark = pytest.mark.gpu


def row(seed, D, run):
    """A row from a 64-bit linear congruential generator: `run` neighbouring channels share a power of two."""
    state = seed

    def draw():
        nonlocal state
        state = (state * 6364136223846793005 + 1442695040888963407) % 2 ** 64
        return (state >> 40) - 2 ** 23

    draw()
    x = np.empty(D, np.float32)
    for i in range(0, D, run):
        p = 2.0 ** -(23 + ((draw() >> 10) & 3))
        x[i:i + run] = [draw() * p for _ in range(run)]
    return x


# Rows whose mean of squares is so near the middle between two float32 values that it mattered in which order a lane
# added the low words of its partner's sum and its own: found by running the sums of 2^31 such rows on a CPU.
@pytest.mark.parametrize("seed,D,run,at,pad", [
    (6812884, 32, 16, slice(0, None, 16), 0), (83640848, 32, 16, slice(0, None, 16), 0),        # two lanes of a warp
    (1550275000, 32, 16, slice(0, None, 16), 0),
    (23594008, 544, 16, slice(0, None, 16), 0),                                                  # a CTA of two warps
    (82726942, 64, 1, slice(0, 32), 1)])                                                         # unaligned: a warp
def test_lanes_of_a_row_agree(seed, D, run, at, pad):
    x = row(seed, D, run)
    x[at] = 2.0 ** -10                     # one channel of every lane: a power of two, whose product is the number itself
    wide = torch.zeros((3, D + pad), device="cuda")
    wide[:, pad:] = torch.from_numpy(x).cuda()
    y, _ = csa2.rms_norm(wide[:, pad:], out_dtype=torch.float32)
    r = y[:, at].cpu().numpy()
    assert (r == r[0, 0]).all(), np.unique(r)
