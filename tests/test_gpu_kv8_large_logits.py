"""Attention over the paged 8-bit cache where logits are so large that a unit of their float32 is a factor of the weights: the token
that leads by far gets all of the weight, whatever the size."""
import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2
from kv8_utils import DEV, bf16, gpu, new_cache, starts, to_gpu
from oracle import kv8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hint", [1, 3, 8, 20, 100])         # streams of 8 and 16 rows, tiles of 64, 128 and 256
@pytest.mark.parametrize("size", [4, 12, 18, 20, 21, 22, 23, 24, 25, 27, 30, 36, 50, 90])
def test_a_leading_token_takes_it_all(size, hint):
    """q . k of the leading token is about 2^size, at its place early, in the middle or late; the others' is below 0.7 of it.  Above
    16 rows a row whose largest logit, in base 2, reaches 2^28 is NaN."""
    r = np.random.default_rng(size)
    H, G, D, n = 2, 4, 64, 64 * 11 - 3
    c = new_cache(r, 3, 11, H, D)
    u = np.where(r.random(D) < 0.5, -1.0, 1.0)
    lead = [5, 300, 690]
    k = bf16(r.standard_normal((3 * n, H, D)))
    for s in range(3):
        k[s * n + lead[s]] = bf16(8 * u)
        k[s * n + lead[s] + 1] = bf16(4 * u)                 # a second one, half as large
        k[s * n + lead[s] - 2] = bf16(4.5 * u)
    v = bf16(r.standard_normal((3 * n, H, D)))
    kv8.append(c, k, v, starts([n] * 3), np.full(3, n, np.int32))
    g = to_gpu(c)
    # rows of the last tokens: all see the leading one
    q = bf16(2.0 ** size / (8 * D) * u * r.uniform(0.7, 1.3, (9, H * G, D)))
    csa2.device_error()
    out, lse = csa2.kv8_attn(g, gpu(q, torch.bfloat16), gpu(starts([3] * 3)), gpu(np.full(3, n, np.int32)), max_new=hint, softmax_scale=1.0,
                             out_dtype=torch.float32)
    assert csa2.device_error() == 0
    out, lse = out.cpu().numpy(), lse.cpu().numpy()
    if hint * G > 16 and size > 28:
        assert np.isnan(out).all() and np.isnan(lse).all()
        return
    for t in range(9):
        s = t // 3
        for h in range(H * G):
            rows = [kv8.rows(c, x, s, range(11), h // G)[:n - 2 + t % 3] for x in "kv"]
            want, l, _ = kv8.attend(q[t, h].astype(np.float64), *rows, np.ones(n - 2 + t % 3, bool), 1.0)
            x = rows[0] @ q[t, h].astype(np.float64)
            assert x.argmax() == lead[s] and np.sort(x)[-2] < 0.7 * x.max()
            if size >= 12:                                   # the others' weights are below 2^-900
                assert (np.abs(out[t, h] - rows[1][lead[s]]) <= 2.0 ** -10 * np.abs(rows[1][lead[s]])).all(), (t, h, out[t, h][:4], want[:4])
            # the logit's own rounding
            assert abs(lse[t, h] - l) <= (D + 8) * 2.0 ** -24 * (np.abs(rows[0]) @ np.abs(q[t, h])).max() + 2.0 ** -13, (lse[t, h], l)
