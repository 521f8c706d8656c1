"""Attention of 17 to 128 rows a sequence and key head over cold pages: two groups share the steps of a stream, and what each
multiplies does not depend on the order in which the copies land."""
import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2
from kv8_utils import DEV, bf16, check_attn, fill, gpu, new_cache, starts, to_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [3, 6, 8, 13, 16])           # 24 to 128 rows
def test_cold_calls_repeat_bit_for_bit(new, D):
    """Streams of 2 to 40 steps, short and long segments; L2 is written over before every call."""
    r = np.random.default_rng(new * D)
    length = [128 * n - 5 for n in (2, 3, 4, 5, 7, 11, 40)]
    c = new_cache(r, len(length), 80, 2, D)
    fill(r, c, length)
    g = to_gpu(c)
    add = [new] * len(length)
    q = bf16(r.standard_normal((sum(add), 16, D)))
    args = (g, gpu(q, torch.bfloat16), gpu(starts(add)), gpu(np.array(length, np.int32)))
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    csa2.device_error()
    first = None
    for i in range(30):
        flush.fill_(i)
        got = csa2.kv8_attn(*args, max_new=new, out_dtype=torch.float32)
        first = first or got
        assert all((a == b).all() for a, b in zip(got, first)), i
    assert csa2.device_error() == 0
    check_attn(*first, c, q, starts(add), length, D ** -0.5, out_eps=2.0 ** -24)
