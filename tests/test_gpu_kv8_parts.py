"""A step of a prompt's chunk and single rows, attended to by two calls: each takes a range of the sequences (its rows of the
page table, its starts and lengths) and leaves the other's rows alone."""
import dataclasses

import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2
from kv8_utils import DEV, bf16, check_attn, fill, gpu, new_cache, starts, to_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("chunk_at", [0, 2, 4])
def test_calls_over_ranges_of_the_sequences(chunk_at):
    r = np.random.default_rng(chunk_at)
    length, add = [130, 64, 700, 1], [1, 1, 1, 1]
    length.insert(chunk_at, 333)
    add.insert(chunk_at, 90)
    c = new_cache(r, 5, 12, 2, 64)
    fill(r, c, length)
    g, start = to_gpu(c), starts(add, 3)
    T = int(start[-1]) + 4
    q = bf16(r.standard_normal((T, 8, 64)))
    out, lse = torch.full((T, 8, 64), 777.0, device=DEV), torch.full((T, 8), 777.0, device=DEV)
    st, le, qd = gpu(start), gpu(np.array(length, np.int32)), gpu(q, torch.bfloat16)
    csa2.device_error()
    for a, b, new in ((0, chunk_at, 1), (chunk_at, chunk_at + 1, 90), (chunk_at + 1, 5, 1)):
        part = dataclasses.replace(g, page_table=g.page_table[a:b])
        if a < b:
            csa2.kv8_attn(part, qd, st[a:b + 1], le[a:b], max_new=new, out=out, lse=lse)
    assert csa2.device_error() == 0
    assert (out[:3] == 777).all() and (out[start[-1]:] == 777).all() and (lse[:3] == 777).all() and (lse[start[-1]:] == 777).all()
    check_attn(out, lse, c, q, start, length, 64 ** -0.5, out_eps=2.0 ** -24)
