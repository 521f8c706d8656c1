"""Threads whose calls go to one stream and share its default workspace: every result is that of calls one after the other."""
import threading

import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2
from kv8_utils import bf16, fill, gpu, new_cache, starts, to_gpu

pytestmark = pytest.mark.gpu


def test_threads_on_one_stream():
    r = np.random.default_rng(23)
    sets = []
    for n in (3000, 5000, 700, 9000):
        c = new_cache(r, 1, 150, 2, 64, spare=0)
        fill(r, c, [n])
        q = bf16(r.standard_normal((3, 16, 64)))
        sets.append((to_gpu(c), gpu(q, torch.bfloat16), gpu(starts([3])), gpu(np.array([n], np.int32))))

    def calls(g, q, start, length):
        pages, count = csa2.kv8_select(g, q, start, length, 9)
        return (pages, count, *csa2.kv8_attn(g, q, start, length, max_new=1), *csa2.kv8_attn(g, q, start, length, max_new=3),
                *csa2.kv8_attn(g, q, start, length, pages=pages))

    csa2.device_error()
    alone = [calls(*s) for s in sets]
    torch.cuda.synchronize()
    got = [[] for _ in sets]
    go = threading.Barrier(len(sets))

    def thread(i):
        go.wait()
        for _ in range(50):
            got[i].append(calls(*sets[i]))

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert csa2.device_error() == 0
    for i, want in enumerate(alone):
        assert len(got[i]) == 50
        assert all((a == b).all() for run in got[i] for a, b in zip(run, want))
