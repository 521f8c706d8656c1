"""Planes of more than 2^32 bytes: pages at both sides of every multiple of 2^31, appended to, selected and attended to."""
import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2
from kv8_utils import DEV, bf16, check_attn, gpu, new_cache, starts
from oracle import kv8

pytestmark = pytest.mark.gpu


def test_planes_beyond_unsigned_32_bit_offsets():
    r = np.random.default_rng(24)
    H, D, n = 2, 128, 12 * 64 - 5
    page = H * 64 * D
    P = (1 << 32) // page + 8000
    c = new_cache(r, 1, 12, H, D, spare=0)
    # where the step's 12 pages lie: at the borders of 2^31 and 2^32 bytes, and the last ones
    at = np.array([0, 1] + [b // page + i for b in (1 << 31, 1 << 32) for i in (-1, 0, 1)] + [P - 4, P - 3, P - 2, P - 1])
    assert len(set(at)) == 12 and (P - 1) * page > 1 << 32
    where = r.permutation(12)
    new = lambda dtype, *s: torch.empty((P, H) + s, dtype=dtype, device=DEV)
    table = gpu(at[where].astype(np.int32)[None])
    g = csa2.Kv8Cache(new(torch.uint8, 64, D), new(torch.uint8, 64, D), new(torch.float32), new(torch.float32), table, new(torch.int8, D),
                      new(torch.float32))
    # what an offset cut to 32 bits would reach instead
    for t in (g.k, g.v):
        t.fill_(0x7F)
    x = [bf16(r.standard_normal((n, H, D))) for _ in range(2)]
    kv8.append(c, x[0], x[1], starts([n]), [n])
    csa2.device_error()
    csa2.kv8_append(g, gpu(x[0], torch.bfloat16), gpu(x[1], torch.bfloat16), gpu(starts([n])), gpu(np.array([n], np.int32)))
    for f in ("k", "v", "k_scale", "v_scale", "mean", "mean_scale"):
        full = slice(0, 11 if f.startswith("mean") else 12)
        got, want = getattr(g, f)[table[0, full].long()].cpu().numpy(), c[f][c["table"][0, full]]
        assert (got.view(np.uint8) == want.view(np.uint8)).all(), f
    others = torch.ones(P, dtype=torch.bool, device=DEV)
    others[table[0].long()] = False
    for t in (g.k, g.v):
        assert all(bool((t[a:a + 4096][others[a:a + 4096]] == 0x7F).all()) for a in range(0, P, 4096))
    q = bf16(r.standard_normal((2, 8, D)))
    args = (g, gpu(q, torch.bfloat16), gpu(starts([2])), gpu(np.array([n], np.int32)))
    pages, _ = csa2.kv8_select(*args, 5)
    lists = [kv8.select(c, q[t], 0, n - 1 + t, 5, 1, 1) for t in range(2)]
    assert pages.cpu().tolist() == lists
    out, lse = csa2.kv8_attn(*args, pages=pages)
    check_attn(out, lse, c, q, starts([2]), [n], D ** -0.5, pages=lists)
    for hint in (1, 4, 8, 20, 100):                          # streams of 8 and 16 rows, tiles of 64, 128 and 256
        out, lse = csa2.kv8_attn(*args, max_new=hint)
        check_attn(out, lse, c, q, starts([2]), [n], D ** -0.5)
    assert csa2.device_error() == 0
