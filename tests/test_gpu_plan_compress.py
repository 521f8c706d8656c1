"""A step's plan feeds the CSA2 layers: page_plan, then the compressor and the Full indexer on its tables, in one graph that
advances its own state, against the same calls on tables that the host made."""
import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2
from oracle import kv8

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("adds", [[(70, 1, 128, 5), (60, 73, 64, 7), (204, 0, 0, 0)], [(1, 1, 1, 1)] * 3])
def test_plan_compress_index(adds):
    S, d, d_ik, H_i, NB, P, k = 4, 128, 64, 8, 8, 8, 32
    most, T = 6, sum(adds[0])
    r = np.random.default_rng(T)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)
    free = r.permutation(S * most).astype(np.int32)
    table, length, head = np.full((S, most), -1, np.int32), np.zeros(S, np.int64), 0
    caches = [csa2.PagedCache.allocate(S, most * 64, d, d_ik, DEV, page_table=torch.arange(S * most, dtype=torch.int32).reshape(S, most)) for _ in range(2)]
    ws = csa2.Workspace(DEV)
    W = torch.randn((d, d_ik), device=DEV).bfloat16()
    C, q, w = torch.zeros((T, d), device=DEV), torch.randn((S, H_i, d_ik), device=DEV).bfloat16(), torch.rand((S, H_i), device=DEV)
    seqs = i32(range(S))
    state = dict(length=i32(length), add=i32(adds[0]), free=i32(free), head=i32([0]))
    plan = csa2.PagePlan.allocate(S, T, DEV)
    plan.length, plan.head = state["length"], state["head"]
    caches[0].page_table.fill_(-1)
    outs = [(torch.full((S, NB * P), -1, dtype=torch.int32, device=DEV), torch.zeros(S, dtype=torch.int32, device=DEV),
             torch.full((S, k), -1, dtype=torch.int32, device=DEV), torch.zeros(S, dtype=torch.int32, device=DEV)) for _ in range(2)]

    def layers(cache, seq, entry, n_vis, out):
        csa2.compress_quant(cache, seq, entry, C=C, W_ik=W, ws=ws)
        csa2.index_full(cache, q, w, seqs, n_vis, most * 64, NB, P, k, out=out, ws=ws)

    def step():
        p = csa2.page_plan(state["length"], state["add"], caches[0].page_table, state["free"], state["head"], T, out=plan)
        layers(caches[0], p.seq, p.pos, p.length, outs[0])

    caches[1].page_table.copy_(caches[0].page_table)
    layers(caches[1], i32(np.zeros(T)), i32(np.arange(T) % 64), i32(np.zeros(S)), outs[1])     # sizes the workspace
    csa2.device_error()
    for t in (caches[1].codes, caches[1].scales, caches[1].idx_k):
        t.zero_()
    state["add"].zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for add in adds:
        C.copy_(torch.randn((T, d), device=DEV))
        state["add"].copy_(i32(add))
        graph.replay()
        want = kv8.plan(length, add, table, free, head, T)
        length, head = want["length"], want["head"]
        assert (want["seq"] >= 0).all()                      # no padding
        caches[1].page_table.copy_(i32(table))
        torch.cuda.synchronize()
        layers(caches[1], i32(want["seq"]), i32(want["pos"]), i32(length), outs[1])
        for a, b in zip((caches[0].codes, caches[0].scales, caches[0].idx_k, *outs[0]), (caches[1].codes, caches[1].scales, caches[1].idx_k, *outs[1])):
            assert (a == b).all()
    assert csa2.device_error() == 0
    state["add"].copy_(i32([0, 0, 0, 1]))                    # the other rows are padding: skipped, and reported
    before = caches[0].codes.clone()
    graph.replay()
    page = int(caches[0].page_table[3, int(length[3]) // 64])
    assert csa2.device_error() == 0x10
    before[page, int(length[3]) % 64] = caches[0].codes[page, int(length[3]) % 64]
    assert (caches[0].codes == before).all()
