"""The attention block that runs the row operators around the hot path: each stage against the
oracle on the stage's own input, eagerly and replayed from a graph."""
import math

import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2, layer
from oracle import attention, formats, rows

pytestmark = pytest.mark.gpu
U, UB = 2.0 ** -24, 2.0 ** -8


def c(t):
    return t.cpu().numpy()


def f64(t):
    return c(t.double())


def fp4(q):
    return c(q.codes), c(q.row_scales())


def check_linear(y, x, w, gx=1.0, gw=1.0):
    ref, mag = rows.fp4_linear(*fp4(x), *fp4(w), gx, gw)
    assert (np.abs(f64(y) - ref) <= (x.cols // 64 + 16) * 4 * U * mag + (2 * U + UB) * np.abs(ref)).all()


def test_layer_stages_against_the_oracle():
    B, n, d_model, Hq, d, W, k = 5, 500, 256, 8, 128, 32, 64
    run, s = layer.build(B, n, d_model, Hq, d, H_i=4, d_ik=64, d_rope=32, W=W, k=k, num_blocks=64, per_block=8, seed=3)
    L = s["layers"][0]
    h, res = c(s["h"].float()), c(s["residual"].float())
    out, topk = L.step(s["h"], s["residual"], s["cache"], s["seq"], s["pos"], s["index"], s["window"])
    assert csa2.device_error() == 0
    # the residual stream and the norm
    r = rows.add(h, res, True)
    assert np.array_equal(c(s["residual"].float()), r)
    y = rows.rms_norm(r, c(L.w_norm.float()), 1e-6)
    assert (np.abs(f64(L.x) - y) <= np.abs(y) * (5 * U + UB) * 1.001).all()
    # FP4 of it, the query projection and its rotation
    codes, scales = rows.fp4_quantize(c(L.x.float()))
    assert np.array_equal(c(L.x4.codes), codes) and np.array_equal(c(L.x4.row_scales()), scales)
    q = csa2.fp4_linear(L.x4, L.w_q)
    check_linear(q, L.x4, L.w_q, 1.0, float(L.w_q.gscale))
    pos, cos, sin = c(s["pos"]), c(L.cos), c(L.sin)
    turned = rows.rope(f64(q).reshape(B, Hq, d), pos, cos, sin, True, False, d - 32)
    assert np.abs(f64(L.q) - turned).max() <= 2 * UB * np.abs(turned).max()
    check_linear(L.q_idx.view(B, -1), L.x4, L.w_iq, 1.0, float(L.w_iq.gscale))
    # attention over the entries the call selected, turned back
    cache, w = s["cache"], s["window"]
    pt, tk, tl = c(cache.page_table), c(topk[0]), c(topk[1])
    for b in range(B):
        e = tk[b, :tl[b]]
        assert tl[b] == k and (np.diff(e) > 0).all()
        pages = pt[b, np.arange(n) // 64], np.arange(n) % 64
        o, _ = attention.sparse_attention(f64(L.q)[b], c(cache.codes)[pages], c(cache.scales)[pages], e, c(w["swa"]),
                                          c(w["swa_scale"]), b * W, W, 1 / math.sqrt(d))
        back = rows.rope(o[None], pos[b:b + 1], cos, sin, True, True, d - 32)[0]
        got = f64(L.a)[b]
        assert np.linalg.norm(got - back) <= (2e-3 + 2 * UB) * np.linalg.norm(back)
    # FP4 of the attention output and the way back
    codes, scales = rows.fp4_quantize(c(L.a.float()).reshape(B, -1), float(L.a4.gscale))
    assert np.array_equal(c(L.a4.codes), codes) and np.array_equal(c(L.a4.row_scales()), scales)
    check_linear(out, L.a4, L.w_o, float(L.a4.gscale), float(L.w_o.gscale))


def test_layer_replays_from_a_graph():
    run, s = layer.build(3, 300, 256, 8, 128, H_i=4, d_ik=64, d_rope=32, W=32, k=64, num_blocks=64, per_block=8, seed=4)
    start = s["residual"].clone()
    first = run().clone()
    s["residual"].copy_(start)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = run()
    for _ in range(2):
        s["residual"].copy_(start)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    assert csa2.device_error() == 0
