"""The attention block's appended entry, its selection and its Reuse layer against the oracle, each stage on the stage's
own input."""
import math

import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2, layer
from oracle import attention, compress, formats, indexer, rows
from parity_utils import (bf16_host_bits, check_index_k, check_index_set, fp4_mismatch_is_tolerated, paged_to_logical,
                          projection_error_bound)

pytestmark = pytest.mark.gpu
U, UB = 2.0 ** -24, 2.0 ** -8
B, N, D_MODEL, HQ, D, D_ROPE, W, K, NB, PER = 5, 500, 256, 8, 128, 32, 32, 64, 16, 8


def c(t):
    return t.cpu().numpy()


def f64(t):
    return c(t.double())


def fp4(q):
    return c(q.codes), c(q.row_scales())


@pytest.fixture(scope="module")
def stepped():
    """A Full layer's step and the Reuse layer's after it, with copies of what each step started from."""
    _, s = layer.build(B, N, D_MODEL, HQ, D, H_i=4, d_ik=64, d_rope=D_ROPE, W=W, k=K, num_blocks=NB, per_block=PER, seed=5)
    cache = s["cache"]
    before = {n: getattr(cache, n).clone() for n in ("codes", "scales", "idx_k")}
    starts, ends, topk, h = [], [], None, s["h"]
    for L in s["layers"]:
        starts.append((c(h.float()), c(s["residual"].float())))
        h, topk = L.step(h, s["residual"], cache, s["seq"], s["pos"], s["index"], s["window"], topk)
        ends.append((c(s["residual"].float()), h.clone(), [t.clone() for t in topk]))
    assert csa2.device_error() == 0
    return s, before, starts, ends


def test_the_new_tokens_entries(stepped):
    s, before, _, _ = stepped
    L, cache = s["layers"][0], s["cache"]
    H, w_kv, w_ik = f64(L.x), f64(L.w_kv), f64(L.w_ik)
    pos, pt = c(s["pos"]), c(cache.page_table)
    want = compress.compress_quant_from_hidden(H, w_kv, None, 1, pos, c(L.cos), c(L.sin), D_ROPE, w_ik)
    page, slot = pt[np.arange(B), pos // 64], pos % 64
    codes, scales, ik = c(cache.codes)[page, slot], c(cache.scales)[page, slot], bf16_host_bits(cache.idx_k)[page, slot]
    err = projection_error_bound(H, w_kv, None, 1, D_ROPE, None, None)
    bad, tolerated = fp4_mismatch_is_tolerated(want["y"], codes, scales, want["codes"], want["scales"], err)
    assert bad == tolerated
    same = (codes == want["codes"]).all(1) & (scales == want["scales"]).all(1)
    assert same.any()
    check_index_k(ik[same], want["idx_k"][same], want["codes"][same], want["scales"][same],
                  bf16_host_bits(L.w_ik))
    # and nothing else of the cache has changed
    for name, old in before.items():
        new = getattr(cache, name).clone()
        at = torch.from_numpy(page).cuda().long(), torch.from_numpy(slot).cuda().long()
        new[at] = old[at]
        assert torch.equal(new.view(torch.uint8), old.view(torch.uint8)), name


def test_the_selection(stepped):
    s, _, _, ends = stepped
    L, cache = s["layers"][0], s["cache"]
    pool, pool_len, topk, topk_len = (c(t) for t in s["index"]["out"])
    q, w, pt, ik = f64(L.q_idx), f64(L.head_weights), c(cache.page_table), formats.bf16_value(bf16_host_bits(cache.idx_k))
    for b in range(B):
        rp, rt, score = indexer.full(q[b], w[b], paged_to_logical(ik, pt, b, N), NB, PER, K)
        assert len(rp) == NB * PER and len(rt) == K
        check_index_set(pool[b, :pool_len[b]], rp, lambda e: score[e], f"pool of query {b}")
        check_index_set(topk[b, :topk_len[b]], rt, lambda e: score[e], f"selection of query {b}")
    # the Reuse layer took this selection and left it as it was
    for a, b in zip(ends[0][2], ends[1][2]):
        assert torch.equal(a, b)
    assert np.array_equal(c(ends[0][2][0]), topk) and np.array_equal(c(ends[0][2][1]), topk_len)


@pytest.mark.parametrize("i", [0, 1])
def test_every_stage_of_a_layer(stepped, i):
    s, _, starts, ends = stepped
    L, cache, window = s["layers"][i], s["cache"], s["window"]
    (h, res), (res_out, out, topk) = starts[i], ends[i]
    r = rows.add(h, res, True)
    assert np.array_equal(res_out, r)
    y = rows.rms_norm(r, c(L.w_norm.float()), 1e-6)
    assert (np.abs(f64(L.x) - y) <= np.abs(y) * (5 * U + UB) * 1.001).all()
    codes, scales = rows.fp4_quantize(c(L.x.float()))
    assert np.array_equal(c(L.x4.codes), codes) and np.array_equal(c(L.x4.row_scales()), scales)

    def check_linear(got, x, w, gx, gw):
        ref, mag = rows.fp4_linear(*fp4(x), *fp4(w), gx, gw)
        assert (np.abs(f64(got) - ref) <= (x.cols // 64 + 16) * 4 * U * mag + (2 * U + UB) * np.abs(ref)).all()

    q = csa2.fp4_linear(L.x4, L.w_q)
    check_linear(q, L.x4, L.w_q, 1.0, float(L.w_q.gscale))
    if L.w_iq is not None:
        check_linear(L.q_idx.view(B, -1), L.x4, L.w_iq, 1.0, float(L.w_iq.gscale))
    pos, cos, sin = c(s["pos"]), c(L.cos), c(L.sin)
    turned = rows.rope(f64(q).reshape(B, HQ, D), pos, cos, sin, True, False, D - D_ROPE)
    assert np.abs(f64(L.q) - turned).max() <= 2 * UB * np.abs(turned).max()
    pt = c(cache.page_table)
    for b in range(B):
        e = c(topk[0])[b, :c(topk[1])[b]]
        o, _ = attention.sparse_attention(f64(L.q)[b], paged_to_logical(c(cache.codes), pt, b, N),
                                          paged_to_logical(c(cache.scales), pt, b, N), e, c(window["swa"]),
                                          c(window["swa_scale"]), b * W, W, 1 / math.sqrt(D))
        back = rows.rope(o[None], pos[b:b + 1], cos, sin, True, True, D - D_ROPE)[0]
        assert np.linalg.norm(f64(L.a)[b] - back) <= (2e-3 + 2 * UB) * np.linalg.norm(back)
    codes, scales = rows.fp4_quantize(c(L.a.float()).reshape(B, -1), float(L.a4.gscale))
    assert np.array_equal(c(L.a4.codes), codes) and np.array_equal(c(L.a4.row_scales()), scales)
    check_linear(out, L.a4, L.w_o, float(L.a4.gscale), float(L.w_o.gscale))
