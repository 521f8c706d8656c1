"""One CSA2 attention block of a decode step, from the residual stream back to it:

    x        = norm(h + residual)                              rms_norm
    cache   <- FP4 entry and indexer K of x                    compress_quant (m = 1)
    x4       = FP4 of x                                        fp4_quant
    q        = rope(x4 . W_q)                                  fp4_linear, rope
    q_idx    = x4 . W_iq;  top-k                               fp4_linear, index_full (Full layers)
    a        = sparse attention(q, cache, top-k, window)       sparse_attn
    out      = FP4 of rope^-1(a) . W_o                         rope (inverse), fp4_quant, fp4_linear

The sliding window is the caller's: a step reads the rows it is given and does not write the new token's
(csa2.swa_quant does).  The entry is key and value at once, so what the attention returns still carries the keys'
rotation; the query's position turns it back.  Every buffer is allocated once, and a step can be
captured in a CUDA graph.  ``python -m fp4_compressed_sparse_02_gb300.layer`` runs a Full layer and
a Reuse layer of a decode batch and prints the time of a step.
"""
import math

import torch

from . import csa2


def quantise_weight(w):
    """Weights [N, K] to FP4 rows with the matrix's scale that puts its largest group scale on the
    largest E4M3 value."""
    g = (w.float().abs().amax() / (6 * 448)).clamp(min=1e-30).reshape(1)
    return csa2.fp4_quant(w, g)


class Csa2Layer:
    """Weights and buffers of one layer for B queries, one new token each.

    w_norm bf16 [d_model]; w_q, w_o, w_iq Fp4Rows [Hq*d, d_model], [d_model, Hq*d], [H_i*d_ik,
    d_model] (w_iq None: a Reuse layer); w_kv, w_ik bf16 [d_model, d], [d, d_ik] (None: the cache is
    written by another layer); a_scale: the matrix scale of the attention output's FP4 (float32 [1])."""

    def __init__(self, B, Hq, d, w_norm, w_q, w_o, cos, sin, *, w_iq=None, head_weights=None, w_kv=None, w_ik=None,
                 a_scale=None, ws=None):
        dev, d_model = w_norm.device, w_norm.shape[0]
        self.Hq, self.d, self.cos, self.sin = Hq, d, cos, sin
        self.w_norm, self.w_q, self.w_o, self.w_iq, self.head_weights = w_norm, w_q, w_o, w_iq, head_weights
        self.w_kv, self.w_ik = w_kv, w_ik
        self.ws = ws or csa2.Workspace(dev)
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=dev)
        self.x = new(B, d_model)
        self.x4 = csa2.Fp4Rows.allocate(B, d_model, dev)
        self.q = new(B, Hq, d)
        self.q_idx = None if w_iq is None else new(B, head_weights.shape[1], w_iq.rows // head_weights.shape[1])
        self.a, self.lse = new(B, Hq, d), new(B, Hq, dtype=torch.float32)
        self.a4 = csa2.Fp4Rows.allocate(B, Hq * d, dev, a_scale)
        self.out = new(B, d_model)

    def step(self, h, residual, cache, seq, pos, index, window, topk=None):
        """h bf16 [B, d_model] is added to residual [B, d_model] (updated in place).  seq, pos int32
        [B]: the tokens' sequences and positions (their entries' indices).  index: dict(n_vis, max_n,
        num_blocks, per_block, k, out) of index_full; window: dict(swa, swa_scale, swa_start, swa_len,
        swa_max).  A Reuse layer takes topk = (topk, topk_len) of an earlier one.  Returns (out bf16
        [B, d_model], the top-k used)."""
        B = h.shape[0]
        csa2.rms_norm(h, self.w_norm, residual=residual, residual_out=residual, out=self.x)
        if self.w_kv is not None:
            csa2.compress_quant(cache, seq, pos, m=1, H=self.x, W_kv=self.w_kv, pos=pos, rope_cos=self.cos,
                                rope_sin=self.sin, W_ik=self.w_ik, ws=self.ws)
        csa2.fp4_quant(self.x, out=self.x4)
        csa2.fp4_linear(self.x4, self.w_q, out=self.q.view(B, -1))
        csa2.rope(self.q, pos, self.cos, self.sin, out=self.q)
        if self.w_iq is not None:
            csa2.fp4_linear(self.x4, self.w_iq, out=self.q_idx.view(B, -1))
            pool = csa2.index_full(cache, self.q_idx, self.head_weights, seq, index["n_vis"], index["max_n"],
                                   index["num_blocks"], index["per_block"], index["k"], out=index["out"], ws=self.ws)
            topk = pool[2:]
        csa2.sparse_attn(cache, self.q, seq, topk[0], topk[1], window["swa"], window["swa_scale"], window["swa_start"],
                         window["swa_len"], window["swa_max"], out=self.a, lse=self.lse, ws=self.ws)
        csa2.rope(self.a, pos, self.cos, self.sin, inverse=True, out=self.a)
        csa2.fp4_quant(self.a.view(B, -1), out=self.a4)
        return csa2.fp4_linear(self.a4, self.w_o, out=self.out), topk


def build(B=32, n=4096, d_model=5120, Hq=64, d=512, H_i=8, d_ik=128, d_rope=64, W=128, k=512, num_blocks=2048,
          per_block=8, seed=0, device="cuda"):
    """A Full layer and a Reuse layer over B sequences of n entries with random weights, inputs and
    cache.  Returns (run, state): run() is one step of both."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rnd = lambda *s, sigma=1.0: (torch.randn(s, generator=g, device=device) * sigma)
    w4 = lambda N, K: quantise_weight(rnd(N, K, sigma=1 / math.sqrt(K)))
    bf = lambda t: t.to(torch.bfloat16)
    cache = csa2.PagedCache.allocate(B, n, d, d_ik, device)
    cache.codes.random_(0, 256, generator=g)
    cache.scales.random_(0x20, 0x40, generator=g)
    cache.idx_k.copy_(bf(rnd(*cache.idx_k.shape)))
    cos, sin = csa2.rope_table(n, d_rope, device=device)
    ws = csa2.Workspace(device)
    a_scale = torch.full((1,), 1 / 64, device=device)

    def layer(full):
        kw = dict(w_iq=w4(H_i * d_ik, d_model), head_weights=rnd(B, H_i, sigma=1 / math.sqrt(H_i)),
                  w_kv=bf(rnd(d_model, d, sigma=1 / math.sqrt(d_model))),
                  w_ik=bf(rnd(d, d_ik, sigma=1 / math.sqrt(d)))) if full else {}
        return Csa2Layer(B, Hq, d, bf(1 + rnd(d_model, sigma=0.1)), w4(Hq * d, d_model), w4(d_model, Hq * d), cos, sin,
                         a_scale=a_scale, ws=ws, **kw)

    layers = [layer(True), layer(False)]
    i32 = lambda t: t.to(torch.int32)
    seq = i32(torch.arange(B, device=device))
    pos = torch.full((B,), n - 1, dtype=torch.int32, device=device)
    swa = (torch.randint(3, 14, (B * W, d), generator=g, device=device) << 3).to(torch.uint8)
    window = dict(swa=swa, swa_scale=torch.rand(B * W, generator=g, device=device) * 0.015 + 0.005, swa_start=i32(seq * W),
                  swa_len=torch.full((B,), W, dtype=torch.int32, device=device), swa_max=W)
    new = lambda *s: torch.empty(s, dtype=torch.int32, device=device)
    index = dict(n_vis=pos + 1, max_n=n, num_blocks=num_blocks, per_block=per_block, k=k,
                 out=(new(B, num_blocks * per_block), new(B), new(B, k), new(B)))
    state = dict(layers=layers, h=bf(rnd(B, d_model)), residual=bf(rnd(B, d_model)), cache=cache, seq=seq, pos=pos,
                 index=index, window=window)

    def run():
        s = state
        out, topk = layers[0].step(s["h"], s["residual"], cache, seq, pos, index, window)
        return layers[1].step(out, s["residual"], cache, seq, pos, index, window, topk)[0]

    return run, state


def main():
    run, _ = build()
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    times = []
    for _ in range(20):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    err = csa2.device_error()
    print(f"one Full and one Reuse layer, 32 queries over 4096 entries: {sorted(times)[10]:.1f} us a step, "
          f"device error word {err}")


if __name__ == "__main__":
    main()
