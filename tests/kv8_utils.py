"""Inputs of the paged 8-bit cache's tests: a NumPy cache, its copy on the GPU, and ragged steps."""
import numpy as np
import torch

from fp4_compressed_sparse_02_gb300 import csa2
from oracle import formats, kv8

DEV = "cuda"


def bf16(x):
    return formats.bf16_value(formats.bf16_round(np.asarray(x, np.float64))).astype(np.float32)


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def new_cache(r, S, most, H, D, spare=2, mean=True, fill=0x7F):
    """An empty cache whose every byte is `fill` (a NaN): what is not written must not be read."""
    P = S * most + spare
    table = r.permutation(P)[:S * most].reshape(S, most).astype(np.int32)
    return {"k": np.full((P, H, 64, D), fill, np.uint8), "v": np.full((P, H, 64, D), fill, np.uint8),
            "k_scale": np.full((P, H), np.nan, np.float32), "v_scale": np.full((P, H), np.nan, np.float32),
            "mean": np.full((P, H, D), 77, np.int8) if mean else None,
            "mean_scale": np.full((P, H), np.nan, np.float32) if mean else None, "table": table}


def to_gpu(c):
    opt = lambda n: None if c[n] is None else gpu(c[n])
    return csa2.Kv8Cache(gpu(c["k"]), gpu(c["v"]), gpu(c["k_scale"]), gpu(c["v_scale"]), gpu(c["table"]), opt("mean"),
                         opt("mean_scale"))


def check_cache(g, c):
    """Bit for bit (NaN scales of unwritten pages compare as bytes)."""
    for name in ("k", "v", "k_scale", "v_scale", "mean", "mean_scale"):
        if c[name] is not None:
            got = getattr(g, name).cpu().numpy()
            bad = np.argwhere(got.view(np.uint8) != c[name].view(np.uint8))
            assert not len(bad), (name, len(bad), bad[0])


def starts(add, before=0):
    return np.concatenate(([0], np.cumsum(add))).astype(np.int32) + np.int32(before)


def fill(r, c, lengths, spread=3):
    """Random contents of `lengths` tokens a sequence, appended in one step by the oracle."""
    H, D = c["k"].shape[1], c["k"].shape[3]
    T = int(sum(lengths))
    x = [bf16(r.standard_normal((T, H, D)) * np.exp2(r.integers(-spread, spread + 1, (T, 1, 1)))) for _ in range(2)]
    kv8.append(c, x[0], x[1], starts(lengths), np.asarray(lengths, np.int32))


def strided(a, dtype, pad):
    """[T, H, D] as a slice of wider rows of NaN."""
    if not pad:
        return gpu(a, dtype)
    T, H, D = a.shape
    t = torch.full((T, H * D + 2 * pad), float("nan"), dtype=dtype, device=DEV)
    t[:, pad:pad + H * D] = gpu(a, dtype).reshape(T, H * D)
    return t[:, pad:pad + H * D].unflatten(1, (H, D))


def check_attn(out, lse, c, q, start, length, scale, window=0, pages=None, out_eps=2.0 ** -8, q_eps=0.0):
    """Every row of the step against the oracle.  The bound, from the precision that the header states: probabilities
    in fp16 (2^-11, or 2^-25 absolute), logits in float32 sums of D terms (D + 8 roundings, twice: numerator and
    sum), 2^-14 for the exponential, the sums over up to 2^10 pages and their merging, one rounding of the result.
    q_eps: how far an element of q may be off, relative to the row's largest."""
    out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    H, D = c["k"].shape[1], c["k"].shape[3]
    Hq = q.shape[1]
    G = Hq // H
    for s in range(len(length)):
        for t in range(start[s], start[s + 1]):
            n = int(length[s] - (start[s + 1] - t) + 1)
            for h in range(H):
                sel = list(range(-(-n // 64))) if pages is None else [j for j in pages[t][h] if 0 <= j < -(-n // 64)]
                pos = (np.array(sel, np.int64)[:, None] * 64 + np.arange(64)).reshape(-1)
                seen = (pos < n) & ((pos >= n - window) if window else True)
                k, v = (kv8.rows(c, x, s, sel, h) for x in "kv")
                for g in range(h * G, (h + 1) * G):
                    o, l, (a, sv, x) = kv8.attend(q[t, g].astype(np.float64), k, v, seen, scale)
                    e = (D + 8) * 2.0 ** -24 * x
                    if q_eps and seen.any():
                        e += q_eps * np.abs(q[t, g]).max() * np.abs(k[seen]).sum(1).max() * scale
                    if not seen.any():
                        assert (out[t, g] == 0).all() and lse[t, g] == -np.inf, (s, t, g)
                        continue
                    bound = (2.0 ** -11 + 2.0 ** -14 + 2 * e) * a + 2.0 ** -25 * sv
                    bound = bound + out_eps * (np.abs(o) + bound)
                    nan = np.isnan(o)
                    assert (np.isnan(out[t, g]) == nan).all(), (s, t, g)
                    err = np.abs(out[t, g] - o)[~nan]
                    assert (err <= bound[~nan]).all(), (s, t, g, float((err / bound[~nan]).max()))
                    if np.isnan(l):
                        assert np.isnan(lse[t, g])
                    else:
                        assert abs(lse[t, g] - l) <= e + 2.0 ** -16 + 2.0 ** -21 * abs(l), (s, t, g, lse[t, g], l)
