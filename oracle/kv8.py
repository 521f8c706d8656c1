"""The paged 8-bit key-value cache in NumPy: tables, append, page selection and attention, page by page and row by
row, float64 except where the definition rounds to float32 or E4M3."""
import math

import numpy as np

from .formats import e4m3_encode, e4m3_value

PAGE = 64


def plan(length, add, table, free, head, tokens):
    """-> dict of start, seq, pos, slot, length, head; `table` is extended in place."""
    S, most = table.shape
    out = dict(start=[0], seq=[], pos=[], slot=[], length=[])
    for s in range(S):
        held, n = max(0, int(length[s])), max(0, int(add[s]))
        n = max(0, min(n, most * PAGE - held, tokens - len(out["seq"])))
        for j in range(-(-held // PAGE), -(-(held + n) // PAGE)):
            table[s, j] = free[head] if head < len(free) else -1
            head = min(head + 1, len(free))
        for p in range(held, held + n):
            page = int(table[s, p // PAGE])
            out["seq"].append(s)
            out["pos"].append(p)
            out["slot"].append(PAGE * page + p % PAGE if page >= 0 else -1)
        out["start"].append(len(out["seq"]))
        out["length"].append(held + n)
    for x in ("seq", "pos", "slot"):
        out[x] += [-1] * (tokens - len(out[x]))
    return {x: np.array(v, np.int64) for x, v in out.items()} | {"head": head}


def power_for(a):
    """The least power of two, 2^-126 at least, that a / 448 does not exceed."""
    e = -126
    while 448.0 * math.ldexp(1.0, e) < a:
        e += 1
    return math.ldexp(1.0, e)


def encode(x):
    """E4M3 bytes of float32 values; NaN is 0x7F."""
    return np.where(np.isnan(x), 0x7F, e4m3_encode(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf))).astype(np.uint8)


def summary(rows):
    """(int8 summary, the factor of the key scale) of 64 rows of E4M3 values [64, D]."""
    m = np.nansum(rows, axis=0)
    u = np.float32(np.abs(m).max()) / np.float32(127)
    if u == 0:
        return np.zeros(m.shape, np.int8), np.float32(0)
    return np.rint(m.astype(np.float32) / u).astype(np.int8), np.float32(u / np.float32(64))


def append(cache, k, v, start, length):
    """cache: dict of k, v uint8 [P, H, 64, D], k_scale, v_scale float32 [P, H], mean, mean_scale (or None), table;
    changed in place.  k, v float32 [T, H, D]."""
    for s in range(len(length)):
        p, end = int(length[s]) - int(start[s + 1] - start[s]), int(length[s])
        t = int(start[s])
        while p < end:
            held, n = p % PAGE, min(PAGE - p % PAGE, end - p)
            page = int(cache["table"][s, p // PAGE])
            for h in range(k.shape[1]):
                for x, name in ((k, "k"), (v, "v")):
                    rows = x[t:t + n, h].astype(np.float32)
                    finite = np.abs(rows[np.isfinite(rows)])
                    scale = power_for(float(finite.max()) if finite.size else 0.0)
                    b = cache[name][page, h]
                    if held:
                        old = float(cache[name + "_scale"][page, h])
                        scale = max(scale, old)
                        if scale > old:
                            b[:held] = encode((e4m3_value(b[:held]) * (old / scale)).astype(np.float32))
                    b[held:held + n] = encode((rows.astype(np.float64) / scale).astype(np.float32))
                    cache[name + "_scale"][page, h] = scale
                if cache["mean"] is not None and held + n == PAGE:
                    m, u = summary(e4m3_value(cache["k"][page, h]))
                    cache["mean"][page, h] = m
                    cache["mean_scale"][page, h] = np.float32(u * cache["k_scale"][page, h])
            p, t = p + n, t + n


def select(cache, q, s, n, k, first, recent):
    """Pages of one token that sees n positions of sequence s, for each key head.  q float32 [Hq, D]."""
    H = cache["k"].shape[1]
    P = -(-n // PAGE)
    out = []
    for h, group in enumerate(np.split(q.astype(np.float64), H)):
        if P <= k:
            out.append(list(range(P)))
            continue
        c = group.sum(0).astype(np.float32)
        finite = np.abs(c[np.isfinite(c)])
        u = (finite.max() if finite.size else np.float32(0)) / np.float32(127)
        with np.errstate(invalid="ignore"):
            r = np.rint(c / u) if u > 0 else np.zeros_like(c)
        r = np.where(np.isnan(r), 0, np.clip(r, -127, 127)).astype(np.int64)
        mid = list(range(first, P - recent))
        ids = [int(cache["table"][s, j]) for j in mid]
        score = [np.float32(np.float32(int(cache["mean"][i, h].astype(np.int64) @ r)) * cache["mean_scale"][i, h]) for i in ids]
        best = sorted(range(len(mid)), key=lambda i: (-score[i], i))[:k - first - recent]
        out.append(sorted(list(range(first)) + [mid[i] for i in best] + list(range(P - recent, P))))
    return out


def rows(cache, plane, s, pages, h):
    """float64 rows [64 * len(pages), D] of these pages of sequence s."""
    ids = [int(cache["table"][s, j]) for j in pages]
    b = e4m3_value(cache[plane][ids, h]) * cache[plane + "_scale"][ids, h].astype(np.float64)[:, None, None]
    return b.reshape(-1, b.shape[-1])


def attend(q, k, v, seen, scale):
    """One query head q [D] over rows k, v [N, D], seen [N]: (out, lse, bounds).  bounds: (sum of softmax |v|, sum of
    |v|, the largest sum |q k| scale), for error bounds."""
    if not seen.any():
        z = np.zeros(q.shape)
        return z, -np.inf, (z, z, 0.0)
    k, v = k[seen], v[seen]
    x = k @ q * scale
    top = x.max()
    p = np.exp(x - top)
    z = p.sum()
    return (p / z) @ v, top + np.log(z), ((p / z) @ np.abs(v), np.abs(v).sum(0), float((np.abs(k) @ np.abs(q)).max() * scale))
