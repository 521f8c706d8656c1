"""What is measured of the paged 8-bit key-value cache beside the CSA2 cache: the tables of a step's
tokens and pages, the append that quantises new keys and values, attention of one to many new tokens
of each sequence over it, and attention over the pages that a cheap score selects for each token.

Definitions (pages of 64 tokens; every listed rounding is the only one):

  plan    sequence s holds length[s] tokens and gets add[s] more, as far as `tokens` rows and its row of
          the page table reach; their rows stand one after the other, sequence by sequence, from start[s]
          on.  Pages that it does not have yet come off free[head], in order of sequence and page.  Row t
          of sequence s at position p: slot = 64 table[s][p / 64] + p % 64; rows past the last are -1.
  append  per page, head and plane (keys, values): scale = the least power of two (2^-126 at least)
          that puts the largest finite new value within 448, or the page's old scale if that is larger
          and the page held tokens; bytes = E4M3(x / scale), infinities saturate; a larger scale
          requantises the page's old bytes.  A page that becomes full gets a summary of its keys:
          m = the sum of its 64 rows of E4M3 values, a = max|m| / 127, summary = round(m / a) in 8-bit
          integers, its scale = (a / 64) x key scale.
  attn    token at position p of sequence s: the softmax over the positions max(0, p + 1 - window) .. p
          of scale q . k, times the values; lse = log of its sum.  Query heads share key heads in groups.
  sparse  for each token and key head: c = the sum of the group's query heads (rounded once to
          float32), r = round(c / (max|c| / 127)); a page's score = (r . summary) as a float32 x the
          summary's scale; kept are the `first` oldest pages, the `recent` newest, and the best of the
          others up to k, equal scores to the older page.  attn over the kept pages.
"""
import math
import random

import torch

own = False

DEV = "cuda"
PAGE = 64
F8 = torch.float8_e4m3fn


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step of 64 requests: one row each, a new page now and then; latency
        dict(name="plan_decode", op="plan", S=64, most=131072, new=1, some=1.0, cap=64, mix=1),
        # a prefill step of many short and long prompts, some of the requests idle
        dict(name="plan_prefill", op="plan", S=512, most=65536, new=1024, some=0.9, cap=262144, mix=2),
        # the same decode step's keys and values: part-filled pages, some of which grow their scale
        dict(name="append_decode", op="append", S=64, most=8192, new=1, some=1.0, Hkv=8, D=128, x="bf16", mix=3),
        # prompts of a prefill step, out of a fused projection
        dict(name="append_prefill", op="append", S=9, most=16384, new=8192, some=1.0, Hkv=8, D=128, x="bf16", mix=4),
        # one token of one request: latency, one sequence over the whole GPU
        dict(name="attn_token", op="attn", S=1, least=4097, most=4097, new=1, some=1.0, Hq=64, Hkv=8, D=128, window=0,
             pad=0, mix=5),
        # a decode batch with contexts of all lengths up to 64K: reading the cache
        dict(name="attn_decode", op="attn", S=64, least=1, most=65536, new=1, some=1.0, Hq=64, Hkv=8, D=128, window=0,
             pad=2048, mix=6),
        # up to six positions a request to be verified
        dict(name="attn_verify", op="attn", S=32, least=8192, most=32768, new=6, some=1.0, Hq=64, Hkv=8, D=128, window=0,
             pad=0, mix=7),
        # a prefill chunk behind a long context and a fresh prompt: the tensor cores
        dict(name="attn_prefill", op="attn", S=2, least=32768, most=32768, new=4096, some=1.0, Hq=64, Hkv=8, D=128,
             window=0, pad=2048, fresh=True, mix=8),
        # odd everything: seven query heads a key head, 64 channels, a sliding window, idle requests
        dict(name="attn_odd_window", op="attn", S=17, least=33, most=20011, new=41, some=0.8, Hq=21, Hkv=3, D=64,
             window=1001, pad=8, mix=9),
        # one token at a context of a million
        dict(name="sparse_token_1m", op="sparse", S=1, least=1048571, most=1048571, new=1, some=1.0, Hq=64, Hkv=8, D=128,
             k=64, mix=10),
        # a decode batch at 32K to 128K
        dict(name="sparse_decode", op="sparse", S=32, least=32768, most=131072, new=1, some=1.0, Hq=64, Hkv=8, D=128,
             k=64, mix=11),
        # a prefill chunk, every token with pages of its own
        dict(name="sparse_prefill", op="sparse", S=1, least=32768, most=32768, new=2048, some=1.0, Hq=64, Hkv=8, D=128,
             k=32, mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "attn", "sparse", "sparse"])
    mix = rng.randrange(1 << 30)
    some = rng.choice([1.0, 1.0, 0.7])
    if op == "plan":
        S = _log(rng, 1, 2048)
        new = _log(rng, 1, min(2048, 262144 // S))
        return dict(op=op, S=S, most=min(_log(rng, 64, 262144), (1 << 25) // S), new=new, some=some,
                    cap=S * new + rng.choice([0, 0, 5]), mix=mix)
    Hkv = rng.choice([1, 2, 3, 8])
    D = rng.choice([64, 128, 128])
    if op == "append":
        S = _log(rng, 1, 256)
        return dict(op=op, S=S, most=_log(rng, 1, 32768), new=_log(rng, 1, min(16384, 65536 // S)), some=some, Hkv=Hkv, D=D,
                    x=rng.choice(["bf16", "bf16", "f32"]), mix=mix)
    G = rng.choice([1, 3, 4, 7, 8, 16])
    if op == "attn":
        least = _log(rng, 1, 32768)
        new = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
        most = max(least, min(_log(rng, 64, 131072), 131072 * 4096 // (new * G * Hkv)))
        S = max(1, min(_log(rng, 1, 128), (1 << 31) // (most * Hkv * D * 2), (1 << 35) // (new * G * Hkv * most)))
        return dict(op=op, S=S, least=least, most=most, new=new, some=some, Hq=G * Hkv, Hkv=Hkv, D=D,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]), pad=rng.choice([0, 0, 8, D]), mix=mix)
    k = rng.choice([4, 13, 32, 64])
    new = 1 if rng.random() < 0.6 else _log(rng, 2, 512)
    most = _log(rng, 512, 262144)
    S = max(1, min(_log(rng, 1, 64), (1 << 31) // (most * Hkv * D * 2), 16384 // new))
    return dict(op=op, S=S, least=max(1, most // 8), most=most, new=new, some=some, Hq=G * Hkv, Hkv=Hkv, D=D, k=k, mix=mix)


def _mix(c):
    """(tokens after the step, new tokens) of each sequence."""
    r = random.Random(c["mix"])
    length, add = [], []
    for s in range(c["S"]):
        n = c["new"] if s == 0 or c["new"] == 1 else r.randint(1, c["new"])
        n = n if s == 0 or r.random() < c["some"] else 0
        old = r.randint(0, c["most"])
        if "least" in c:                                     # the length after the step lies between the two
            total = c["most"] if s == 0 else r.randint(c["least"], c["most"])
            n = min(n, total)
            if c.get("fresh") and s:
                total = n                                    # a prompt without a past
            length.append(total)
        else:
            length.append(old + n)
        add.append(n)
    return length, add


def _size(t):
    return 2 if t == "bf16" else 4


def _visible(c):
    """Pairs of a token and a position that it sees."""
    length, add = _mix(c)
    n = 0
    for a, b in zip(length, add):
        w = c.get("window", 0) or a
        lo = a - b + 1                                       # what the first new token sees, without the window
        k = max(0, min(b, w - lo + 1))                       # tokens whose window is not full
        n += k * lo + k * (k - 1) // 2 + (b - k) * w
    return n


def work(case):
    c = case
    length, add = _mix(c)
    T = sum(add)
    if c["op"] == "plan":
        pages = sum(-(-a // PAGE) - -(-(a - b) // PAGE) for a, b in zip(length, add))
        return {"bytes": 12 * c["cap"] + 16 * c["S"] + 8 * pages, "flops": 0}
    H, D = c["Hkv"], c["D"]
    if c["op"] == "append":
        touched = sum(-(-a // PAGE) - (a - b) // PAGE for a, b in zip(length, add) if b)
        return {"bytes": T * H * D * 2 * (_size(c["x"]) + 1) + touched * H * 8, "flops": 4.0 * T * H * D}
    G = c["Hq"] // H
    io = T * c["Hq"] * (4 * D + 4)
    if c["op"] == "attn":
        kv = sum(min(a, b - 1 + (c["window"] or a)) for a, b in zip(length, add) if b)
        return {"bytes": kv * H * (2 * D + 8 / PAGE) + io, "flops": 4.0 * _visible(c) * c["Hq"] * D}
    pages = [min(c["k"], -(-(a - b + 1 + i) // PAGE)) for a, b in zip(length, add) for i in range(b)]
    most = sum(-(-a // PAGE) for a, b in zip(length, add) if b)
    scored = sum((a - b + 1 + i) // PAGE for a, b in zip(length, add) for i in range(b))
    return {"bytes": most * H * (D + 4) + min(sum(pages), most) * H * (2 * D * PAGE + 8) + io + 4 * T * H * (c["k"] + 1),
            "flops": 4.0 * sum(pages) * PAGE * c["Hq"] * D + 2.0 * scored * H * D}


# ---- inputs -----------------------------------------------------------------------------------

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _start(add):
    return _i32([sum(add[:i]) for i in range(len(add) + 1)]) if len(add) < 64 else torch.nn.functional.pad(
        _i32(add).cumsum(0), (1, 0)).to(torch.int32)


def _plane(P, H, D, g):
    """E4M3 bytes of N(0, 1) values, and the powers of two that scale them to about that."""
    x = torch.empty((P, H, PAGE, D), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 28) // (H * PAGE * D))
    for a in range(0, P, step):
        n = min(P, a + step) - a
        x[a:a + n] = (64 * torch.randn((n, H, PAGE, D), generator=g, device=DEV)).clamp(-448, 448).to(F8).view(torch.uint8)
    return x, torch.exp2(torch.randint(-7, -4, (P, H), generator=g, device=DEV).float())


def _summary(rows, scale):
    """(summary, its scale) of pages of E4M3 values [..., 64, D] in float32."""
    m = rows.sum(-2)                                         # exact: whole multiples of 2^-9 below 2^15
    a = m.abs().amax(-1, keepdim=True) / torch.full((), 127.0, device=DEV)
    r = torch.where(a > 0, (m / a).round().clamp(-127, 127), 0)
    return r.to(torch.int8), (a.squeeze(-1) * (1 / 64)) * scale


def _cache(c, length, g, means):
    H, D = c["Hkv"], c["D"]
    need = [-(-n // PAGE) for n in length]
    P = sum(need) + 3
    s = {}
    s["k"], s["k_scale"] = _plane(P, H, D, g)
    s["v"], s["v_scale"] = _plane(P, H, D, g)
    table = torch.zeros((len(length), max(need) + 1), dtype=torch.int32, device=DEV)
    at = torch.arange(table.shape[1], device=DEV)[None] < _i32(need)[:, None]
    table[at] = torch.randperm(P, generator=g, device=DEV)[:sum(need)].to(torch.int32)
    s["table"] = table
    if means:
        s["mean"] = torch.zeros((P, H, D), dtype=torch.int8, device=DEV)
        s["mean_scale"] = torch.zeros((P, H), device=DEV)
        step = max(1, (1 << 28) // (H * PAGE * D))
        for a in range(0, P, step):
            s["mean"][a:a + step], s["mean_scale"][a:a + step] = _summary(s["k"][a:a + step].view(F8).float(),
                                                                         s["k_scale"][a:a + step])
    return s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    length, add = _mix(c)
    T = sum(add)
    if c["op"] == "plan":
        S, mp = c["S"], max(-(-n // PAGE) for n in length) + 2
        old = [a - b for a, b in zip(length, add)]
        need = sum(-(-a // PAGE) for a in length)
        ids = torch.randperm(need + 64, generator=g, device=DEV).to(torch.int32)
        have = torch.arange(mp, device=DEV)[None] * PAGE < _i32(old)[:, None]
        table = torch.full((S, mp), -1, dtype=torch.int32, device=DEV)
        held = sum(-(-a // PAGE) for a in old)
        table[have] = ids[:held]
        return {"case": c, "length": _i32(old), "add": _i32(add), "table": table, "free": ids[held:].clone(), "head": _i32([0])}
    H, D = c["Hkv"], c["D"]
    s = _cache(c, length, g, c["op"] != "attn")
    s |= {"case": c, "start": _start(add), "length": _i32(length)}
    if c["op"] == "append":
        # keys and values are slices of a fused projection; tokens differ in size, so that scales grow
        x = torch.randn((T, H * D * 2 + 64), generator=g, device=DEV)
        x = (x * torch.exp2(torch.randn((T, 1), generator=g, device=DEV))).to(_TYPES[c["x"]])
        s["x"], s["y"] = x[:, 64:64 + H * D].unflatten(1, (H, D)), x[:, 64 + H * D:].unflatten(1, (H, D))
    else:
        w = c["Hq"] * D
        q = torch.randn((T, w + c.get("pad", 0)), generator=g, device=DEV)
        s["q"] = (q * torch.exp2(torch.rand((T, 1), generator=g, device=DEV))).to(torch.bfloat16)[:, :w].unflatten(1, (c["Hq"], D))
    return s


# ---- the plain form ---------------------------------------------------------------------------

def _plan_plain(s):
    c, table, free = s["case"], s["table"], s["free"]
    S, mp = table.shape
    old = s["length"].long()
    add = torch.minimum(s["add"].long(), mp * PAGE - old)
    end = add.cumsum(0).clamp(max=c["cap"])
    start = torch.nn.functional.pad(end, (1, 0))
    new = old + start[1:] - start[:-1]
    p0, p1 = (old + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    base = s["head"] + (p1 - p0).cumsum(0) - p1
    j = torch.arange(mp, device=DEV)[None]
    at = (base[:, None] + j).clamp(0, free.shape[0] - 1)
    table.copy_(torch.where((j >= p0[:, None]) & (j < p1[:, None]), free[at], table))
    t = torch.arange(c["cap"], device=DEV)
    seq = torch.searchsorted(end, t, right=True)
    real = t < end[-1]
    q = seq.clamp(max=S - 1)
    pos = new[q] - end[q] + t
    slot = table[q, (pos // PAGE).clamp(0, mp - 1)] * PAGE + pos % PAGE
    i = lambda v: torch.where(real, v, -1).to(torch.int32)
    return {"start": start.to(torch.int32), "seq": i(seq), "pos": i(pos), "slot": i(slot), "length": new.to(torch.int32),
            "head": (s["head"] + (p1 - p0).sum()).to(torch.int32), "table": table}


def _scale_for(x):
    """The least power of two 2^e, e >= -126, with |x| / 2^e <= 448, in float32."""
    m, e = torch.frexp(x)                                    # x = m 2^e, m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.ldexp(torch.ones((), device=DEV), torch.where(x > 0, e, -126).clamp(min=-126))


def _append_plain(s):
    c, start, length = s["case"], s["start"].long(), s["length"].long()
    T = s["x"].shape[0]
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(start[1:].contiguous(), t, right=True)
    pos = length[seq] - start[seq + 1] + t
    page = s["table"][seq, pos // PAGE].long()
    slot = pos % PAGE
    P = s["k"].shape[0]
    first = torch.full((P,), PAGE, device=DEV).scatter_reduce_(0, page, slot, "amin")          # the first new slot of a page
    last = torch.full((P,), -1, device=DEV).scatter_reduce_(0, page, slot, "amax")
    touched = torch.zeros((P,), dtype=torch.bool, device=DEV).index_fill_(0, page, True)
    old = torch.arange(PAGE, device=DEV)[None] < torch.where(touched, first, 0)[:, None]       # slots held before
    for x, plane, scale in ((s["x"], s["k"], s["k_scale"]), (s["y"], s["v"], s["v_scale"])):
        top = torch.where(x.isfinite(), x, 0).float().abs().amax(-1)
        need = torch.zeros_like(scale).index_reduce_(0, page, _scale_for(top), "amax")
        new = torch.where(touched[:, None], torch.maximum(need, torch.where(first[:, None] > 0, scale, 0)), scale)
        grown = (new > scale) & touched[:, None]
        ids, heads = torch.nonzero(grown & (first[:, None] > 0), as_tuple=True)
        ratio = (scale[ids, heads] / new[ids, heads])[:, None, None]
        was = plane[ids, heads]
        held = old[ids][:, :, None]
        plane[ids, heads] = torch.where(held, (was.view(F8).float() * ratio).to(F8).view(torch.uint8), was)
        scale.copy_(new)
        v = x.float() / new[page][:, :, None]
        plane[page, :, slot] = v.clamp(-448, 448).to(F8).view(torch.uint8)
    full = torch.nonzero(touched & (last == PAGE - 1)).squeeze(1)
    s["mean"][full], s["mean_scale"][full] = _summary(s["k"][full].view(F8).float(), s["k_scale"][full])
    return _append_outputs(s)


def _append_outputs(s):
    return {"k": s["k"].view(F8), "v": s["v"].view(F8), "k_scale": s["k_scale"], "v_scale": s["v_scale"], "mean": s["mean"],
            "mean_scale": s["mean_scale"]}


def _softmax_plain(q, k, v, seen):
    """q [.., M, D], k, v [.., N, D], seen [.., M, N] in float32 -> (out, lse)."""
    x = torch.where(seen, q @ k.transpose(-1, -2) * q.shape[-1] ** -0.5, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    z = p.sum(-1, keepdim=True)
    return (p / z) @ v, (top + torch.log(z)).squeeze(-1)


def _attn_plain(s):
    c = s["case"]
    H, D, G = c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    length, add = _mix(c)
    out, lse, at = [], [], 0
    for i, (n, b) in enumerate(zip(length, add)):
        page = s["table"][i, :-(-n // PAGE)].long()
        k, v = ((s[x][page].view(F8).float() * s[x + "_scale"][page][:, :, None, None]).transpose(0, 1).flatten(1, 2)[:, :n]
                for x in "kv")
        pos = torch.arange(n, device=DEV)
        step = max(1, (1 << 30) // (c["Hq"] * n))
        for j in range(0, b, step):
            m = min(b - j, step)
            q = s["q"][at + j:at + j + m].float().unflatten(1, (H, G)).permute(1, 0, 2, 3).flatten(1, 2)
            p = n - b + j + torch.arange(m, device=DEV).repeat_interleave(G)[:, None]
            seen = pos <= p
            if c["window"]:
                seen &= pos > p - c["window"]
            o, l = _softmax_plain(q, k, v, seen)
            out.append(o.unflatten(1, (m, G)).transpose(0, 1).flatten(1, 2))
            lse.append(l.unflatten(1, (m, G)).transpose(0, 1).flatten(1, 2))
        at += b
    return {"out": torch.cat(out).to(torch.bfloat16), "lse": torch.cat(lse)}


def _select_plain(s, c, a, seq, seen):
    """Pages [t, H, k] of tokens a .. a + t of sequences seq that see `seen` positions."""
    H, D, k = c["Hkv"], c["D"], c["k"]
    pages = (seen + PAGE - 1) // PAGE
    most = s["table"].shape[1]
    x = s["q"][a:a + seq.shape[0]].unflatten(1, (H, -1)).double().sum(2).float()
    top = x.abs().amax(-1, keepdim=True) / torch.full((), 127.0, device=DEV)
    r = torch.where(top > 0, (x / top).round().clamp(-127, 127), 0)
    phys = s["table"][seq].long()                            # [t, most]
    dot = (s["mean"][phys].float() * r[:, None]).sum(-1)     # exact whole numbers
    score = dot * s["mean_scale"][phys]
    j = torch.arange(most, device=DEV)[None]
    score = torch.where(((j < 1) | (j >= pages[:, None] - 1))[:, :, None], math.inf, score)
    score = torch.where((j < pages[:, None])[:, :, None], score, -math.inf).transpose(1, 2)
    best = score.sort(dim=-1, descending=True, stable=True)[1][..., :k]
    best = torch.where(best < pages[:, None, None], best, most).sort(-1)[0]
    best = torch.where(best < most, best, -1)
    return torch.nn.functional.pad(best, (0, k - best.shape[-1]), value=-1)


def _sparse_plain(s):
    c = s["case"]
    H, D = c["Hkv"], c["D"]
    T, k = s["q"].shape[0], c["k"]
    start, length = s["start"].long(), s["length"].long()
    got = []
    step = max(1, min((1 << 29) // (H * k * PAGE * D), (1 << 29) // (H * s["table"].shape[1] * D)))
    for a in range(0, T, step):
        t = torch.arange(a, min(T, a + step), device=DEV)
        seq = torch.searchsorted(start[1:].contiguous(), t, right=True)
        seen = length[seq] - start[seq + 1] + t + 1
        pages = _select_plain(s, c, a, seq, seen)
        phys = torch.gather(s["table"][seq].long()[:, None].expand(-1, H, -1), 2, pages.clamp(min=0))
        head = torch.arange(H, device=DEV)[None, :, None]
        kk, vv = ((s[x][phys, head].view(F8).float() * s[x + "_scale"][phys, head][..., None, None]).flatten(2, 3) for x in "kv")
        pos = (pages[..., None] * PAGE + torch.arange(PAGE, device=DEV)).flatten(2)
        ok = ((pages >= 0).repeat_interleave(PAGE, 2) & (pos < seen[:, None, None]))[:, :, None]
        o, l = _softmax_plain(s["q"][t].float().unflatten(1, (H, -1)), kk, vv, ok)
        got.append((pages.to(torch.int32), (pages >= 0).sum(-1).to(torch.int32), o.flatten(1, 2).to(torch.bfloat16), l.flatten(1, 2)))
    return {n: torch.cat(v) for n, v in zip(("pages", "count", "out", "lse"), zip(*got))}


# ---- one pass ---------------------------------------------------------------------------------

def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"plan": _plan_plain, "append": _append_plain, "attn": _attn_plain, "sparse": _sparse_plain}[c["op"]](s)
    from fp4_compressed_sparse_02_gb300 import csa2
    if c["op"] == "plan":
        p = csa2.page_plan(s["length"], s["add"], s["table"], s["free"], s["head"], c["cap"])
        return {"start": p.start, "seq": p.seq, "pos": p.pos, "slot": p.slot, "length": p.length, "head": p.head,
                "table": s["table"]}
    cache = csa2.Kv8Cache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s.get("mean"), s.get("mean_scale"))
    if c["op"] == "append":
        csa2.kv8_append(cache, s["x"], s["y"], s["start"], s["length"])
        return _append_outputs(s)
    if c["op"] == "attn":
        out, lse = csa2.kv8_attn(cache, s["q"], s["start"], s["length"], max_new=c["new"], window=c["window"])
        return {"out": out, "lse": lse}
    pages, count = csa2.kv8_select(cache, s["q"], s["start"], s["length"], c["k"])
    out, lse = csa2.kv8_attn(cache, s["q"], s["start"], s["length"], pages=pages)
    return {"pages": pages, "count": count, "out": out, "lse": lse}


# ---- 64 bits ----------------------------------------------------------------------------------

def _exact_rows(s, name, ids, heads):
    """float64 rows [.., 64, D] of pages `ids`, heads `heads`: the bytes taken apart by hand."""
    b = s[name][ids, heads].long()
    e, m = b // 8 % 16, (b % 8).double()
    x = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
    return x * (1 - 2.0 * (b // 128)) * s[name + "_scale"][ids, heads].double()[..., None, None]


def _exact_attn(q, k, v, hidden):
    x = torch.einsum("gd,nd->gn", q, k) / math.sqrt(q.shape[-1])
    x = x.masked_fill(hidden, -math.inf)
    l = torch.logsumexp(x, -1)
    return torch.exp(x - l[:, None]) @ v, l


def _exact_pages(s, i, t, h, n):
    """The kept pages of one token and key head, from whole numbers and one rounding."""
    c = s["case"]
    G, k, P = c["Hq"] // c["Hkv"], c["k"], -(-n // PAGE)
    if P <= k:
        return torch.arange(P, device=DEV)
    x = s["q"][t, h * G:(h + 1) * G].double().sum(0).float()
    a = x.abs().max() / torch.full((), 127.0, device=DEV)
    r = torch.round(x / a).double() if float(a) > 0 else torch.zeros_like(x).double()
    mid = torch.arange(1, P - 1, device=DEV)
    ids = s["table"][i, mid].long()
    score = ((s["mean"][ids, h].double() @ r) * s["mean_scale"][ids, h].double()).float()
    order = torch.argsort(-score, stable=True)[:k - 2]
    return torch.cat((mid[order].sort()[0], mid.new_tensor([0, P - 1]))).sort()[0]


def _to_e4m3(v):
    """The nearest E4M3 value (ties to even), saturating, in float64."""
    m = v.abs().clamp(max=448)
    step = torch.exp2(torch.floor(torch.log2(m.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign((m / step).round() * step, v)


def _exact_append(s, length, add):
    """Page by page: the new scale from a logarithm, old rows moved to it, new rows rounded once."""
    out = {x: s[x].view(F8).double() for x in "kv"} | {x + "_scale": s[x + "_scale"].double() for x in "kv"}
    out |= {"mean": None, "mean_scale": s["mean_scale"].double()}
    at = 0
    for i, (n, b) in enumerate(zip(length, add)):
        p = n - b
        while p < n:
            a, e = p % PAGE, min(PAGE, n - p + p % PAGE)
            page = int(s["table"][i, p // PAGE])
            for x, name in ((s["x"], "k"), (s["y"], "v")):
                r = x[at:at + e - a].double().transpose(0, 1)                      # [H, new, D]
                top = r.abs().amax((1, 2)).clamp(min=2.0 ** -1000)
                sc = torch.exp2(torch.round(torch.log2(top / 448)).clamp(min=-126))
                sc = torch.where(448 * sc < top, 2 * sc, sc)
                was = out[name + "_scale"][page]
                new = torch.maximum(sc, was) if a else sc
                if a:
                    out[name][page, :, :a] = _to_e4m3(out[name][page, :, :a] * (was / new)[:, None, None])
                out[name][page, :, a:e] = _to_e4m3(r / new[:, None, None])
                out[name + "_scale"][page] = new
            if e == PAGE:
                out["mean_scale"][page] = out["k"][page].sum(1).abs().amax(-1) / 127 / 64 * out["k_scale"][page]
            at, p = at + e - a, p + e - a
    return out


def exact(case, seed):
    c = dict(case)
    length, add = _mix(c)
    if c["op"] == "plan":
        return None                                          # whole numbers
    if c["op"] == "append":
        return _exact_append(prepare(case, seed), length, add)
    T, H, G = sum(add), c["Hkv"], c["Hq"] // c["Hkv"]
    sparse = c["op"] == "sparse"
    if sparse and T * H > 4096 or (not sparse and sum(b * n for n, b in zip(length, add)) * c["Hq"] * c["D"] > 2e12):
        return None
    s = prepare(case, seed)
    out = torch.empty((T, c["Hq"], c["D"]), dtype=torch.float64, device=DEV)
    lse = torch.empty((T, c["Hq"]), dtype=torch.float64, device=DEV)
    at = 0
    for i, (n, b) in enumerate(zip(length, add)):
        for h in range(H):
            if sparse:
                for j in range(b):
                    seen = n - b + j + 1
                    pages = _exact_pages(s, i, at + j, h, seen)
                    ids = s["table"][i, pages].long()
                    pos = (pages[:, None] * PAGE + torch.arange(PAGE, device=DEV)).flatten()
                    k, v = (_exact_rows(s, x, ids, h).flatten(0, 1) for x in "kv")
                    rows = slice(h * G, (h + 1) * G)
                    out[at + j, rows], lse[at + j, rows] = _exact_attn(s["q"][at + j, rows].double(), k, v, pos >= seen)
            elif b:
                ids = s["table"][i, :-(-n // PAGE)].long()
                k, v = (_exact_rows(s, x, ids, h).flatten(0, 1)[:n] for x in "kv")
                pos = torch.arange(n, device=DEV)[None]
                for j in range(0, b, 256):
                    m = min(256, b - j)
                    p = (n - b + j + torch.arange(m, device=DEV)).repeat_interleave(G)[:, None]
                    hidden = (pos > p) | (pos <= p - (c["window"] or n + 1))
                    rows = slice(h * G, (h + 1) * G)
                    o, l = _exact_attn(s["q"][at + j:at + j + m, rows].double().flatten(0, 1), k, v, hidden)
                    out[at + j:at + j + m, rows], lse[at + j:at + j + m, rows] = o.unflatten(0, (m, G)), l.unflatten(0, (m, G))
        at += b
    none = {"pages": None, "count": None} if sparse else {}
    return {**none, "out": out, "lse": lse}
