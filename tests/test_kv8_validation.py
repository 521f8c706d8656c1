"""Refusals of the paged 8-bit cache's calls on CPU (a valid argument struct with one field changed, fake addresses
that are never read), its Python checks, and the pins of the oracle they are tested against."""
import ctypes
import math

import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import _lib, build, csa2
from oracle import kv8
from oracle.formats import e4m3_value
from test_devices import OnDevice, machine  # noqa: F401

P, U = 0x10000, 0x10002           # aligned and 2-byte aligned fake device addresses
INVALID, SHAPE = 1, 2


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


CACHE = dict(k=P, v=P, k_scale=P, v_scale=P, mean=P, mean_scale=P, page_table=P, num_pages=8, page_size=64, num_seqs=2,
             max_pages=4, Hkv=2, D=128)


def make(cls, kw, **base):
    a = cls()
    a.struct_size = ctypes.sizeof(a)
    values = {**base, **kw}
    if hasattr(a, "cache"):
        values = {**{"c_" + n: v for n, v in CACHE.items()}, **values}
    for n, v in values.items():
        setattr(a.cache if n.startswith("c_") else a, n[2:] if n.startswith("c_") else n, v)
    return a


def plan(**kw):
    return make(_lib.PagePlanArgs, kw, S=2, max_pages=4, tokens=8, num_free=3, length=P, add=P, free_pages=P, free_head=P,
                page_table=P, start=P, seq=P, pos=P, slot=P, new_length=P, new_head=P)


ROWS = dict(T=4, S=2, start=P, length=P)


def append(**kw):
    return make(_lib.Kv8AppendArgs, kw, k=P, v=P, k_stride_t=256, k_stride_h=128, v_stride_t=256, v_stride_h=128, **ROWS)


def select(**kw):
    return make(_lib.Kv8SelectArgs, kw, Hq=8, k=8, first=1, recent=1, max_length=256, q=P, q_stride_t=1024, q_stride_h=128,
                pages=P, count=P, **ROWS)


def attn(**kw):
    return make(_lib.Kv8AttnArgs, kw, Hq=8, max_new=4, window=0, softmax_scale=0.1, q=P, q_stride_t=1024, q_stride_h=128, out=P,
                lse=P, **ROWS)


COMMON = [(dict(struct_size=8), INVALID, b"struct_size"), (dict(c_page_size=32), SHAPE, b"page_size"), (dict(c_num_pages=0), INVALID, b"num_pages"),
          (dict(c_num_pages=(1 << 25) + 1), SHAPE, b"num_pages"), (dict(c_max_pages=(1 << 24) + 1), SHAPE, b"max_pages"),
          (dict(c_max_pages=0), INVALID, b"max_pages"), (dict(c_D=96), SHAPE, b"D must"), (dict(c_Hkv=0), SHAPE, b"Hkv"),
          (dict(c_Hkv=257), SHAPE, b"Hkv"), (dict(S=3), INVALID, b"S must"), (dict(S=-1), INVALID, b"S must"), (dict(T=-1), INVALID, b"T must"),
          (dict(c_page_table=None), INVALID, b"page_table"), (dict(c_mean_scale=None), INVALID, b"go together"),
          (dict(c_mean=P + 8), INVALID, b"16-byte"), (dict(start=None), INVALID, b"start"), (dict(length=U), INVALID, b"length")]
PLANES = [(dict(c_k=None), INVALID, b"NULL"), (dict(c_v=P + 8), INVALID, b"16-byte"), (dict(c_v_scale=None), INVALID, b"NULL"),
          (dict(c_k_scale=U), INVALID, b"aligned")]
QUERY = [(dict(Hq=7), SHAPE, b"Hq"), (dict(Hq=0), SHAPE, b"Hq"), (dict(Hq=2 * 129), SHAPE, b"Hq"), (dict(q=None), INVALID, b"q is"),
         (dict(q=P + 1), INVALID, b"q is")]
CASES = [
    ("csa2_page_plan", plan, [
        (dict(struct_size=8), INVALID, b"struct_size"), (dict(S=-1), SHAPE, b"S must"), (dict(S=(1 << 20) + 1), SHAPE, b"S must"),
        (dict(tokens=-1), SHAPE, b"tokens"), (dict(max_pages=0), SHAPE, b"max_pages"), (dict(num_free=-1), INVALID, b"num_free"),
        (dict(start=None), INVALID, b"start"), (dict(new_head=None), INVALID, b"new_head"), (dict(add=None), INVALID, b"add"),
        (dict(page_table=None), INVALID, b"page_table"), (dict(free_pages=None), INVALID, b"free_pages"), (dict(slot=None), INVALID, b"slot"),
        (dict(pos=U), INVALID, b"aligned"), (dict(length=U), INVALID, b"aligned")]),
    ("csa2_kv8_append", append, COMMON + PLANES + [
        (dict(x_dtype=2), INVALID, b"x_dtype"), (dict(k=None), INVALID, b"k/v"), (dict(v=P + 1), INVALID, b"k/v"),
        (dict(k=U, x_dtype=1), INVALID, b"k/v")]),
    ("csa2_kv8_select", select, COMMON + QUERY + [
        (dict(c_mean=None, c_mean_scale=None), INVALID, b"summaries"), (dict(k=1), SHAPE, b"k must"), (dict(k=4097), SHAPE, b"k must"),
        (dict(first=-1), INVALID, b"first"), (dict(recent=0), INVALID, b"recent"), (dict(first=8), INVALID, b"first"),
        (dict(recent=8), INVALID, b"first"), (dict(max_length=-1), SHAPE, b"max_length"), (dict(max_length=(1 << 21) + 1), SHAPE, b"max_length"),
        (dict(pages=None), INVALID, b"pages"), (dict(count=U), INVALID, b"pages/count")]),
    ("csa2_kv8_attn", attn, COMMON + PLANES + QUERY + [
        (dict(max_new=-1), INVALID, b"max_new"), (dict(window=-1), INVALID, b"window"), (dict(softmax_scale=0.0), INVALID, b"softmax_scale"),
        (dict(softmax_scale=math.nan), INVALID, b"softmax_scale"), (dict(out_dtype=2), INVALID, b"out_dtype"), (dict(out=None), INVALID, b"out is"),
        (dict(out=U, out_dtype=1), INVALID, b"out is"), (dict(pages=P, list_len=0), SHAPE, b"list_len"), (dict(pages=P, list_len=4097), SHAPE, b"list_len"),
        (dict(pages=U, list_len=4), INVALID, b"pages"), (dict(lse=U), INVALID, b"pages/lse")]),
]
WITH_WS = {"csa2_kv8_select", "csa2_kv8_attn"}


@pytest.mark.parametrize("fn,base,kw,status,text", [(f, b, *c) for f, b, cs in CASES for c in cs])
def test_refused(L, fn, base, kw, status, text):
    a = base(**kw)
    more = (None, 0) if fn in WITH_WS else ()
    assert getattr(L, fn)(ctypes.byref(a), *more, None) == status
    assert text in L.csa2_last_error_message()
    if fn in WITH_WS:
        n = ctypes.c_size_t(0)
        assert getattr(L, fn + "_workspace")(ctypes.byref(a), ctypes.byref(n)) == status


@pytest.mark.parametrize("fn,base", [(f, b) for f, b, _ in CASES])
def test_null_struct_refused(L, fn, base):
    assert getattr(L, fn)(None, *((None, 0) if fn in WITH_WS else ()), None) == INVALID


@pytest.mark.parametrize("fn,base", [(f, b) for f, b, _ in CASES if f in WITH_WS])
def test_workspace_size_and_refusal(L, fn, base):
    n = ctypes.c_size_t(0)
    assert getattr(L, fn + "_workspace")(ctypes.byref(base()), ctypes.byref(n)) == 0
    assert getattr(L, fn + "_workspace")(ctypes.byref(base()), None) == INVALID
    if n.value:
        assert getattr(L, fn)(ctypes.byref(base()), P, n.value - 1, None) == 3
        assert getattr(L, fn)(ctypes.byref(base()), P + 128, n.value, None) == INVALID
        assert getattr(L, fn)(ctypes.byref(base()), None, n.value, None) == INVALID


def test_exports(L):
    assert all(hasattr(L, n) for n in _lib.EXPORTS)


# ---- the Python face --------------------------------------------------------------------------------

B16, F32, U8, I8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int8, torch.int32


def cache(t, means=True):
    m = (t("mean", I8, 9, 2, 64), t("mean_scale", F32, 9, 2)) if means else (None, None)
    return csa2.Kv8Cache(t("k_plane", U8, 9, 2, 64, 64), t("v_plane", U8, 9, 2, 64, 64), t("k_scale", F32, 9, 2),
                         t("v_scale", F32, 9, 2), t("page_table", I32, 3, 4), *m)


def ws(t):
    w = csa2.Workspace("cpu")
    w.get = lambda nbytes: t("workspace", U8, 256)
    return w


def plan_out(t):
    return csa2.PagePlan(t("start", I32, 4), t("seq", I32, 8), t("pos", I32, 8), t("slot", I32, 8), t("new_length", I32, 3), t("new_head", I32, 1))


CALLS = {
    "page_plan": (lambda t: csa2.page_plan(t("length", I32, 3), t("add", I32, 3), t("page_table", I32, 3, 4), t("free_pages", I32, 5),
                                           t("free_head", I32, 1), 8, out=plan_out(t)),
                  ["add", "page_table", "free_pages", "free_head", "start", "seq", "pos", "slot", "new_length", "new_head"]),
    "kv8_append": (lambda t: csa2.kv8_append(cache(t), t("k", B16, 5, 2, 64), t("v", B16, 5, 2, 64), t("start", I32, 4), t("length", I32, 3)),
                   ["v", "start", "length"]),
    "kv8_select": (lambda t: csa2.kv8_select(cache(t), t("q", B16, 5, 6, 64), t("start", I32, 4), t("length", I32, 3), 4,
                                             out=(t("pages", I32, 5, 2, 4), t("count", I32, 5, 2)), ws=ws(t)), ["start", "length", "pages", "count"]),
    "kv8_attn": (lambda t: csa2.kv8_attn(cache(t), t("q", B16, 5, 6, 64), t("start", I32, 4), t("length", I32, 3), pages=t("pages", I32, 5, 2, 4),
                                         out=t("out", B16, 5, 6, 64), lse=t("lse", F32, 5, 6), ws=ws(t)),
                 ["start", "length", "pages", "out", "lse"]),
}
PLANE_NAMES = ["k_plane", "v_plane", "k_scale", "v_scale", "page_table", "mean", "mean_scale"]


def call(name, dev, moved=None):
    return CALLS[name][0](lambda n, dtype, *shape: OnDevice(1 - dev if n == moved else dev, dtype, *shape))


@pytest.mark.parametrize("dev", [0, 1])
@pytest.mark.parametrize("name", CALLS)
def test_runs_on_its_tensors_device(machine, name, dev):  # noqa: F811
    call(name, dev)
    assert [(d, s) for _, d, s in machine] == [(dev, 100 + dev)]
    assert torch._C._cuda_getDevice() == 0


@pytest.mark.parametrize("name,moved", [(n, o) for n, (_, named) in CALLS.items() for o in named + (PLANE_NAMES if n != "page_plan" else [])])
def test_refuses_operands_of_another_device(machine, name, moved):  # noqa: F811
    with pytest.raises(ValueError, match="cuda:1"):
        call(name, 0, moved)
    assert machine == []


def cpu_cache(H=2, D=64, means=True):
    return csa2.Kv8Cache.allocate(4, H, D, torch.zeros((2, 3), dtype=I32), means)


@pytest.mark.parametrize("text,fn", [
    ("CUDA", lambda: csa2.page_plan(*(torch.zeros(n, dtype=I32) for n in (2, 2)), torch.zeros((2, 3), dtype=I32), torch.zeros(4, dtype=I32),
                                    torch.zeros(1, dtype=I32), 4)),
    ("length and add", lambda: csa2.page_plan(torch.zeros(2), torch.zeros(3), torch.zeros((2, 3)), torch.zeros(4), torch.zeros(1), 4)),
    ("heads and channels", lambda: csa2.kv8_append(cpu_cache(), torch.zeros((5, 3, 64)), torch.zeros((5, 3, 64)), None, None)),
    ("heads and channels", lambda: csa2.kv8_append(cpu_cache(), torch.zeros((5, 2, 64)), torch.zeros((4, 2, 64)), None, None)),
    ("one type", lambda: csa2.kv8_append(cpu_cache(), torch.zeros((5, 2, 64)), torch.zeros((5, 2, 64)).bfloat16(), None, None)),
    ("start must", lambda: csa2.kv8_append(cpu_cache(), torch.zeros((5, 2, 64)), torch.zeros((5, 2, 64)), torch.zeros(2), torch.zeros(2))),
    ("start must", lambda: csa2.kv8_append(cpu_cache(), torch.zeros((5, 2, 64)), torch.zeros((5, 2, 64)), torch.zeros(4), torch.zeros(3))),
    ("channels", lambda: csa2.kv8_attn(cpu_cache(), torch.zeros((5, 4, 128)).bfloat16(), None, None)),
    ("dtype", lambda: csa2.kv8_attn(cpu_cache(), torch.zeros((5, 4, 64)), None, None)),
    ("pages must", lambda: csa2.kv8_attn(cpu_cache(), torch.zeros((5, 4, 64)).bfloat16(), None, None, pages=torch.zeros((5, 4, 3)))),
    ("out must", lambda: csa2.kv8_attn(cpu_cache(), torch.zeros((5, 4, 64)).bfloat16(), None, None, out=torch.zeros((5, 4, 65)))),
    ("lse must", lambda: csa2.kv8_attn(cpu_cache(), torch.zeros((5, 4, 64)).bfloat16(), None, None, lse=torch.zeros((5, 3)))),
    ("out must", lambda: csa2.kv8_select(cpu_cache(), torch.zeros((5, 4, 64)).bfloat16(), None, None, 4, out=(torch.zeros(1), torch.zeros(1)))),
    ("CUDA", lambda: csa2.kv8_select(cpu_cache(), torch.zeros((5, 4, 64)).bfloat16(), torch.zeros(3, dtype=I32), torch.zeros(2, dtype=I32), 4)),
])
def test_python_refusals(text, fn):
    with pytest.raises((ValueError, TypeError), match=text):
        fn()


# ---- pins of the oracle -----------------------------------------------------------------------------

def test_power_for_borders():
    for a, want in [(0.0, 2.0 ** -126), (448.0, 1.0), (448.5, 2.0), (1.75, 2.0 ** -8), (np.nextafter(np.float32(1.75), np.float32(2)), 2.0 ** -7),
                    (3.4e38, 2.0 ** 120), (1e-45, 2.0 ** -126)]:
        s = kv8.power_for(float(a))
        assert s == want and a <= 448 * s


def test_sums_of_a_page_are_exact_in_float32():
    """64 E4M3 values are whole multiples of 2^-9 whose sum stays below 2^24 of them."""
    assert 64 * 448 * 512 < 2 ** 24
    v = e4m3_value(np.arange(0x7F))
    assert (v * 512 == np.rint(v * 512)).all()


def test_append_token_by_token_holds_what_one_step_holds_when_scales_agree():
    r = np.random.default_rng(0)
    x = r.uniform(1, 2, (130, 1, 64)).astype(np.float32)      # every magnitude needs the same scale but the last binade
    x[:, 0, 0] = 1.99
    new = lambda: {"k": np.zeros((3, 1, 64, 64), np.uint8), "v": np.zeros((3, 1, 64, 64), np.uint8), "k_scale": np.zeros((3, 1), np.float32),
                   "v_scale": np.zeros((3, 1), np.float32), "mean": np.zeros((3, 1, 64), np.int8), "mean_scale": np.zeros((3, 1), np.float32),
                   "table": np.array([[2, 0, 1]])}
    a, b = new(), new()
    kv8.append(a, x, -x, [0, 130], [130])
    for t in range(130):
        kv8.append(b, x[t:t + 1], -x[t:t + 1], [0, 1], [t + 1])
    assert all((a[n] == b[n]).all() for n in a)


def test_a_grown_scale_keeps_old_values_within_one_rounding():
    r = np.random.default_rng(1)
    c = {"k": np.zeros((1, 1, 64, 64), np.uint8), "v": np.zeros((1, 1, 64, 64), np.uint8), "k_scale": np.zeros((1, 1), np.float32),
         "v_scale": np.zeros((1, 1), np.float32), "mean": None, "table": np.array([[0]])}
    x = r.standard_normal((2, 1, 64)).astype(np.float32)
    x[1] *= 16
    kv8.append(c, x[:1], x[:1], [0, 1], [1])
    before = e4m3_value(c["k"][0, 0, 0]) * c["k_scale"][0, 0]
    kv8.append(c, x[1:], x[1:], [0, 1], [2])
    after, s = e4m3_value(c["k"][0, 0, 0]) * c["k_scale"][0, 0], float(c["k_scale"][0, 0])
    assert (np.abs(after - before) <= np.maximum(2.0 ** -4 * np.abs(before), 2.0 ** -10 * s)).all()


def test_attend_over_one_row_returns_it():
    v = np.arange(64.0)[None]
    out, lse, _ = kv8.attend(np.ones(64), np.ones((1, 64)), v, np.array([True]), 0.5)
    assert (out == v[0]).all() and lse == 32.0
    assert kv8.attend(np.ones(64), np.ones((1, 64)), v, np.array([False]), 0.5)[1] == -np.inf


def test_select_keeps_the_best_middle_pages():
    c = {"k": np.zeros((9, 1, 64, 64), np.uint8), "mean": np.zeros((9, 1, 64), np.int8), "mean_scale": np.ones((9, 1), np.float32),
         "table": np.arange(9)[None]}
    c["mean"][[3, 5, 6], 0, 0] = [10, 90, 90]
    q = np.zeros((2, 64), np.float32)
    q[:, 0] = 1
    assert kv8.select(c, q, 0, 9 * 64, 4, 1, 1) == [[0, 5, 6, 8]]
    assert kv8.select(c, q, 0, 9 * 64, 3, 1, 1) == [[0, 5, 8]]          # equal scores: the older page
    assert kv8.select(c, -q, 0, 8 * 64 + 1, 4, 1, 1) == [[0, 1, 2, 8]]
    assert kv8.select(c, q, 0, 3 * 64, 4, 1, 1) == [[0, 1, 2]]


def test_workspace_keeps_what_graphs_hold(monkeypatch):
    capturing = [False]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    w = csa2.Workspace("cpu")
    a = w.get(10)
    b = w.get(20)
    assert w.outgrown == [] and b.numel() == 20 and a is not b
    capturing[0] = True
    assert w.get(15) is b
    with pytest.raises(RuntimeError, match="sized before"):
        w.get(21)
    capturing[0] = False
    w.get(30)
    w.get(40)
    assert [x.numel() for x in w.outgrown] == [20]
