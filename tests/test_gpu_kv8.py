"""The paged 8-bit cache on the GPU against the NumPy oracle: tables and appended bytes bit for bit, page lists
exactly, attention within the stated precision."""
import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2
from kv8_utils import DEV, bf16, check_attn, check_cache, fill, gpu, new_cache, starts, strided, to_gpu
from oracle import kv8

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(autouse=True)
def no_device_error(request):
    if "raises" not in request.node.name:
        csa2.device_error()
    yield
    if "raises" not in request.node.name:
        assert csa2.device_error() == 0


# ---- page_plan ------------------------------------------------------------------------------------

def run_plan(length, add, most, free, head, tokens, table, err=0):
    S = len(length)
    want_table = table.copy()
    want = kv8.plan(length, add, want_table, free, head, tokens)
    g = [gpu(np.asarray(x, np.int32)) for x in (length, add, table, free, [head])]
    p = csa2.page_plan(*g, tokens)
    assert csa2.device_error() == err
    for x in ("start", "seq", "pos", "slot", "length", "head"):
        got = getattr(p, x).cpu().numpy()
        assert (got == want[x]).all(), (x, got, want[x])
    assert (g[2].cpu().numpy() == want_table).all()
    return p


def held_table(r, length, most, P):
    table = np.full((len(length), most), -1, np.int32)
    ids = r.permutation(P).astype(np.int32)
    at = 0
    for s, n in enumerate(length):
        m = -(-n // 64)
        table[s, :m] = ids[at:at + m]
        at += m
    return table, ids[at:]


@pytest.mark.parametrize("S,longest,new,spare", [(1, 0, 1, 0), (1, 63, 1, 0), (1, 64, 130, 3), (7, 200, 1, 0), (33, 500, 90, 5),
                                                 (1024, 100, 3, 0), (1025, 100, 7, 9), (3000, 130, 2, 1), (5, 4000, 9000, 0)])
def test_plan(S, longest, new, spare):
    r = np.random.default_rng(S + longest)
    length = r.integers(0, longest + 1, S)
    add = r.integers(0, new + 1, S) * (r.random(S) < 0.8)
    most = (longest + new) // 64 + 2
    table, free = held_table(r, length, most, S * most)
    run_plan(length, add, most, free, 2, int(add.sum()) + spare, table)


def test_plan_empty_and_no_rows():
    run_plan([5, 64, 0], [0, 0, 0], 4, np.arange(3), 0, 7, np.zeros((3, 4), np.int32))
    run_plan([5], [0], 4, np.zeros(0), 0, 0, np.zeros((1, 4), np.int32))


def test_plan_free_pages_run_out_raises():
    r = np.random.default_rng(1)
    length, add = np.array([60, 0, 128]), np.array([200, 65, 64])
    table, free = held_table(r, length, 8, 50)
    csa2.device_error()
    run_plan(length, add, 8, free[:5], 1, 400, table, err=0x200)


def test_plan_rows_or_table_run_out_raises():
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    csa2.device_error()
    run_plan([250, 0, 3], [10, 20, 30], 4, np.arange(100, 120), 0, 30, table, err=0x400)      # 6 + 20 + 4 rows
    run_plan([300, 256, 3], [10, 20, 1], 4, np.arange(100, 120), 0, 30, table, err=0x400)     # a row longer than its table


def test_plan_negative_counts_raises():
    csa2.device_error()
    run_plan([-5, 10], [3, -2], 4, np.arange(9), 0, 8, np.zeros((2, 4), np.int32), err=0x4)


@pytest.mark.parametrize("tokens,new", [(60, 3), (4096, 30), (4097, 30)])
def test_plan_advances_its_own_state_in_a_graph(tokens, new):
    """Captured once, replayed: lengths, table and free list advance as step by step."""
    r = np.random.default_rng(3)
    S, most = 37, 6
    length, add = r.integers(0, 130, S), r.integers(0, new, S)
    table, free = held_table(r, length, most, S * most)
    g = dict(length=gpu(length.astype(np.int32)), add=gpu(add.astype(np.int32)), table=gpu(table), free=gpu(free), head=gpu(np.zeros(1, np.int32)))
    out = csa2.PagePlan.allocate(S, tokens, DEV)
    out.length, out.head = g["length"], g["head"]
    step = lambda: csa2.page_plan(g["length"], g["add"], g["table"], g["free"], g["head"], tokens, out=out)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    head = 0
    for _ in range(4):
        graph.replay()
        want = kv8.plan(length, add, table, free, head, tokens)
        length, head = want["length"], want["head"]
        for x in ("start", "seq", "pos", "slot", "length", "head"):
            assert (getattr(out, x).cpu().numpy() == want[x]).all(), x
        assert (g["table"].cpu().numpy() == table).all()


# ---- kv8_append -----------------------------------------------------------------------------------

def append_both(c, g, k, v, start, length, dtype, pad=0):
    kv8.append(c, k, v, start, length)
    csa2.kv8_append(g, strided(k, dtype, pad), strided(v, dtype, pad), gpu(start), gpu(np.asarray(length, np.int32)))


@pytest.mark.parametrize("H,D", [(1, 128), (3, 64), (8, 128)])
@pytest.mark.parametrize("dtype,pad", [(torch.bfloat16, 0), (torch.bfloat16, 8), (torch.float32, 4), (torch.bfloat16, 1), (torch.float32, 1)])
def test_append_steps(H, D, dtype, pad):
    """Several ragged steps: fresh pages, part-filled ones whose scale grows, full ones, idle sequences."""
    r = np.random.default_rng(H * D + pad)
    c = new_cache(r, 5, 6, H, D)
    g = to_gpu(c)
    length = np.zeros(5, np.int64)
    for step, add in enumerate([(1, 64, 63, 0, 130), (1, 1, 1, 5, 0), (70, 0, 1, 59, 62), (1, 128, 0, 1, 1)]):
        length = length + add
        T = sum(add)
        mk = lambda: r.standard_normal((T, H, D)) * np.exp2(r.integers(-8, 9, (T, 1, 1)) + 4 * step)
        x = [mk().astype(np.float32) if dtype is torch.float32 else bf16(mk()) for _ in range(2)]
        append_both(c, g, x[0], x[1], starts(add), length, dtype, pad)
        check_cache(g, c)


def test_append_values():
    """Zero pages, infinities, NaN, the borders of the scale, the largest and smallest magnitudes."""
    r = np.random.default_rng(0)
    c = new_cache(r, 8, 1, 2, 64)
    x = np.zeros((8, 64, 2, 64), np.float32)
    x[1] = bf16(r.standard_normal((64, 2, 64)))
    x[1, 5, 0, 3], x[1, 9, 1, 7], x[1, 10, 0, 0] = np.inf, -np.inf, np.nan
    x[2, :, :, 0] = 1.75                                     # 448 x a power of two exactly
    x[3, :, :, 0] = 1.7578125                                # the bf16 above it
    x[4] = bf16(3.38e38 * np.sign(r.standard_normal((64, 2, 64))))
    x[5] = bf16(1e-38 * r.standard_normal((64, 2, 64)))
    x[6] = np.nan
    x[7] = np.float32(2.0 ** -133)
    g = to_gpu(c)
    add = np.full(8, 64)
    append_both(c, g, x.reshape(512, 2, 64), -x.reshape(512, 2, 64), starts(add), add, torch.bfloat16)
    check_cache(g, c)


def test_append_padding_rows_and_a_captured_step():
    """Rows before the first sequence and after the last are not touched; a captured step replays."""
    r = np.random.default_rng(5)
    c = new_cache(r, 3, 3, 2, 128)
    g = to_gpu(c)
    add = np.array([3, 0, 70])
    x = [np.full((90, 2, 128), np.nan, np.float32) for _ in range(2)]
    for y in x:
        y[7:80] = bf16(r.standard_normal((73, 2, 128)))
    start, length = starts(add, 7), add + [10, 5, 0]
    fill(r, c, [10, 5, 0])
    for n in ("k", "v", "k_scale", "v_scale", "mean", "mean_scale"):
        getattr(g, n).copy_(gpu(c[n]))
    args = [gpu(x[0], torch.bfloat16), gpu(x[1], torch.bfloat16), gpu(start), gpu(length.astype(np.int32))]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.kv8_append(g, *args)
    graph.replay()
    graph.replay()                                           # the same step again writes the same bytes
    sub = [y[7:80] for y in x]
    kv8.append(c, sub[0], sub[1], starts(add), length)
    check_cache(g, c)


def test_append_bad_page_raises():
    """A page id outside the cache is reported and its tokens are skipped; the others are written."""
    r = np.random.default_rng(6)
    c = new_cache(r, 3, 2, 1, 64)
    g = to_gpu(c)
    x = [bf16(r.standard_normal((30, 1, 64))) for _ in range(2)]
    start, length = starts([10, 10, 10]), np.full(3, 10)
    keep = {n: v.copy() for n, v in c.items()}
    kv8.append(c, x[0], x[1], start, length)
    bad = int(c["table"][1, 0])
    for n in ("k", "v", "k_scale", "v_scale"):
        c[n][bad] = keep[n][bad]
    g.page_table[1, 0] = c["k"].shape[0]
    csa2.device_error()
    csa2.kv8_append(g, gpu(x[0], torch.bfloat16), gpu(x[1], torch.bfloat16), gpu(start), gpu(length.astype(np.int32)))
    assert csa2.device_error() == 0x1
    check_cache(g, c)


# ---- kv8_select -----------------------------------------------------------------------------------

def run_select(c, g, q, start, length, k, first=1, recent=1, pad=0, **kw):
    T, H = q.shape[0], c["k"].shape[1]
    out = (torch.full((T, H, k), 12345, dtype=I32, device=DEV), torch.full((T, H), 12345, dtype=I32, device=DEV))
    pages, count = csa2.kv8_select(g, strided(q, torch.bfloat16, pad), gpu(start), gpu(np.asarray(length, np.int32)), k,
                                   first=first, recent=recent, out=out, **kw)
    got, num = pages.cpu().numpy(), count.cpu().numpy()
    for s in range(len(length)):
        for t in range(start[s], start[s + 1]):
            n = int(length[s] - (start[s + 1] - t) + 1)
            for h, want in enumerate(kv8.select(c, q[t], s, n, k, first, recent)):
                assert num[t, h] == len(want) and list(got[t, h]) == want + [-1] * (k - len(want)), (s, t, h)
    for t in [*range(start[0]), *range(start[-1], T)]:
        assert (got[t] == 12345).all() and (num[t] == 12345).all()
    return pages


@pytest.mark.parametrize("H,G,D,k,first,recent", [(1, 1, 64, 2, 1, 1), (2, 8, 128, 5, 1, 1), (3, 7, 128, 13, 0, 2), (2, 16, 64, 9, 3, 3),
                                                  (1, 64, 128, 6, 5, 1), (2, 4, 128, 4, 2, 2)])
def test_select(H, G, D, k, first, recent):
    r = np.random.default_rng(k * D + G)
    length, add = [1, 64, 65, 700, 1280, 1281, 900], [1, 3, 1, 5, 1, 2, 0]
    c = new_cache(r, 7, 21, H, D)
    fill(r, c, length)
    q = bf16(r.standard_normal((sum(add) + 6, H * G, D)) * np.exp2(r.integers(-6, 7, (sum(add) + 6, 1, 1))))
    run_select(c, to_gpu(c), q, starts(add, 2), length, k, first, recent, pad=8 if D == 64 else 1)


def test_select_ties_and_special_queries():
    """Pages alike (ties go to the older one), zero, infinite and NaN queries, zero pages."""
    r = np.random.default_rng(9)
    c = new_cache(r, 1, 40, 2, 64)
    fill(r, c, [64 * 40 - 7])
    ids = c["table"][0]
    for j in range(3, 30, 3):
        c["mean"][ids[j]], c["mean_scale"][ids[j]] = c["mean"][ids[2]], c["mean_scale"][ids[2]]
    for j in (5, 8, 11):
        c["mean"][ids[j]], c["mean_scale"][ids[j]] = 0, 0
    q = bf16(r.standard_normal((12, 6, 64)))
    q[0], q[1, 0, 0], q[2, 3, 5], q[3, :, 7] = 0, np.inf, np.nan, -np.inf
    run_select(c, to_gpu(c), q, starts([12]), [64 * 40 - 7], 12)


def test_select_long_table():
    """A million tokens: 16,384 pages of one sequence."""
    r = np.random.default_rng(2)
    n = 64 * 16384 - 5
    c = dict(k=np.zeros((16384, 1, 0, 64), np.uint8), table=r.permutation(16384).astype(np.int32)[None],
             mean=r.integers(-127, 128, (16384, 1, 64)).astype(np.int8),
             mean_scale=np.exp2(r.integers(-3, 3, (16384, 1))).astype(np.float32))
    plane = torch.zeros((16384, 1, 64, 64), dtype=torch.uint8, device=DEV)
    scale = torch.ones((16384, 1), device=DEV)
    g = csa2.Kv8Cache(plane, plane, scale, scale, gpu(c["table"]), gpu(c["mean"]), gpu(c["mean_scale"]))
    q = bf16(r.standard_normal((3, 4, 64)))
    run_select(c, g, q, starts([3]), [n], 512)
    run_select(c, g, q[:1], starts([1]), [n], 64)
    run_select(c, g, q[:1], starts([1]), [n], 4096, first=4, recent=4)


def test_select_length_beyond_its_bound_raises():
    r = np.random.default_rng(4)
    c = new_cache(r, 2, 10, 1, 64)
    fill(r, c, [600, 100])
    csa2.device_error()
    pages, count = csa2.kv8_select(to_gpu(c), gpu(bf16(r.standard_normal((2, 1, 64))), torch.bfloat16), gpu(starts([1, 1])),
                                   gpu(np.array([600, 100], np.int32)), 2, max_length=128)
    assert csa2.device_error() == 0x4
    assert pages.cpu().numpy().reshape(2, 2).tolist() == [[-1, -1], [0, 1]] and count.cpu().flatten().tolist() == [0, 2]


# ---- kv8_attn -------------------------------------------------------------------------------------

def run_attn(c, g, q, start, length, pad=0, dtype=torch.bfloat16, pages=None, window=0, scale=None, check=True, q_eps=0.0, **kw):
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), 777.0, dtype=dtype, device=DEV)
    lse = torch.full((T, Hq), 777.0, device=DEV)
    p = None if pages is None else gpu(np.asarray(pages, np.int32))
    csa2.kv8_attn(g, strided(q, torch.bfloat16, pad), gpu(start), gpu(np.asarray(length, np.int32)), pages=p, window=window,
                  softmax_scale=scale, out=out, lse=lse, **kw)
    rest = [*range(start[0]), *range(start[-1], T)]
    assert (out[rest] == 777).all() and (lse[rest] == 777).all()
    if check:
        check_attn(out, lse, c, q, start, length, scale or D ** -0.5, window, pages, 2.0 ** -24 if dtype is torch.float32 else 2.0 ** -8, q_eps)
    return out, lse


STEPS = {"token": ([1, 63, 64, 65, 700, 129], [1, 1, 1, 1, 1, 1]), "idle": ([300, 5, 128], [0, 1, 0]),
         "verify": ([6, 70, 200, 128], [6, 3, 1, 5]), "chunk": ([40, 333, 130], [40, 37, 0]), "one": ([1000], [1])}


@pytest.mark.parametrize("hint", [1, 8, 20, 100])
@pytest.mark.parametrize("H,G,D", [(2, 8, 128), (1, 1, 64), (3, 7, 64), (1, 16, 128), (2, 5, 128), (1, 20, 64), (1, 64, 128)])
@pytest.mark.parametrize("step", STEPS)
def test_attn(step, H, G, D, hint):
    length, add = STEPS[step]
    r = np.random.default_rng(G * D + len(length))
    c = new_cache(r, len(length), 17, H, D)
    fill(r, c, length)
    q = bf16(r.standard_normal((sum(add) + 3, H * G, D)) * 2)
    run_attn(c, to_gpu(c), q, starts(add, 1), length, pad=(0, 8, 1)[G % 3], dtype=torch.float32 if G == 5 else torch.bfloat16,
             max_new=hint)


@pytest.mark.parametrize("hint", [1, 8, 20, 100])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 100000])
def test_attn_window(window, hint):
    r = np.random.default_rng(window)
    length, add = [1, 64, 130, 705, 300], [1, 1, 7, 21, 0]
    c = new_cache(r, 5, 12, 2, 128)
    fill(r, c, length)
    q = bf16(r.standard_normal((sum(add), 6, 128)))
    run_attn(c, to_gpu(c), q, starts(add), length, window=window, max_new=hint)


@pytest.mark.parametrize("hint", [1, 8, 20, 100])
@pytest.mark.parametrize("window", [1, 65, 200])
def test_attn_window_with_its_old_pages_given_back(window, hint):
    """Table entries of pages behind the window are not looked at."""
    r = np.random.default_rng(window)
    length, add = [64, 130, 705, 321], [1, 7, 21, 1]
    c = new_cache(r, 4, 12, 2, 128)
    fill(r, c, length)
    for s in range(4):
        c["table"][s, :max(0, length[s] - add[s] + 1 - window) // 64] = -1
    q = bf16(r.standard_normal((sum(add), 6, 128)))
    run_attn(c, to_gpu(c), q, starts(add), length, window=window, max_new=hint)


def test_attn_without_a_hint():
    """The default takes the kernel that the step's rows allow for: the same bits as with the hint."""
    r = np.random.default_rng(5)
    c = new_cache(r, 3, 12, 2, 128)
    fill(r, c, [200, 64, 700])
    g, q = to_gpu(c), bf16(r.standard_normal((9, 16, 128)))
    for add in ([1, 1, 1], [3, 5, 1]):
        args = (c, g, q[:sum(add)], starts(add), [200, 64, 700])
        got, want = run_attn(*args), run_attn(*args, max_new=sum(add) - 2, check=False)
        assert all((a == b).all() for a, b in zip(got, want))


@pytest.mark.parametrize("H,G,D,n", [(2, 8, 128, 1), (1, 1, 64, 5), (3, 7, 64, 9), (1, 16, 128, 4), (1, 40, 128, 7), (2, 4, 128, 70)])
def test_attn_listed_pages(H, G, D, n):
    """Lists of other lengths, orders and with nothing in them; a page twice counts twice."""
    r = np.random.default_rng(G)
    length, add = [1, 65, 700, 640], [1, 2, 5, 1]
    c = new_cache(r, 4, 11, H, D)
    fill(r, c, length)
    T = sum(add)
    pages = np.full((T, H, n), -1)
    for t in range(T):
        for h in range(H):
            m = r.integers(0, n + 1)
            pages[t, h, r.permutation(n)[:m]] = r.integers(0, 11, m)
    pages[0] = -1                                            # an empty row
    q = bf16(r.standard_normal((T, H * G, D)))
    run_attn(c, to_gpu(c), q, starts(add), length, pages=pages)
    run_attn(c, to_gpu(c), q, starts(add), length, pages=pages, window=100)


@pytest.mark.parametrize("hint", [1, 3, 20, 40, 100])
def test_attn_nan_in_masked_places(hint):
    """A NaN key or value of the newest token reaches that token's row alone."""
    r = np.random.default_rng(11)
    length, add = [70, 200], [6, 40]
    c = new_cache(r, 2, 4, 2, 64)
    fill(r, c, length)
    for s, n in enumerate(length):
        page, slot = c["table"][s, (n - 1) // 64], (n - 1) % 64
        c["v"][page, 0, slot, 5] = 0x7F
        c["k"][page, 1, slot, 9] = 0xFF
    q = bf16(r.standard_normal((46, 6, 64)))
    run_attn(c, to_gpu(c), q, starts(add), length, max_new=hint)


@pytest.mark.parametrize("hint", [1, 2, 8, 16, 100])
def test_attn_scales_far_apart(hint):
    """Pages whose key and value scales differ by 2^12, queries of other magnitudes, equal keys."""
    r = np.random.default_rng(12)
    length, add = [300, 500], [3, 33]
    c = new_cache(r, 2, 8, 1, 128)
    fill(r, c, length)
    c["v_scale"][:] = np.exp2(r.integers(-9, 4, c["v_scale"].shape))
    c["k_scale"][:] = np.exp2(r.integers(-12, -7, c["k_scale"].shape))
    q = bf16(r.standard_normal((36, 8, 128)) * np.exp2(r.integers(-20, 4, (36, 8, 1))))
    q[0, 0] = 0
    run_attn(c, to_gpu(c), q, starts(add), length, max_new=hint, dtype=torch.float32)


@pytest.mark.parametrize("hint", [1, 2, 8, 16, 100])
def test_attn_queries_of_wide_range(hint):
    """Rows whose elements span 2^24, keys alike: every element counts.  Above 16 rows an element is off by at most 2^-17 of
    its row's largest."""
    r = np.random.default_rng(15)
    length, add = [200, 300], [3, 20]
    c = new_cache(r, 2, 5, 1, 128)
    fill(r, c, length)
    q = bf16(r.standard_normal((23, 8, 128)) * np.exp2(r.integers(-24, 1, (23, 8, 128))))
    q[0, 1] = 0
    q[1, 2, :100] = 0
    run_attn(c, to_gpu(c), q, starts(add), length, max_new=hint, dtype=torch.float32, q_eps=2.0 ** -17 if hint * 8 > 16 else 0.0)


@pytest.mark.parametrize("hint", [1, 3, 20, 100])
def test_attn_infinite_queries_reach_their_own_rows_alone(hint):
    r = np.random.default_rng(16)
    length, add = [150, 70], [4, 9]
    c = new_cache(r, 2, 3, 1, 64)
    fill(r, c, length)
    q = bf16(r.standard_normal((13, 6, 64)))
    g = to_gpu(c)
    want, _ = run_attn(c, g, q, starts(add), length, max_new=hint)
    q[2, 3, 5], q[7, 0, 1], q[9, 5, 63] = np.inf, np.nan, -np.inf
    out, lse = run_attn(c, g, q, starts(add), length, max_new=hint, check=False)
    bad = torch.zeros((13, 6), dtype=torch.bool, device=DEV)
    bad[2, 3] = bad[7, 0] = bad[9, 5] = True
    assert (out[~bad] == want[~bad]).all() and out[bad].isnan().all()


@pytest.mark.parametrize("hint", [1, 2, 8, 100])
@pytest.mark.parametrize("S", [33, 70, 2100])
def test_attn_many_sequences(S, hint):
    """More sequences than a warp looks at in one go, and more than the plan of the large tiles copies."""
    r = np.random.default_rng(S)
    length = r.integers(0, 100, S)
    add = np.minimum(length, r.integers(0, 3, S))
    c = new_cache(r, S, 2, 1, 64, spare=1)
    fill(r, c, length, spread=1)
    q = bf16(r.standard_normal((int(add.sum()), 4, 64)))
    run_attn(c, to_gpu(c), q, starts(add), length, max_new=hint)


@pytest.mark.parametrize("hint", [1, 100])
def test_attn_one_long_sequence(hint):
    """Many spans of one stream, and the same bits on a repeated call, on another stream and with a workspace of its own."""
    r = np.random.default_rng(17)
    n = 64 * 150 - 9
    c = new_cache(r, 1, 150, 1, 128, spare=0)
    fill(r, c, [n])
    g = to_gpu(c)
    q = bf16(r.standard_normal((3, 8, 128)))
    out, lse = run_attn(c, g, q, starts([3]), [n], max_new=hint)
    for _ in range(2):
        with torch.cuda.stream(torch.cuda.Stream()):
            a, b = run_attn(c, g, q, starts([3]), [n], max_new=hint, ws=csa2.Workspace(DEV), check=False)
            torch.cuda.current_stream().synchronize()
        assert (a == out).all() and (b == lse).all()


def test_calls_on_two_streams_at_once():
    """Default workspaces belong to a stream: interleaved calls do not disturb each other."""
    r = np.random.default_rng(18)
    sets = []
    for n in (3000, 5000):
        c = new_cache(r, 1, 90, 2, 64, spare=0)
        fill(r, c, [n])
        q = bf16(r.standard_normal((2, 16, 64)))
        sets.append((to_gpu(c), gpu(q, torch.bfloat16), gpu(starts([2])), gpu(np.array([n], np.int32)), torch.cuda.Stream()))
    alone = []
    for g, q, start, length, _ in sets:
        pages, _ = csa2.kv8_select(g, q, start, length, 9)
        alone.append((pages, *csa2.kv8_attn(g, q, start, length, max_new=1), *csa2.kv8_attn(g, q, start, length, pages=pages)))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (g, q, start, length, stream) in enumerate(sets):
            with torch.cuda.stream(stream):
                pages, _ = csa2.kv8_select(g, q, start, length, 9)
                got[i].append((pages, *csa2.kv8_attn(g, q, start, length, max_new=1), *csa2.kv8_attn(g, q, start, length, pages=pages)))
    torch.cuda.synchronize()
    for i in range(2):
        assert all((a == b).all() for run in got[i] for a, b in zip(run, alone[i]))
    graphs, held = [], []
    for g, q, start, length, _ in sets:                      # and so do graphs that are replayed side by side
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            pages, _ = csa2.kv8_select(g, q, start, length, 9)
            held.append((pages, *csa2.kv8_attn(g, q, start, length, max_new=1), *csa2.kv8_attn(g, q, start, length, pages=pages)))
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(sets[i][4]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all((a == b).all() for a, b in zip(held[i], alone[i]))


def test_a_graph_outlives_its_workspace_growing():
    """A workspace grows after a capture that used it: the graph still writes into memory of its own."""
    r = np.random.default_rng(19)
    c = new_cache(r, 1, 40, 1, 64, spare=0)
    fill(r, c, [2500])
    g = to_gpu(c)
    q = gpu(bf16(r.standard_normal((1, 8, 64))), torch.bfloat16)
    args = (g, q, gpu(starts([1])), gpu(np.array([2500], np.int32)))
    stream, ws = torch.cuda.Stream(), csa2.Workspace(DEV)
    with torch.cuda.stream(stream):
        want, _ = csa2.kv8_attn(*args, max_new=1, ws=ws)
        out = torch.zeros_like(want)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            csa2.kv8_attn(*args, max_new=1, out=out, ws=ws)
        csa2.kv8_attn(*args, max_new=100, ws=ws)             # needs more
        other = [torch.full((1 << 20,), 7, dtype=torch.uint8, device=DEV) for _ in range(64)]
        graph.replay()
        stream.synchronize()
    assert (out == want).all() and all((x == 7).all() for x in other)


def test_pages_beyond_32_bits():
    """Planes of 2.6 GB: the last pages, appended to, selected and attended to."""
    r = np.random.default_rng(20)
    H, D, P = 2, 128, 160000
    c = new_cache(r, 1, 12, H, D, spare=0)
    new = lambda dtype, *s: torch.empty((P, H) + s, dtype=dtype, device=DEV)
    far = c["table"].max() + 1
    table = gpu((c["table"] + (P - far)).astype(np.int32))
    g = csa2.Kv8Cache(new(torch.uint8, 64, D), new(torch.uint8, 64, D), new(torch.float32), new(torch.float32), table,
                      new(torch.int8, D), new(torch.float32))
    n = 12 * 64 - 5
    x = [bf16(r.standard_normal((n, H, D))) for _ in range(2)]
    kv8.append(c, x[0], x[1], starts([n]), [n])
    csa2.kv8_append(g, gpu(x[0], torch.bfloat16), gpu(x[1], torch.bfloat16), gpu(starts([n])), gpu(np.array([n], np.int32)))
    tail = csa2.Kv8Cache(*(getattr(g, f)[P - far:] for f in ("k", "v", "k_scale", "v_scale")), gpu(c["table"]), g.mean[P - far:], g.mean_scale[P - far:])
    ids = c["table"][0]
    for f in ("k", "v", "k_scale", "v_scale"):
        got, want = getattr(tail, f).cpu().numpy()[ids[:-1]], c[f][ids[:-1]]
        assert (got == want).all(), f
    q = bf16(r.standard_normal((2, 8, D)))
    pages = run_select(c, g, q, starts([2]), [n], 5)
    run_attn(c, g, q, starts([2]), [n], pages=pages.cpu().numpy())
    for hint in (1, 100):
        run_attn(c, g, q, starts([2]), [n], max_new=hint)


def test_empty_calls():
    r = np.random.default_rng(22)
    c = new_cache(r, 2, 2, 1, 64)
    fill(r, c, [70, 3])
    g = to_gpu(c)
    z = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)
    start, length = gpu(starts([0, 0])), gpu(np.array([70, 3], np.int32))
    csa2.kv8_append(g, z(0, 1, 64), z(0, 1, 64), start, length)
    assert csa2.kv8_select(g, z(0, 2, 64), start, length, 4)[0].shape == (0, 1, 4)
    assert csa2.kv8_attn(g, z(0, 2, 64), start, length)[0].shape == (0, 2, 64)
    csa2.kv8_append(g, z(5, 1, 64), z(5, 1, 64), start, length)        # rows of padding alone
    check_cache(g, c)
    run_attn(c, g, np.ones((5, 2, 64), np.float32), starts([0, 0]), [70, 3])
    none = torch.empty(0, dtype=I32, device=DEV)
    p = csa2.page_plan(none, none, torch.empty((0, 4), dtype=I32, device=DEV), none, gpu(np.zeros(1, np.int32)), 3)
    assert p.start.tolist() == [0] and p.seq.tolist() == p.slot.tolist() == [-1] * 3 and p.head.tolist() == [0]


def test_attn_bad_pages_raises():
    r = np.random.default_rng(13)
    c = new_cache(r, 2, 4, 1, 64)
    fill(r, c, [200, 130])
    g = to_gpu(c)
    q = bf16(r.standard_normal((2, 2, 64)))
    want, _ = run_attn(c, g, q, starts([1, 1]), [200, 130])
    g.page_table[0, 1] = -7
    csa2.device_error()
    out, _ = run_attn(c, g, q, starts([1, 1]), [200, 130], check=False)
    assert csa2.device_error() == 0x1 and (out[1] == want[1]).all() and out[0].isfinite().all()
    pages = np.array([[[0, 9, 2]], [[0, 1, 2]]])
    run_attn(c, g, q, starts([1, 1]), [200, 130], pages=pages, check=False)
    assert csa2.device_error() == 0x2


def test_attn_rows_shorter_than_their_tokens_raises():
    """length below the new tokens: the rows before the sequence's begin see nothing."""
    r = np.random.default_rng(14)
    c = new_cache(r, 1, 4, 1, 64)
    fill(r, c, [3])
    csa2.device_error()
    out, lse = run_attn(c, to_gpu(c), bf16(r.standard_normal((5, 2, 64))), starts([5]), [3], check=False)
    assert csa2.device_error() == 0x2
    assert (out[:2] == 0).all() and (lse[:2] == -np.inf).all() and (out[2:] != 0).any()


def test_steps_of_a_server():
    """Plan, append, select and attend together, step by step from one captured graph a kind of step: prefill, then
    decode; every state against the oracle's."""
    r = np.random.default_rng(21)
    S, most, H, G, D, k = 4, 14, 2, 4, 64, 5
    c = new_cache(r, S, most, H, D)
    free = c["table"].reshape(-1).copy()
    c["table"][:] = -1
    g = to_gpu(c)
    g.page_table.fill_(-1)
    length, head = np.zeros(S, np.int64), 0
    st = dict(length=gpu(np.zeros(S, np.int32)), add=gpu(np.zeros(S, np.int32)), free=gpu(free), head=gpu(np.zeros(1, np.int32)))
    for cap, steps in ((700, [(65, 700 - 65 - 1 - 300, 1, 300), (10, 0, 500, 3)]), (6, [(1, 1, 1, 1), (1, 0, 1, 1), (2, 1, 0, 1)])):
        x = [torch.zeros((cap, h, D), dtype=torch.bfloat16, device=DEV) for h in (H * G, H, H)]
        out = csa2.PagePlan.allocate(S, cap, DEV)
        out.length, out.head = st["length"], st["head"]
        res = {}

        def step():
            p = csa2.page_plan(st["length"], st["add"], g.page_table, st["free"], st["head"], cap, out=out)
            csa2.kv8_append(g, x[1], x[2], p.start, p.length)
            pages, _ = csa2.kv8_select(g, x[0], p.start, p.length, k)
            res.update(dense=csa2.kv8_attn(g, x[0], p.start, p.length, max_new=cap),
                       sparse=csa2.kv8_attn(g, x[0], p.start, p.length, pages=pages), pages=pages)

        st["add"].zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for add in steps:
            y = [bf16(r.standard_normal(t.shape)) for t in x]
            for t, v in zip(x, y):
                t.copy_(gpu(v, torch.bfloat16))
            st["add"].copy_(gpu(np.asarray(add, np.int32)))
            graph.replay()
            want = kv8.plan(length, add, c["table"], free, head, cap)
            length, head, T = want["length"], want["head"], int(want["start"][-1])
            kv8.append(c, y[1][:T], y[2][:T], want["start"], length)
            check_cache(g, c)
            start = want["start"].astype(np.int32)
            lists = [[None] * H for _ in range(T)]
            got = res["pages"].cpu().numpy()
            for s in range(S):
                for t in range(start[s], start[s + 1]):
                    n = int(length[s] - (start[s + 1] - t) + 1)
                    lists[t] = kv8.select(c, y[0][t], s, n, k, 1, 1)
                    for h in range(H):
                        assert [j for j in got[t, h] if j >= 0] == lists[t][h]
            check_attn(*res["dense"], c, y[0], start, length, D ** -0.5)
            check_attn(*res["sparse"], c, y[0], start, length, D ** -0.5, pages=lists)
