"""Calls of several threads on one stream, on CPU: a call that takes a workspace launches kernels that pass data through it, so
that no other call may launch into the same workspace in between.  The library is a stand-in that takes a while."""
import threading
import time

import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2
from test_devices import OnDevice, machine  # noqa: F401
from test_kv8_validation import ws

B16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def at0(name, dtype, *shape):
    return OnDevice(0, dtype, *shape)


def reindex(shared):
    cache = csa2.PagedCache(at0("codes", U8, 3, 64, 64), at0("scales", U8, 3, 64, 8), at0("idx_k", B16, 3, 64, 64), at0("table", I32, 1, 3))
    csa2.index_reindex(cache, at0("q", B16, 2, 4, 64), at0("w", F32, 2, 4), at0("seq", I32, 2), at0("pool", I32, 2, 16), at0("len", I32, 2),
                       k=8, out=(at0("topk", I32, 2, 8), at0("topk_len", I32, 2)), ws=shared)


@pytest.mark.parametrize("own", ["given", "default"])
@pytest.mark.parametrize("name", ["kv8_select", "kv8_attn", "index_reindex"])
def test_threads_share_a_workspace_one_call_at_a_time(machine, monkeypatch, name, own):  # noqa: F811
    launched = []

    class Slow:
        def __getattr__(self, fn):
            def call(*args):
                if fn.endswith("_workspace"):
                    return 0
                launched.append(threading.get_ident())       # the first kernel
                time.sleep(0.002)                            # ctypes lets other threads run meanwhile
                launched.append(threading.get_ident())       # and the one that reads what it left
                return 0
            return call

    monkeypatch.setattr(csa2._lib, "lib", lambda: Slow())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    shared = ws(at0)
    monkeypatch.setitem(csa2._ws_of, (0, 100), shared)
    monkeypatch.setitem(csa2._default_ws, "cuda:0", shared)
    q, step = at0("q", B16, 5, 6, 64), (at0("start", I32, 4), at0("length", I32, 3))
    cache = csa2.Kv8Cache(at0("k", U8, 9, 2, 64, 64), at0("v", U8, 9, 2, 64, 64), at0("ks", F32, 9, 2), at0("vs", F32, 9, 2), at0("table", I32, 3, 4),
                          at0("mean", torch.int8, 9, 2, 64), at0("mean_scale", F32, 9, 2))
    given = shared if own == "given" else None
    calls = {"kv8_select": lambda: csa2.kv8_select(cache, q, *step, 4, out=(at0("pages", I32, 5, 2, 4), at0("count", I32, 5, 2)), ws=given),
             "kv8_attn": lambda: csa2.kv8_attn(cache, q, *step, out=at0("out", B16, 5, 6, 64), lse=at0("lse", F32, 5, 6), ws=given),
             "index_reindex": lambda: reindex(given)}
    go = threading.Barrier(4)

    def thread():
        go.wait()
        for _ in range(5):
            calls[name]()

    threads = [threading.Thread(target=thread) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(launched) == 40
    assert all(a == b for a, b in zip(launched[::2], launched[1::2]))


def test_threads_get_one_default_workspace_a_stream(monkeypatch):
    """First calls at the same time: both find the same one."""
    made = []

    class Counted:
        def __init__(self, device):
            time.sleep(0.01)
            made.append(self)

    monkeypatch.setattr(csa2, "Workspace", Counted)
    monkeypatch.setattr(csa2, "_ws_of", {})
    monkeypatch.setattr(csa2, "_default_ws", {})
    got = []
    find = [lambda: csa2._stream_ws(0, 7, "cuda:0"), lambda: csa2._ws(None, "cuda:0")]
    threads = [threading.Thread(target=lambda f=f: got.append(f())) for f in find for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 8 and len(set(map(id, got))) == 2
