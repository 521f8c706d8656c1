"""Calls on a GPU that is not the current one, and operands spread over several, on CPU: tensors that stand in for
CUDA ones, and a library that records which device was current when it was called."""
import math

import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2


class OnDevice:
    """A contiguous tensor of a CUDA device that does not exist: everything a call looks at, and an address."""
    is_cuda = True

    def __init__(self, dev, dtype, *shape):
        self.dev, self.dtype, self.shape = dev, dtype, torch.Size(shape)
        self.device = torch.device("cuda", dev)

    def get_device(self):
        return self.dev

    def stride(self, dim=None):
        s = tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))
        return s if dim is None else s[dim]

    def is_contiguous(self):
        return True

    def numel(self):
        return math.prod(self.shape)

    def data_ptr(self):
        return 0x1000 * (self.dev + 1)


@pytest.fixture
def machine(monkeypatch):
    """Two GPUs, device 0 current.  Returns the list of (function, device that was current, stream) of every call."""
    current, calls = [0], []

    class device:
        def __init__(self, d):
            self.d = d.index if isinstance(d, torch.device) else d

        def __enter__(self):
            self.before, current[0] = current[0], self.d

        def __exit__(self, *a):
            current[0] = self.before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if not name.endswith("_workspace"):
                    calls.append((name, current[0], getattr(args[-1], "value", args[-1])))
                return 0
            return call

    class stream:
        def __init__(self, d):
            self.cuda_stream = 100 + d

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: stream(current[0] if d is None else d))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    monkeypatch.setattr(csa2._lib, "lib", lambda: Library())
    monkeypatch.setattr(csa2, "_gpus", 2)
    return calls


B16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def fp4(dev, rows, cols, g=None):
    return csa2.Fp4Rows(OnDevice(dev, U8, rows, cols // 2), OnDevice(dev, U8, (rows + 127) // 128, (cols + 63) // 64, 512),
                        OnDevice(dev if g is None else g, F32, 1))


# name -> a call whose operands are made by t(operand, dtype, shape) or q(operand, rows, cols), so that a test can
# move one of them to another device
ROWS = {
    "rms_norm": lambda t, q: csa2.rms_norm(t("x", B16, 4, 64), t("weight", B16, 64), residual=t("residual", B16, 4, 64),
                                           residual_out=t("residual_out", B16, 4, 64), out=t("out", B16, 4, 64)),
    "rms_norm_fp8": lambda t, q: csa2.rms_norm_fp8(t("x", B16, 4, 64), t("weight", F32, 64), out=t("out", U8, 4, 64),
                                                   out_scale=t("out_scale", F32, 4, 1)),
    "rms_norm_fp4": lambda t, q: csa2.rms_norm_fp4(t("x", B16, 4, 64), t("weight", F32, 64), out=q("out", 4, 64)),
    "rope": lambda t, q: csa2.rope(t("x", B16, 4, 2, 64), t("pos", I32, 4), t("cos", F32, 9, 16), t("sin", F32, 9, 16),
                                   out=t("out", B16, 4, 2, 64)),
    "rope_table": lambda t, q: csa2.rope_table(9, 32, out=(t("cos", F32, 9, 16), t("sin", F32, 9, 16))),
    "fp4_quant": lambda t, q: csa2.fp4_quant(t("x", B16, 4, 64), out=q("out", 4, 64)),
    "fp4_linear": lambda t, q: csa2.fp4_linear(q("x", 4, 64), q("w", 8, 64), out=t("out", B16, 4, 8)),
}


OPERANDS = {
    "rms_norm": ["x", "weight", "residual", "residual_out", "out"], "rms_norm_fp8": ["x", "weight", "out", "out_scale"],
    "rms_norm_fp4": ["x", "weight", "out", "out.gscale"], "rope": ["x", "pos", "cos", "sin", "out"], "rope_table": ["cos", "sin"],
    "fp4_quant": ["x", "out", "out.gscale"], "fp4_linear": ["x", "x.gscale", "w", "w.gscale", "out"]}


def run(call, dev, moved=None):
    """The call with every operand on dev but `moved`, which is on the other device."""
    at = lambda name: 1 - dev if name == moved else dev
    return call(lambda name, dtype, *shape: OnDevice(at(name), dtype, *shape),
                lambda name, r, c: fp4(at(name), r, c, at(name + ".gscale") if moved != name else None))


def cache(t):
    return csa2.PagedCache(t("codes", U8, 3, 64, 64), t("scales", U8, 3, 64, 8), t("idx_k", B16, 3, 64, 64),
                           t("page_table", I32, 2, 2))


HOT = {
    "compress_quant": (lambda t, q: csa2.compress_quant(
        cache(t), t("seq", I32, 4), t("entry", I32, 4), H=t("H", B16, 4, 256), W_kv=t("W_kv", B16, 256, 128), pos=t("pos", I32, 4),
        rope_cos=t("rope_cos", F32, 9, 16), rope_sin=t("rope_sin", F32, 9, 16), W_ik=t("W_ik", B16, 128, 64), ws=ws(t)),
        ["seq", "entry", "H", "W_kv", "pos", "rope_cos", "rope_sin", "W_ik"]),
    "compress_append": (lambda t, q: csa2.compress_append(
        cache(t), t("H", B16, 2, 256), t("seq", I32, 2), t("tok_pos", I32, 2), t("W_kv", B16, 256, 128), ws=ws(t)),
        ["H", "seq", "tok_pos", "W_kv"]),
    "index_full": (lambda t, q: csa2.index_full(
        cache(t), t("q_idx", B16, 2, 4, 64), t("w", F32, 2, 4), t("seq_of", I32, 2), t("n_vis", I32, 2), 100, 64, 8, 16,
        out=(t("pool", I32, 2, 512), t("pool_len", I32, 2), t("topk", I32, 2, 16), t("topk_len", I32, 2)), ws=ws(t)),
        ["q_idx", "w", "seq_of", "n_vis", "pool", "topk_len"]),
    "index_reindex": (lambda t, q: csa2.index_reindex(
        cache(t), t("q_idx", B16, 2, 4, 64), t("w", F32, 2, 4), t("seq_of", I32, 2), t("pool", I32, 2, 512), t("pool_len", I32, 2), 16,
        out=(t("topk", I32, 2, 16), t("topk_len", I32, 2)), ws=ws(t)), ["q_idx", "pool", "topk"]),
    "sparse_attn": (lambda t, q: csa2.sparse_attn(
        cache(t), t("q", B16, 2, 8, 128), t("seq_of", I32, 2), t("topk", I32, 2, 16), t("topk_len", I32, 2), t("swa", U8, 64, 128),
        t("swa_scale", F32, 64), t("swa_start", I32, 2), t("swa_len", I32, 2), 32, out=t("out", B16, 2, 8, 128),
        lse=t("lse", F32, 2, 8), ws=ws(t)), ["q", "seq_of", "topk", "swa", "swa_scale", "out", "lse"]),
    "swa_quant": (lambda t, q: csa2.swa_quant(t("x", B16, 4, 128), t("swa", U8, 64, 128), t("swa_scale", F32, 64), t("row_idx", I32, 4)),
                  ["x", "swa", "swa_scale", "row_idx"]),
}
PLANES = ["codes", "scales", "idx_k", "page_table", "workspace"]


def ws(t):
    w = csa2.Workspace("cpu")
    w.get = lambda nbytes: t("workspace", U8, 256)
    return w


@pytest.mark.parametrize("dev", [0, 1])
@pytest.mark.parametrize("name", ROWS)
def test_row_operators_run_on_their_tensors_device(machine, name, dev):
    run(ROWS[name], dev)
    assert [(d, s) for _, d, s in machine] == [(dev, 100 + dev)]
    assert torch._C._cuda_getDevice() == 0                # and the caller's device is current again


@pytest.mark.parametrize("name,moved", [(n, o) for n in ROWS for o in OPERANDS[n]])
def test_row_operators_refuse_operands_of_another_device(machine, name, moved):
    with pytest.raises(ValueError, match="cuda:1"):
        run(ROWS[name], 0, moved)
    assert machine == []


@pytest.mark.parametrize("dev", [0, 1])
@pytest.mark.parametrize("name", HOT)
def test_hot_path_runs_on_its_tensors_device(machine, name, dev):
    run(HOT[name][0], dev)
    assert [(d, s) for _, d, s in machine] == [(dev, 100 + dev)]
    assert torch._C._cuda_getDevice() == 0


@pytest.mark.parametrize("name,moved", [(n, o) for n, (_, named) in HOT.items()
                                        for o in named + (PLANES if n != "swa_quant" else [])])
def test_hot_path_refuses_operands_of_another_device(machine, name, moved):
    with pytest.raises(ValueError, match="cuda:1"):
        run(HOT[name][0], 0, moved)
    assert machine == []


def test_rows_on_the_cpu_have_no_fields():
    with pytest.raises(ValueError, match="CUDA"):
        csa2.Fp4Rows.allocate(4, 64, "cpu").fields()
