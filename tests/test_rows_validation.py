"""Refusals of the row operators on CPU: a valid argument struct (fake device pointers, never
dereferenced) with one field changed returns the stated status before any CUDA call; and the pins
of the oracle they are tested against."""
import ctypes
import math

import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import _lib, build, csa2
from oracle import formats, rows

P, U = 0x10000, 0x10002           # aligned and 2-byte aligned fake device addresses
INVALID, SHAPE = 1, 2


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def make(cls, kw, **base):
    a = cls()
    a.struct_size = ctypes.sizeof(a)
    for k, v in {**base, **kw}.items():
        if k.startswith("out4_"):
            setattr(a.out4, k[5:], v)
        elif k[:2] in ("x_", "w_", "o_") and cls in (_lib.Fp4LinearArgs, _lib.Fp4QuantArgs) and k not in ("x_dtype", "x_stride"):
            setattr(getattr(a, {"x_": "x", "w_": "w", "o_": "out"}[k[:2]]), k[2:], v)
        else:
            setattr(a, k, v)
    return a


def norm(**kw):
    return make(_lib.RmsNormArgs, kw, T=4, D=64, x=P, x_stride=64, eps=1e-6, out=P, out_stride=64, out_form=0)


def rope(**kw):
    return make(_lib.RopeArgs, kw, T=4, H=2, D=64, d_rope=32, rot_first=32, x=P, out=2 * P, x_stride_t=128, x_stride_h=64,
                out_stride_t=128, out_stride_h=64, pos=P, rope_cos=P, rope_sin=P, rope_max_pos=8)


def table(**kw):
    return make(_lib.RopeTableArgs, kw, positions=4, d_rope=32, theta=1e4, factor=2.0, orig_positions=64, beta_fast=32.0,
                beta_slow=1.0, magnitude=1.0, rope_cos=P, rope_sin=P)


def quant(**kw):
    return make(_lib.Fp4QuantArgs, kw, x=P, x_stride=64, o_codes=P, o_scales=P, o_rows=4, o_cols=64)


def linear(**kw):
    return make(_lib.Fp4LinearArgs, kw, x_codes=P, x_scales=P, x_rows=4, x_cols=64, w_codes=P, w_scales=P, w_rows=8,
                w_cols=64, out=P)


CASES = [
    ("csa2_rms_norm", norm, [
        (dict(T=-1), INVALID, b"T < 0"), (dict(D=0), SHAPE, b"D must"), (dict(D=32769), SHAPE, b"D must"),
        (dict(x_dtype=2), INVALID, b"x_dtype"), (dict(eps=-1.0), INVALID, b"eps"), (dict(eps=math.nan), INVALID, b"eps"),
        (dict(weight=P, weight_dtype=3), INVALID, b"weight_dtype"), (dict(weight=U, weight_dtype=1), INVALID, b"weight"),
        (dict(out_form=4), INVALID, b"out_form"), (dict(out_form=2, out_scale=P, scale_group=64), SHAPE, b"scale_group"),
        (dict(out_form=2), INVALID, b"out_scale"), (dict(out_form=3), INVALID, b"out4"),
        (dict(out_form=3, D=72, out4_rows=4, out4_cols=72, out4_codes=P, out4_scales=P), SHAPE, b"multiple of 16"),
        (dict(out_form=3, out4_rows=4, out4_cols=64, out4_codes=P), INVALID, b"NULL"),
        (dict(out_form=3, out4_rows=4, out4_cols=64, out4_codes=P, out4_scales=U), INVALID, b"aligned"),
        (dict(x=None), INVALID, b"x is NULL"), (dict(x=U, x_dtype=1), INVALID, b"aligned"),
        (dict(x=P + 1), INVALID, b"aligned"), (dict(out=None), INVALID, b"out is NULL"),
        (dict(out=U, out_form=1), INVALID, b"aligned"), (dict(out_stride=63), INVALID, b"overlap"),
        (dict(residual=P), INVALID, b"residual_out is NULL"), (dict(residual_out=P), INVALID, b"without"),
        (dict(residual=P, residual_out=P, res_dtype=2, residual_out_stride=64), INVALID, b"res_dtype"),
        (dict(residual=P, residual_out=P, residual_out_stride=63), INVALID, b"overlap"),
        (dict(residual=P, residual_out=P + 1, residual_out_stride=64), INVALID, b"aligned"),
        (dict(struct_size=8), INVALID, b"struct_size")]),
    ("csa2_rope", rope, [
        (dict(T=-1), INVALID, b"T or H"), (dict(H=-1), INVALID, b"T or H"), (dict(D=4097), SHAPE, b"D must"),
        (dict(D=0), SHAPE, b"D must"), (dict(d_rope=0), SHAPE, b"d_rope"), (dict(d_rope=31), SHAPE, b"d_rope"),
        (dict(rot_first=33), INVALID, b"rot_first"), (dict(rot_first=-1), INVALID, b"rot_first"), (dict(d_rope=66), INVALID, b"rot_first"),
        (dict(dtype=2), INVALID, b"dtype"), (dict(x=None), INVALID, b"NULL"), (dict(out=None), INVALID, b"NULL"),
        (dict(pos=None), INVALID, b"NULL"), (dict(rope_cos=None), INVALID, b"NULL"), (dict(rope_sin=None), INVALID, b"NULL"),
        (dict(rope_max_pos=0), INVALID, b"rope_max_pos"), (dict(x=P + 1), INVALID, b"aligned"),
        (dict(out=U, dtype=1), INVALID, b"aligned"), (dict(pos=U), INVALID, b"aligned"),
        (dict(out=P, out_stride_t=256), INVALID, b"in place"), (dict(out_stride_h=63), INVALID, b"overlap"),
        (dict(out_stride_t=127), INVALID, b"overlap"), (dict(out_stride_t=64, out_stride_h=255), INVALID, b"overlap"),
        (dict(struct_size=8), INVALID, b"struct_size")]),
    ("csa2_rope_table", table, [
        (dict(positions=-1), SHAPE, b"positions"), (dict(positions=(1 << 24) + 1), SHAPE, b"positions"),
        (dict(d_rope=258), SHAPE, b"d_rope"), (dict(d_rope=3), SHAPE, b"d_rope"), (dict(scaling=3), INVALID, b"scaling"),
        (dict(theta=1.0), INVALID, b"theta"), (dict(theta=math.nan), INVALID, b"theta"), (dict(theta=math.inf), INVALID, b"theta"),
        (dict(magnitude=0.0), INVALID, b"magnitude"), (dict(scaling=1, factor=0.5), INVALID, b"factor"),
        (dict(scaling=2, orig_positions=0), INVALID, b"orig_positions"), (dict(scaling=2, beta_slow=32.0), INVALID, b"beta_slow"),
        (dict(scaling=2, beta_slow=math.nan), INVALID, b"beta_slow"), (dict(rope_cos=None), INVALID, b"NULL"),
        (dict(rope_sin=U), INVALID, b"aligned"), (dict(struct_size=8), INVALID, b"struct_size")]),
    ("csa2_fp4_quant", quant, [
        (dict(x_dtype=2), INVALID, b"x_dtype"), (dict(o_cols=72), SHAPE, b"multiple of 16"), (dict(o_cols=0), SHAPE, b"cols"),
        (dict(o_rows=-1), SHAPE, b"rows"), (dict(o_rows=(1 << 23) + 1), SHAPE, b"rows"), (dict(o_codes=None), INVALID, b"NULL"),
        (dict(o_scales=P + 8), INVALID, b"aligned"), (dict(o_gscale=U), INVALID, b"gscale"), (dict(x=None), INVALID, b"x is NULL"),
        (dict(x=U, x_dtype=1), INVALID, b"aligned"), (dict(struct_size=8), INVALID, b"struct_size")]),
    ("csa2_fp4_linear", linear, [
        (dict(x_cols=48, w_cols=48), SHAPE, b"multiple of 32"), (dict(w_cols=128), INVALID, b"x.cols"),
        (dict(x_rows=-1), SHAPE, b"rows"), (dict(w_rows=-2), SHAPE, b"rows"), (dict(x_codes=None), INVALID, b"NULL"),
        (dict(w_scales=P + 8), INVALID, b"aligned"), (dict(out=None), INVALID, b"out is NULL"), (dict(out=U, out_dtype=1), INVALID, b"aligned"),
        (dict(out_dtype=2), INVALID, b"out_dtype"), (dict(struct_size=8), INVALID, b"struct_size")]),
]


@pytest.mark.parametrize("fn,kw,status,words,build_args", [
    pytest.param(fn, kw, st, w, b, id=f"{fn}-{'-'.join(f'{k}={v}' for k, v in kw.items())}") for fn, b, cs in CASES for kw, st, w in cs])
def test_refusals(L, fn, kw, status, words, build_args):
    assert getattr(L, fn)(ctypes.byref(build_args(**kw)), None) == status
    assert words in L.csa2_last_error_message()


@pytest.mark.parametrize("fn,b", [(c[0], c[1]) for c in CASES])
def test_null_and_empty(L, fn, b):
    assert getattr(L, fn)(None, None) == INVALID
    empty = {"csa2_rms_norm": dict(T=0, x=None, out=None), "csa2_rope": dict(T=0, x=None, out=None),
             "csa2_rope_table": dict(positions=0, rope_cos=None, rope_sin=None),
             "csa2_fp4_quant": dict(o_rows=0, x=None, o_codes=None, o_scales=None),
             "csa2_fp4_linear": dict(x_rows=0, x_codes=None, x_scales=None, out=None)}[fn]
    assert getattr(L, fn)(ctypes.byref(b(**empty)), None) == 0
    assert fn in _lib.EXPORTS


def test_python_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: csa2.rms_norm(x), lambda: csa2.rms_norm_fp8(x), lambda: csa2.rms_norm_fp4(x), lambda: csa2.fp4_quant(x),
                 lambda: csa2.rope(x.view(4, 1, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(2, 16), torch.zeros(2, 16))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="scaling"):
        csa2.rope_table(4, 32, scaling="ntk", device="cpu")
    with pytest.raises(ValueError, match="multiple of 16"):
        csa2.Fp4Rows.allocate(3, 24, "cpu")
    q = csa2.Fp4Rows.allocate(130, 80, "cpu")
    assert q.scales.shape == (2, 2, 512) and q.row_scales().shape == (130, 5)
    with pytest.raises(ValueError, match="belong"):
        csa2.Fp4Rows(q.codes, q.scales[:1]).fields()
    with pytest.raises(ValueError, match="one element"):
        csa2.Fp4Rows(q.codes, q.scales, torch.zeros(2)).fields()


def test_packed_structs_have_the_c_layout():
    for packed, st in [(csa2._RMS_NORM, _lib.RmsNormArgs), (csa2._ROPE, _lib.RopeArgs), (csa2._FP4_QUANT, _lib.Fp4QuantArgs),
                       (csa2._FP4_LINEAR, _lib.Fp4LinearArgs)]:
        assert packed.size == ctypes.sizeof(st)
        n = len(packed.unpack(bytes(packed.size)))
        a = st.from_buffer_copy(packed.pack(*range(1, n + 1)))
        got = []

        def walk(v):
            for name, kind in v._fields_:
                x = getattr(v, name)
                walk(x) if issubclass(kind, ctypes.Structure) else got.append(x)

        walk(a)
        assert got == list(range(1, n + 1))


def test_scale_tiles_round_trip():
    s = np.random.default_rng(0).integers(0, 256, (300, 9), dtype=np.uint8)
    q = csa2.Fp4Rows(torch.zeros((300, 72), dtype=torch.uint8), torch.from_numpy(rows.scale_tiles(s)))
    assert np.array_equal(q.row_scales().numpy(), s)


def test_oracle_norm_steps_stay_near_the_definition():
    r = np.random.default_rng(1)
    h, w = r.standard_normal((7, 333)).astype(np.float32), r.standard_normal(333).astype(np.float32)
    a, b = rows.rms_norm_f32(h, w, 1e-6), rows.rms_norm(h, w, 1e-6)
    assert (np.abs(a - b) <= np.abs(b) * 5 * 2.0 ** -24 * 1.001).all()
    assert np.allclose(np.mean(rows.rms_norm(h, None, 0.0) ** 2, -1), 1, rtol=1e-12)


def test_oracle_rope_turns_back_and_keeps_norms():
    r = np.random.default_rng(2)
    x, pos = r.standard_normal((5, 2, 20)), np.array([0, 3, 9, 1, 7])
    a = np.outer(np.arange(10), rows.frequencies(8))
    cos, sin = np.cos(a), np.sin(a)
    for inter in (True, False):
        y = rows.rope(x, pos, cos, sin, inter, False, 4)
        assert np.allclose(rows.rope(y, pos, cos, sin, inter, True, 4), x, rtol=0, atol=1e-14)
        assert np.array_equal(y[0], x[0]) and np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.array_equal(y[..., :4], x[..., :4]) and np.array_equal(y[..., 12:], x[..., 12:])
    # pairs of the two layouts are the same pairs in another order
    perm = np.concatenate([np.arange(4), 4 + 2 * np.arange(4), 5 + 2 * np.arange(4), np.arange(12, 20)])
    assert np.allclose(rows.rope(x, pos, cos, sin, True, False, 4)[..., perm], rows.rope(x[..., perm], pos, cos, sin, False, False, 4))


def test_oracle_yarn_ends():
    f, y = rows.frequencies(64), rows.frequencies(64, scaling="yarn", factor=16.0, orig=4096)
    assert y[0] == f[0] and y[-1] == f[-1] / 16 and (np.diff(y) < 0).all()
    assert np.allclose(rows.frequencies(64, scaling="yarn", factor=1.0, orig=4096), f, rtol=1e-15)


def test_oracle_linear_of_grid_values():
    q = formats.fp4_quantize(np.array([[1, 2, 3, 4, 6, -6] + [0] * 10], np.float32) * 2)
    y, mag = rows.fp4_linear(*q, *q, 0.5, 2.0)
    assert y[0, 0] == 4 * (1 + 4 + 9 + 16 + 72) and mag[0, 0] == y[0, 0]
