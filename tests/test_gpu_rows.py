"""Residual norm, rotary positions and the FP4 quantiser on the GPU against the float64 oracle."""
import math

import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2, synth
from oracle import formats, rows

pytestmark = pytest.mark.gpu
U = 2.0 ** -24           # half a float32 step
UB = 2.0 ** -8           # half a bf16 step, relative to the value's binade at worst
DEV = "cuda"


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def strided(a, dtype, pad):
    """The matrix as rows of a wider one, starting `pad` elements in."""
    if not pad:
        return gpu(a, dtype)
    t = torch.full((a.shape[0], a.shape[1] + 2 * pad), float("nan"), dtype=dtype, device=DEV)
    t[:, pad:pad + a.shape[1]] = gpu(a, dtype)
    return t[:, pad:pad + a.shape[1]]


def values(r, shape, bf16):
    """Rows of very different magnitudes with a few loud channels; exact in the type."""
    x = r.standard_normal(shape) * np.exp2(r.integers(-6, 7, shape[:1] + (1,) * (len(shape) - 1)))
    x[..., :: 37] *= 16
    x = x.astype(np.float32)
    return formats.bf16_value(formats.bf16_round(x)).astype(np.float32) if bf16 else x


T = {True: torch.bfloat16, False: torch.float32}
SHAPES = [(1, 1), (1, 16), (3, 17), (2, 128), (5, 130), (129, 64), (7, 1001), (4, 5120), (130, 256), (2, 16384),
          (1, 16400), (2, 32768)]


def norm_inputs(shape, xb, rb, seed=0):
    r = np.random.default_rng(seed)
    x = values(r, shape, xb)
    res = values(r, shape, rb)
    w = formats.bf16_value(formats.bf16_round(1 + 0.2 * r.standard_normal(shape[1]))).astype(np.float32)
    return x, res, w


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("xb,rb,pad", [(True, None, 0), (False, None, 3), (True, True, 8), (True, False, 0),
                                       (False, False, 1), (False, True, 5)])
@pytest.mark.parametrize("shape", SHAPES)
def test_rms_norm(shape, xb, rb, pad, out):
    x, res, w = norm_inputs(shape, xb, bool(rb))
    tx = strided(x, T[xb], pad)
    h = x if rb is None else rows.add(x, res, rb)
    tr = None if rb is None else strided(res, T[rb], pad)
    y, hr = csa2.rms_norm(tx, gpu(w, torch.bfloat16), eps=1e-5, residual=tr, out_dtype=out)
    if rb is None:
        assert hr is None
    else:
        assert torch.equal(hr.float().cpu(), torch.from_numpy(h))
    ref = rows.rms_norm(h, w, 1e-5)
    # the mean and its sum with eps (half weight each), root, reciprocal, two products
    tol = np.abs(ref) * (5 * U + (UB if out == torch.bfloat16 else 0)) * 1.001
    assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("xb,rb,pad", [(True, True, 0), (False, None, 1), (True, False, 16)])
@pytest.mark.parametrize("shape", SHAPES)
def test_rms_norm_fp8(shape, xb, rb, pad, group):
    x, res, w = norm_inputs(shape, xb, bool(rb), 1)
    h = x if rb is None else rows.add(x, res, rb)
    tr = None if rb is None else strided(res, T[rb], pad)
    codes, sc, hr = csa2.rms_norm_fp8(strided(x, T[xb], pad), gpu(w, torch.bfloat16), residual=tr, group=group)
    rc, rs = rows.fp8_groups(rows.rms_norm_f32(h, w, 1e-6), group)
    assert np.array_equal(sc.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)


@pytest.mark.parametrize("gscale", [None, 0.0371])
@pytest.mark.parametrize("xb,rb,pad", [(True, True, 0), (False, None, 1), (True, False, 16)])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[1] % 16 == 0] + [(3, 48), (127, 80), (128, 64), (257, 4128)])
def test_rms_norm_fp4(shape, xb, rb, pad, gscale):
    x, res, w = norm_inputs(shape, xb, bool(rb), 2)
    h = x if rb is None else rows.add(x, res, rb)
    tr = None if rb is None else strided(res, T[rb], pad)
    g = None if gscale is None else torch.full((1,), gscale, device=DEV)
    q, hr = csa2.rms_norm_fp4(strided(x, T[xb], pad), gpu(w, torch.bfloat16), residual=tr, gscale=g)
    rc, rs = rows.fp4_quantize(rows.rms_norm_f32(h, w, 1e-6), gscale)
    assert np.array_equal(q.row_scales().cpu().numpy(), rs)
    assert np.array_equal(q.codes.cpu().numpy(), rc)
    assert np.array_equal(q.scales.cpu().numpy(), rows.scale_tiles(rs))


def test_rms_norm_in_place_and_no_weight():
    x, res, _ = norm_inputs((33, 640), True, True, 3)
    tx, tr = gpu(x, torch.bfloat16), gpu(res, torch.bfloat16)
    h = rows.add(x, res, True)
    y, hr = csa2.rms_norm(tx, residual=tr, residual_out=tr, out=tx)
    assert hr is tr and y is tx
    assert torch.equal(tr.float().cpu(), torch.from_numpy(h))
    ref = rows.rms_norm(h, None, 1e-6)
    assert (np.abs(y.double().cpu().numpy() - ref) <= np.abs(ref) * (4 * U + UB) * 1.001).all()


@pytest.mark.parametrize("D,pad", [(256, 0), (1024, 0), (256, 1)])
def test_rms_norm_extremes(D, pad):
    """Zero rows, squares beyond float32, and non-finite values, row by row, on each kernel."""
    x = np.zeros((6, D), np.float32)
    x[1] = 3e18                                     # the sum of squares overflows, the mean does not
    x[2] = 1e38                                     # the mean overflows: r = 0
    x[3, 5], x[4, 7] = np.inf, np.nan
    x[3, 6] = x[4, 8] = 1
    x[5] = np.linspace(-1, 1, D)
    y, _ = csa2.rms_norm(strided(x, torch.float32, pad), out_dtype=torch.float32)
    y = y.cpu().numpy()
    assert (y[0] == 0).all() and np.allclose(y[1], 1, rtol=8 * U, atol=0) and (y[2] == 0).all()
    assert np.isnan(y[3, 5]) and (np.delete(y[3], 5) == 0).all() and np.isnan(y[4]).all()
    ref = rows.rms_norm(x[5], None, 1e-6)
    assert (np.abs(y[5] - ref) <= np.abs(ref) * 5 * U).all()
    q, _ = csa2.rms_norm_fp4(strided(x, torch.float32, pad))
    s = q.row_scales().cpu().numpy()
    assert (s[0] == 0).all() and (s[4] == 0x7F).all() and (q.codes[4] == 0).all()


# ---- FP4 quantiser --------------------------------------------------------------------------

@pytest.mark.parametrize("gscale", [None, 0.0371, 64.0])
@pytest.mark.parametrize("bf16,pad", [(True, 0), (False, 0), (True, 1), (False, 4)])
@pytest.mark.parametrize("shape", [(1, 16), (1, 32768), (2, 48), (127, 64), (128, 80), (129, 256), (300, 272), (33, 1040)])
def test_fp4_quant(shape, bf16, pad, gscale):
    r = np.random.default_rng(4)
    x = values(r, shape, bf16)
    x *= np.exp2(r.integers(-20, 12, (shape[0], shape[1] // 16))).repeat(16, 1).astype(np.float32)
    x[0, :16] = 0
    x[-1, -16:] = -0.0
    g = None if gscale is None else torch.full((1,), gscale, device=DEV)
    q = csa2.fp4_quant(strided(x, T[bf16], pad), g)
    rc, rs = rows.fp4_quantize(x, gscale)
    assert np.array_equal(q.row_scales().cpu().numpy(), rs)
    assert np.array_equal(q.codes.cpu().numpy(), rc)
    assert np.array_equal(q.scales.cpu().numpy(), rows.scale_tiles(rs))


def test_fp4_quant_borders():
    """For every E4M3 scale: each border between two codes, the float32 before and after it."""
    scale = formats.e4m3_value(np.arange(1, 127)).astype(np.float32)
    x = np.zeros((126, 48), np.float32)
    for i, m in enumerate([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]):
        v = scale * np.float32(m)
        for j, u in enumerate((v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(np.inf)))):
            x[:, 16 * j + 2 * i] = u
            x[:, 16 * j + 2 * i + 1] = -u
    x[:, 14::16] = (6 * scale)[:, None]             # the group's amax: its scale is `scale`
    q = csa2.fp4_quant(gpu(x))
    rc, rs = rows.fp4_quantize(x)
    assert np.array_equal(q.row_scales().cpu().numpy(), rs)
    assert (rs == np.arange(1, 127)[:, None]).all()
    assert np.array_equal(q.codes.cpu().numpy(), rc)


@pytest.mark.parametrize("bf16", [True, False])
def test_fp4_quant_random_gscales(bf16):
    """Matrix scales over 80 octaves (and beyond, where the kernel divides): the quotients x / gscale
    decide the codes bit for bit."""
    r = np.random.default_rng(12)
    x = values(r, (64, 1024), bf16)
    for e in [-75, -61, -40, -12, -3, 0, 5, 20, 59, 63]:
        g = np.float32(np.ldexp(1 + r.random(), e))
        with np.errstate(over="ignore"):
            y = (x * np.float32(2.0 ** e)).astype(np.float32)
        y = formats.bf16_value(formats.bf16_round(y)).astype(np.float32) if bf16 else y
        q = csa2.fp4_quant(gpu(y, T[bf16]), gpu(np.array([g], np.float32)))
        rc, rs = rows.fp4_quantize(y, g)
        assert np.array_equal(q.row_scales().cpu().numpy(), rs), e
        assert np.array_equal(q.codes.cpu().numpy(), rc), e


def test_fp4_quant_scale_borders():
    """Groups whose amax is at, just below and just above 6 times each border between E4M3 values."""
    v = formats.e4m3_value(np.arange(0, 127))
    m = ((v[1:] + v[:-1]) / 2).astype(np.float32) * np.float32(6)
    x = np.zeros((126, 48), np.float32)
    for j, u in enumerate((m, np.nextafter(m, np.float32(0)), np.nextafter(m, np.float32(np.inf)))):
        x[:, 16 * j + 3] = -u
        x[:, 16 * j + 4] = u / 2
    q = csa2.fp4_quant(gpu(x))
    rc, rs = rows.fp4_quantize(x)
    assert np.array_equal(q.row_scales().cpu().numpy(), rs) and np.array_equal(q.codes.cpu().numpy(), rc)


def test_fp4_quant_nonfinite():
    x = np.ones((4, 32), np.float32)
    x[0, 3], x[1, 3], x[2, 3], x[3, :16] = np.inf, -np.inf, np.nan, 3e38
    q = csa2.fp4_quant(gpu(x))
    s, c = q.row_scales().cpu().numpy(), formats.fp4_unpack(q.codes.cpu().numpy())
    assert list(s[:, 0]) == [0x7E, 0x7E, 0x7F, 0x7E]
    assert c[0, 3] == 7 and c[1, 3] == 15 and (c[2, :16] == 0).all() and (c[3, :16] == 7).all()
    ref = rows.fp4_quantize(np.ones((1, 16), np.float32))
    assert (s[:, 1] == ref[1][0, 0]).all() and (q.codes[:, 8:].cpu().numpy() == ref[0]).all()


# ---- rotary positions ------------------------------------------------------------------------

@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T_,H,D,d_rope,first,pad", [
    (1, 1, 2, 2, None, 0), (1, 64, 512, 64, None, 0), (5, 3, 128, 128, None, 0), (3, 8, 192, 64, 0, 8),
    (4, 2, 100, 32, 33, 0), (2, 5, 65, 6, None, 1), (300, 2, 64, 32, 16, 3), (1, 2, 4096, 4096, None, 1), (7, 24, 96, 48, None, 0)])
def test_rope(T_, H, D, d_rope, first, pad, bf16, interleaved, inverse):
    r = np.random.default_rng(5)
    P = 5000
    cos, sin = synth.rope_tables(P, d_rope)
    x = values(r, (T_, H, D), bf16)
    pos = r.integers(0, P, T_).astype(np.int32)
    tx = strided(x.reshape(T_, H * D), T[bf16], pad).unflatten(1, (H, D))
    y = csa2.rope(tx, gpu(pos), gpu(cos), gpu(sin), interleaved=interleaved, inverse=inverse, first=first)
    f = D - d_rope if first is None else first
    ref = rows.rope(x, pos, cos, sin, interleaved, inverse, f)
    mag = rows.rope(np.abs(x), pos, np.abs(cos), -np.abs(sin), interleaved, False, f)
    mag = np.maximum(mag, rows.rope(np.abs(x), pos, np.abs(cos), np.abs(sin), interleaved, False, f))
    # two products and a sum, then the type
    tol = mag * 2 * U * 1.001 + np.abs(ref) * (U + (UB if bf16 else 0))
    got = y.double().cpu().numpy()
    turned = np.zeros(D, bool)
    turned[f:f + d_rope] = True
    assert (np.abs(got - ref) <= tol * (1 + UB))[..., turned].all()
    assert np.array_equal(got[..., ~turned], x[..., ~turned].astype(np.float64))
    back = csa2.rope(tx, gpu(pos), gpu(cos), gpu(sin), interleaved=interleaved, inverse=inverse, first=first, out=tx)
    assert back is tx and torch.equal(tx, y)        # in place
    assert csa2.device_error() == 0


def test_rope_head_major_and_bad_positions():
    """Tokens as the inner rows (a [H, T, D] tensor seen as [T, H, D]); bad positions are copied."""
    r = np.random.default_rng(6)
    cos, sin = synth.rope_tables(100, 32)
    x = values(r, (4, 9, 64), True)
    pos = np.array([0, 99, 100, -1, 5, 2 ** 31 - 1, 7, 50, -2 ** 31], np.int32)
    tx = gpu(x, torch.bfloat16).transpose(0, 1)
    out = torch.empty((4, 9, 64), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    csa2.rope(tx, gpu(pos), gpu(cos), gpu(sin), out=out)
    assert csa2.device_error() == 0x40
    ok = (pos >= 0) & (pos < 100)
    ref = rows.rope(x.transpose(1, 0, 2)[ok], pos[ok], cos, sin, True, False, 32)
    got = out.double().cpu().numpy()
    assert np.abs(got[ok] - ref).max() <= 2 * UB * np.abs(ref).max()
    assert np.array_equal(got[~ok], x.transpose(1, 0, 2)[~ok].astype(np.float64))
    assert csa2.device_error() == 0


def test_rope_gradient():
    """The inverse is the gradient: d(sum g . rope(x)) / dx by central differences of the float64 form."""
    r = np.random.default_rng(7)
    cos, sin = synth.rope_tables(300, 8)
    x, g = r.standard_normal((2, 1, 12)), r.standard_normal((2, 1, 12)).astype(np.float32)
    pos = np.array([3, 299], np.int32)
    for inter in (True, False):
        got = csa2.rope(gpu(g), gpu(pos), gpu(cos), gpu(sin), interleaved=inter, inverse=True).double().cpu().numpy()
        num = np.zeros_like(x)
        for i in np.ndindex(x.shape):
            e = np.zeros_like(x)
            e[i] = 0.5
            f = [np.sum(g * rows.rope(x + s * e, pos, cos, sin, inter, False, 4)) for s in (1, -1)]
            num[i] = f[0] - f[1]
        # linear in x: the difference is exact up to float64; three float32 roundings on our side
        assert np.abs(got - num).max() <= 4 * U * np.abs(g).max() * math.sqrt(2) + 1e-12


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=8.0), dict(theta=500000.0),
                                dict(scaling="yarn", factor=40.0, orig_positions=4096, magnitude=1.3689),
                                dict(scaling="yarn", factor=1.0, orig_positions=1, beta_fast=2.0, beta_slow=0.5)])
@pytest.mark.parametrize("P,d_rope", [(1, 2), (3, 34), (1000, 64), (70000, 128), (1 << 24, 2)])
def test_rope_table(P, d_rope, kw):
    cos, sin = csa2.rope_table(P, d_rope, **kw)
    o = {("orig" if k == "orig_positions" else k): v for k, v in kw.items() if k != "magnitude"}
    f, mag = rows.frequencies(d_rope, **o), kw.get("magnitude", 1.0)
    p = np.unique(np.concatenate([np.arange(min(P, 2000)), np.linspace(0, P - 1, 5000).astype(np.int64)]))
    a = p[:, None] * f[None]
    at = torch.from_numpy(p).to(DEV)
    # half a step of the value and one of the function below 1, the product with the magnitude, and
    # the float64 angle itself (p f is rounded in the oracle: 2^-52 of up to 2^24)
    tol = mag * 2.5 * U + P * 2.0 ** -50
    assert np.abs(cos[at].double().cpu().numpy() - mag * np.cos(a)).max() <= tol
    assert np.abs(sin[at].double().cpu().numpy() - mag * np.sin(a)).max() <= tol


def test_empty_rows():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    assert csa2.rms_norm(e)[0].shape == (0, 64)
    assert csa2.rms_norm_fp8(e)[0].shape == (0, 64)
    assert csa2.rms_norm_fp4(e)[0].rows == 0
    assert csa2.fp4_quant(e).scales.shape == (0, 1, 512)
    cos, sin = csa2.rope_table(0, 32)
    assert cos.shape == (0, 16)
    cos, sin = csa2.rope_table(4, 32)
    for s in [(0, 3, 64), (3, 0, 64)]:
        x = torch.empty(s, dtype=torch.bfloat16, device=DEV)
        assert csa2.rope(x, torch.zeros(s[0], dtype=torch.int32, device=DEV), cos, sin).shape == s
