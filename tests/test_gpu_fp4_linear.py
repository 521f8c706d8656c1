"""The FP4 product on the block-scaled tensor cores against the float64 oracle."""
import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2
from oracle import rows

pytestmark = pytest.mark.gpu
U, UB = 2.0 ** -24, 2.0 ** -8
DEV = "cuda"


def fp4(r, R, K, g=None, lo=0x08, hi=0x58):
    """Random codes, scale bytes of a wide range (2^-6 .. 2^4), in tiles; and row by row."""
    codes = r.integers(0, 256, (R, K // 2), dtype=np.uint8)
    sc = r.integers(lo, hi, (R, K // 16), dtype=np.uint8)
    t = csa2.Fp4Rows(torch.from_numpy(codes).to(DEV), torch.from_numpy(rows.scale_tiles(sc)).to(DEV),
                     None if g is None else torch.full((1,), g, device=DEV))
    return t, codes, sc


def check(y, xc, xs, wc, ws, gx=1.0, gw=1.0):
    K = xc.shape[1] * 2
    ref, mag = rows.fp4_linear(xc, xs, wc, ws, gx, gw)
    # Products and scales are exact.  Each 64-column step adds to a float32 accumulator with at most
    # two steps of the largest partial sum lost; the split over CTAs adds at most 15 more sums.
    tol = ((K + 63) // 64 + 16) * 4 * U * mag + 2 * U * np.abs(ref) + (UB * np.abs(ref) if y.dtype == torch.bfloat16 else 0)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,K", [
    (1, 1, 32), (1, 128, 64), (1, 129, 96), (2, 100, 256), (16, 8, 288), (17, 1000, 1024), (33, 128, 4128),
    (64, 300, 512), (65, 256, 2048), (128, 128, 320), (129, 640, 1056), (200, 130, 96), (300, 77, 4096), (513, 257, 544),
    (1, 4096, 16384), (7, 512, 32768), (257, 1024, 160)])
def test_fp4_linear(T, N, K, out):
    r = np.random.default_rng(T * 1000003 + N * 1009 + K)
    x, xc, xs = fp4(r, T, K, 0.75)
    w, wc, ws = fp4(r, N, K, 0.0123)
    y = csa2.fp4_linear(x, w, out_dtype=out)
    check(y, xc, xs, wc, ws, 0.75, 0.0123)
    assert torch.equal(y, csa2.fp4_linear(x, w, out_dtype=out))       # bit for bit
    assert csa2.device_error() == 0


@pytest.mark.parametrize("T,N,K,out", [
    (130, 77 * 256, 12288, torch.bfloat16),        # 77 tiles of pairs: a last round of one tile, split and launched apart
    (700, 40 * 256 + 3, 160, torch.bfloat16),      # several rounds, rows that TMA cannot address
    (700, 40 * 256 + 3, 160, torch.float32),
    (640, 40 * 256, 288, torch.float32),
    (520, 19000, 8192, torch.bfloat16),
    (192, 5120, 20480, torch.bfloat16),            # 20 tiles of pairs, the sum split in a cluster
    (161, 5119, 20480, torch.float32),
    (129, 5117, 20512, torch.bfloat16),
    (500, 1000, 16384, torch.bfloat16),            # 32 tiles of single CTAs, split
    (1000, 4999, 96, torch.float32)])              # 320 tiles of single CTAs' size
def test_fp4_linear_many_tiles(T, N, K, out):
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    r8 = lambda *s: torch.randint(0, 256, s, generator=g, device=DEV, dtype=torch.uint8)
    sc = lambda R: torch.randint(0x28, 0x48, ((R + 127) // 128, (K + 63) // 64, 512), generator=g, device=DEV,
                                 dtype=torch.uint8)
    x, w = csa2.Fp4Rows(r8(T, K // 2), sc(T)), csa2.Fp4Rows(r8(N, K // 2), sc(N))
    if K % 64:                     # scales past the last column are zero
        for m in (x, w):
            m.scales[:, -1].view(-1, 128, 4)[:, :, 2:] = 0
    y = csa2.fp4_linear(x, w, out_dtype=out)
    assert csa2.device_error() == 0
    assert torch.equal(y, csa2.fp4_linear(x, w, out_dtype=out))
    cols = np.unique(np.concatenate([np.arange(40), np.arange(N - 300, N), np.linspace(0, N - 1, 100).astype(int)]))
    c = lambda t: t.cpu().numpy()
    at = torch.from_numpy(cols).to(DEV)
    check(y[:, at], c(x.codes), c(x.row_scales()), c(w.codes[at]), c(w.row_scales()[at]))


def test_fp4_linear_exact_sums():
    """Powers of two whose sums are exact in float32: every step of K counts once, in its place."""
    T, N, K = 40, 200, 1120
    xc = np.zeros((T, K // 2), np.uint8)
    wc = np.full((N, K // 2), 0x22, np.uint8)       # code 2 = 1.0
    xs, ws = np.full((T, K // 16), 0x38, np.uint8), np.full((N, K // 16), 0x38, np.uint8)
    for t in range(T):                              # token t: ones in columns [0, 28 t)
        n = 28 * t
        xc[t, :n // 2] = 0x22
        xs[t, :] = 0x38 + 8 * (t % 3)               # scales 1, 2, 4
    for n in range(N):
        ws[n, :] = 0x38 - 8 * (n % 4)               # 1, 1/2, 1/4, 1/8
    d = lambda c, s: csa2.Fp4Rows(torch.from_numpy(c).to(DEV), torch.from_numpy(rows.scale_tiles(s)).to(DEV))
    y = csa2.fp4_linear(d(xc, xs), d(wc, ws), out_dtype=torch.float32).cpu().numpy()
    want = (28.0 * np.arange(T) * 2.0 ** (np.arange(T) % 3))[:, None] * 2.0 ** -(np.arange(N) % 4)[None]
    assert np.array_equal(y, want.astype(np.float32))


@pytest.mark.parametrize("T", [3, 40, 150])
def test_fp4_linear_every_scale_place(T):
    """One nonzero scale at a time: rows, columns and 16-column groups are not mixed up."""
    N, K = 140, 320
    r = np.random.default_rng(9)
    wc, ws = r.integers(0, 256, (N, K // 2), dtype=np.uint8), r.integers(0x30, 0x40, (N, K // 16), dtype=np.uint8)
    xc = r.integers(0, 256, (T, K // 2), dtype=np.uint8)
    xs = np.zeros((T, K // 16), np.uint8)
    xs[np.arange(T), (7 * np.arange(T)) % (K // 16)] = 0x38
    d = lambda c, s: csa2.Fp4Rows(torch.from_numpy(c).to(DEV), torch.from_numpy(rows.scale_tiles(s)).to(DEV))
    check(csa2.fp4_linear(d(xc, xs), d(wc, ws), out_dtype=torch.float32), xc, xs, wc, ws)


@pytest.mark.parametrize("T", [5, 300])
def test_fp4_linear_nan_scale_stays_in_its_row(T):
    r = np.random.default_rng(10)
    N, K = 200, 512
    x, xc, xs = fp4(r, T, K)
    w, wc, ws = fp4(r, N, K)
    xs[3, 7], ws[150, 1] = 0x7F, 0x7F
    d = lambda c, s: csa2.Fp4Rows(torch.from_numpy(c).to(DEV), torch.from_numpy(rows.scale_tiles(s)).to(DEV))
    y = csa2.fp4_linear(d(xc, xs), d(wc, ws), out_dtype=torch.float32).cpu().numpy()
    nan = np.zeros((T, N), bool)
    nan[3], nan[:, 150] = True, True
    assert np.array_equal(np.isnan(y), nan)


def test_fp4_linear_empty():
    e = csa2.Fp4Rows.allocate
    assert csa2.fp4_linear(e(0, 64, DEV), e(5, 64, DEV)).shape == (0, 5)
    assert csa2.fp4_linear(e(5, 64, DEV), e(0, 64, DEV)).shape == (5, 0)


def test_quantised_product_end_to_end():
    """norm -> FP4 -> product against the float64 product of the dequantised operands."""
    r = np.random.default_rng(11)
    x = r.standard_normal((37, 640)).astype(np.float32)
    wt = (r.standard_normal((96, 640)) / 25).astype(np.float32)
    g = float(np.abs(wt).max() / (6 * 448))
    q, _ = csa2.rms_norm_fp4(torch.from_numpy(x).to(DEV))
    w = csa2.fp4_quant(torch.from_numpy(wt).to(DEV), torch.full((1,), g, device=DEV))
    y = csa2.fp4_linear(q, w, out_dtype=torch.float32)
    c = lambda t: t.cpu().numpy()
    check(y, c(q.codes), c(q.row_scales()), c(w.codes), c(w.row_scales()), 1.0, g)
    full = rows.rms_norm(x, None, 1e-6) @ wt.T.astype(np.float64)
    # FP4 keeps about 2.5 bits: the product is near the unquantised one, in norm
    assert np.linalg.norm(c(y) - full) <= 0.25 * np.linalg.norm(full)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,N,K", [
    (33, 2045, 4128), (64, 2176, 8192), (50, 9216, 3616),      # pairs on up to 64 tokens
    (65, 2045, 3616), (128, 5120, 4096), (97, 9100, 16384),    # up to 128
    (129, 2048, 4640), (192, 3001, 8192), (131, 9216, 4640),   # up to 192
    (193, 2050, 4640), (256, 5120, 8224),                      # up to 256
    (300, 4096, 32768), (512, 2044, 32768)])                   # wide pairs, the sum split in a cluster
def test_fp4_linear_pairs_split(T, N, K, out):
    test_fp4_linear_many_tiles(T, N, K, out)


@pytest.mark.parametrize("T,K,N", [(40, 4096, 2100), (100, 4096, 2100), (150, 5120, 2100), (250, 5120, 2100)])
def test_fp4_linear_pairs_rows_and_scales(T, K, N):
    """One nonzero scale a row, and a row and a feature of NaN scales: neither halves nor parts are mixed up."""
    r = np.random.default_rng(12)
    wc, ws = r.integers(0, 256, (N, K // 2), dtype=np.uint8), r.integers(0x30, 0x40, (N, K // 16), dtype=np.uint8)
    xc = r.integers(0, 256, (T, K // 2), dtype=np.uint8)
    xs = np.zeros((T, K // 16), np.uint8)
    xs[np.arange(T), (7 * np.arange(T)) % (K // 16)] = 0x38
    d = lambda c, s: csa2.Fp4Rows(torch.from_numpy(c).to(DEV), torch.from_numpy(rows.scale_tiles(s)).to(DEV))
    check(csa2.fp4_linear(d(xc, xs), d(wc, ws), out_dtype=torch.float32), xc, xs, wc, ws)
    xs[T - 3, K // 16 - 1], ws[150, 1], ws[N - 1, K // 32] = 0x7F, 0x7F, 0x7F
    y = csa2.fp4_linear(d(xc, xs), d(wc, ws), out_dtype=torch.float32).cpu().numpy()
    nan = np.zeros((T, N), bool)
    nan[T - 3], nan[:, 150], nan[:, N - 1] = True, True, True
    assert np.array_equal(np.isnan(y), nan)
