"""The row operators where element offsets pass 2^31, on other streams than the default one, and the norm of rows
that start off every boundary."""
import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2, synth
from oracle import rows

pytestmark = pytest.mark.gpu
U, UB = 2.0 ** -24, 2.0 ** -8
DEV = "cuda"
R = 2 ** 31 // 32768 + 40            # rows of 32768 whose last ones lie past 2^31 elements


def c(t):
    return t.cpu().numpy()


@pytest.fixture(scope="module")
def big():
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    x = torch.empty((R, 32768), dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=g)
    return x


def test_norm(big):
    x = big.view(-1, 8192)
    T = x.shape[0]
    y, _ = csa2.rms_norm(x)
    q, _ = csa2.rms_norm_fp4(x)
    for t in (0, T // 2, T - 1):
        h = c(x[t:t + 1].float())
        ref = rows.rms_norm(h, None, 1e-6)
        assert (np.abs(c(y[t:t + 1].double()) - ref) <= np.abs(ref) * (4 * U + UB) * 1.001).all()
        rc, rs = rows.fp4_quantize(rows.rms_norm_f32(h, None, 1e-6))
        assert np.array_equal(c(q.codes[t:t + 1]), rc)
        tile = c(q.scales[t // 128])
        got = tile.reshape(128, 32, 4, 4)[:, t % 32, t % 128 // 32].reshape(1, -1)
        assert np.array_equal(got, rs)


def test_quant(big):
    q = csa2.fp4_quant(big)
    for t in (0, R // 2, R - 1):
        rc, rs = rows.fp4_quantize(c(big[t:t + 1].float()))
        assert np.array_equal(c(q.codes[t:t + 1]), rc)
        assert np.array_equal(c(q.scales[t // 128]).reshape(512, 32, 4, 4)[:, t % 32, t % 128 // 32].reshape(1, -1), rs)


def test_rope(big):
    x = big.view(R, 64, 512)
    cos, sin = synth.rope_tables(1000, 64)
    t = lambda a: torch.from_numpy(a).to(DEV)
    pos = np.arange(R).astype(np.int32) % 1000
    y = csa2.rope(x, t(pos), t(cos), t(sin))
    for i in (0, R - 1):
        ref = rows.rope(c(x[i:i + 1].double()), pos[i:i + 1], cos, sin, True, False, 448)
        assert np.abs(c(y[i:i + 1].double()) - ref).max() <= 2 * UB * np.abs(ref).max()
    assert csa2.device_error() == 0


@pytest.mark.parametrize("N", [32768, 32767])
def test_linear(N):
    """A result of more than 2^31 elements."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    K = 64
    r8 = lambda *s: torch.randint(0, 256, s, generator=g, device=DEV, dtype=torch.uint8)
    sc = lambda n: torch.randint(0x30, 0x40, ((n + 127) // 128, 1, 512), generator=g, device=DEV, dtype=torch.uint8)
    x, w = csa2.Fp4Rows(r8(R, K // 2), sc(R)), csa2.Fp4Rows(r8(N, K // 2), sc(N))
    y = csa2.fp4_linear(x, w)
    assert csa2.device_error() == 0
    at = np.array([0, R // 2, R - 2, R - 1])
    xs = c(x.scales).reshape(-1, 32, 4, 4)
    scales = np.stack([xs[t // 128, t % 32, t % 128 // 32] for t in at])
    ref, mag = rows.fp4_linear(c(x.codes)[at], scales, c(w.codes), c(w.row_scales()))
    err = np.abs(c(y[torch.from_numpy(at).to(DEV)].double()) - ref)
    assert (err <= 17 * 4 * U * mag + (2 * U + UB) * np.abs(ref)).all()


def test_on_another_stream():
    """Calls follow the current stream: each input is written there, behind work that takes a while."""
    side = torch.cuda.Stream()
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    x = torch.randn((300, 1024), generator=g, device=DEV).bfloat16()
    w = csa2.fp4_quant(torch.randn((512, 1024), generator=g, device=DEV))
    cos, sin = csa2.rope_table(64, 32)
    pos = (torch.arange(300, device=DEV) % 64).to(torch.int32)

    def chain(h):
        q, r = csa2.rms_norm_fp4(h, residual=h)
        y = csa2.fp4_linear(q, w)
        return csa2.rope(y.view(300, 8, 64), pos, cos, sin), r

    want = [t.clone() for t in chain(x)]
    torch.cuda.synchronize()
    late = torch.zeros_like(x)
    with torch.cuda.stream(side):
        busy = torch.randn((8192, 8192), device=DEV)
        for _ in range(20):
            busy = busy @ busy * 1e-4
        late.copy_(x)
        got = chain(late)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [1, 31, 33, 511, 512, 513, 1023, 16383, 16385])
@pytest.mark.parametrize("T", [1, 3, 5, 130])
def test_norm_unaligned(T, D):
    """Rows that start off every boundary: a warp each up to 512 channels, a CTA each beyond."""
    r = np.random.default_rng(D + T)
    x = r.standard_normal((T, D)).astype(np.float32)
    x[T // 2] = 0
    x[T - 1] *= 3e18                                 # squares beyond float32, summed again scaled
    wide = torch.full((T, D + 2), float("nan"), device=DEV)
    wide[:, 1:-1] = torch.from_numpy(x).to(DEV)
    w = (1 + 0.1 * r.standard_normal(D)).astype(np.float32)
    out = torch.full((T, D + 4), 7.0, device=DEV)
    y, _ = csa2.rms_norm(wide[:, 1:-1], torch.from_numpy(w).to(DEV), out_dtype=torch.float32, out=out[:, 3:3 + D])
    ref = rows.rms_norm(x, w, 1e-6)
    assert (np.abs(c(y.double()) - ref) <= np.abs(ref) * 5 * U * 1.001).all()
    assert (out[:, :3] == 7).all() and (out[:, 3 + D:] == 7).all()      # nothing beside the rows
    codes, scale, _ = csa2.rms_norm_fp8(wide[:, 1:-1], torch.from_numpy(w).to(DEV))
    rc, rs = rows.fp8_groups(rows.rms_norm_f32(x, w, 1e-6), 0)
    assert np.array_equal(c(scale), rs) and np.array_equal(c(codes), rc)
    if D % 16 == 0:
        q, _ = csa2.rms_norm_fp4(wide[:, 1:-1])
        rc, rs = rows.fp4_quantize(rows.rms_norm_f32(x, None, 1e-6))
        assert np.array_equal(c(q.codes), rc) and np.array_equal(c(q.scales), rows.scale_tiles(rs))


@pytest.mark.parametrize("D", [256, 1040])
def test_norm_unaligned_not_finite(D):
    x = torch.ones((5, D + 1), device=DEV)
    x[1, 5], x[3, 9] = float("inf"), float("nan")
    x[4] = 0
    y, _ = csa2.rms_norm(x[:, 1:], out_dtype=torch.float32)
    y = c(y)
    one = c(csa2.rms_norm(torch.ones((1, D), device=DEV), out_dtype=torch.float32)[0])
    assert (y[0] == one[0]).all() and (y[2] == one[0]).all() and (y[4] == 0).all()
    assert np.isnan(y[1, 4]) and (np.delete(y[1], 4) == 0).all() and np.isnan(y[3]).all()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,H,D,d_rope,first", [(1, 1, 2, 2, 0), (3, 9, 66, 64, 1), (40, 17, 130, 66, 64), (2500, 70, 34, 34, 0)])
def test_rope_unaligned(T, H, D, d_rope, first, bf16, interleaved):
    """Heads in eights and the rest of them, on rows that start off every boundary; into new rows and in place."""
    r = np.random.default_rng(H)
    x = torch.from_numpy(r.standard_normal((T, H * D + 3)).astype(np.float32)).to(DEV)
    x = x.bfloat16() if bf16 else x
    h = x[:, 1:1 + H * D].unflatten(1, (H, D))
    before, sides = h.clone(), x[:, [0, -2, -1]].clone()
    cos, sin = synth.rope_tables(500, d_rope)
    pos = r.integers(0, 500, T).astype(np.int32)
    t = lambda a: torch.from_numpy(a).to(DEV)
    y = csa2.rope(h, t(pos), t(cos), t(sin), interleaved=interleaved, first=first)
    assert torch.equal(h, before)
    ref = rows.rope(c(before.double()), pos, cos, sin, interleaved, False, first)
    mag = np.maximum(*(rows.rope(np.abs(c(before.double())), pos, np.abs(cos), s * np.abs(sin), interleaved, False, first)
                       for s in (-1, 1)))
    # two products and a sum, then the type; what does not turn is copied
    tol = mag * 2 * U * 1.001 + np.abs(ref) * (U + (UB if bf16 else 0))
    assert (np.abs(c(y.double()) - ref) <= tol * (1 + UB)).all()
    assert torch.equal(y[..., :first], before[..., :first])
    assert torch.equal(y[..., first + d_rope:], before[..., first + d_rope:])
    assert csa2.rope(h, t(pos), t(cos), t(sin), interleaved=interleaved, first=first, out=h) is h
    assert torch.equal(h, y) and torch.equal(x[:, [0, -2, -1]], sides)
    assert csa2.device_error() == 0
