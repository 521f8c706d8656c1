"""The row operators around the hot path: residual addition with a root-mean-square norm, rotary
positions and their tables, FP4 rows with a scale of the whole matrix, and their product.

Test infrastructure (see oracle/__init__.py).  The pages name none of these steps' details; the
definitions are those of include/csa2.h.  Steps that decide codes are float32 operations (each
correctly rounded), as in formats.py; everything else is float64.
"""
import math

import numpy as np

from . import formats


def add(x, residual, bf16):
    """h = x + residual in float32, rounded to bf16 where the residual stream is bf16."""
    h = (np.asarray(x, np.float32) + np.asarray(residual, np.float32)).astype(np.float32)
    return formats.bf16_value(formats.bf16_round(h)).astype(np.float32) if bf16 else h


def rms_norm_f32(h, weight, eps):
    """y in the float32 steps of the definition; the mean is rounded once from float64."""
    h = np.asarray(h, np.float32)
    ms = np.mean(h.astype(np.float64) ** 2, axis=-1, keepdims=True).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = (np.float32(1) / np.sqrt(ms + np.float32(eps))).astype(np.float32)
        y = (h * r).astype(np.float32)
        return y if weight is None else (y * np.asarray(weight, np.float32)).astype(np.float32)


def rms_norm(h, weight, eps):
    """The norm in float64."""
    h = np.asarray(h, np.float64)
    y = h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps)
    return y if weight is None else y * np.asarray(weight, np.float64)


def fp8_groups(y, group):
    """E4M3 bytes and one float32 scale per `group` channels (0: the row), the last group may be
    short: formats.fp8_rows_quantize of each."""
    D = y.shape[-1]
    n = group or D
    parts = [formats.fp8_rows_quantize(y[:, a:a + n]) for a in range(0, D, n)]
    return np.concatenate([b for b, _ in parts], axis=1), np.stack([s for _, s in parts], axis=1)


def frequencies(d_rope, theta=10000.0, scaling="none", factor=1.0, orig=0, beta_fast=32.0, beta_slow=1.0):
    i = np.arange(d_rope // 2, dtype=np.float64)
    f = theta ** (-2 * i / d_rope)
    if scaling == "linear":
        return f / factor
    if scaling == "yarn":
        def channel(turns):
            return d_rope * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo = max(math.floor(channel(beta_fast)), 0)
        hi = min(math.ceil(channel(beta_slow)), d_rope - 1)
        slow = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return f / factor * slow + f * (1 - slow)
    return f


def rope(x, pos, cos, sin, interleaved, inverse, first):
    """x [T, H, D] float64; cos, sin [positions, d_rope/2]; the channels from `first` on turn."""
    x = np.asarray(x, np.float64)
    c, s = cos[pos].astype(np.float64)[:, None], sin[pos].astype(np.float64)[:, None]
    s = -s if inverse else s
    n = cos.shape[1]
    a = first + (2 * np.arange(n) if interleaved else np.arange(n))
    b = a + (1 if interleaved else n)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def scale_tiles(scales):
    """Scale bytes [R, C] in tiles [ceil(R/128), ceil(C/4), 512], byte by byte, zero elsewhere."""
    R, C = scales.shape
    t = np.zeros((-(-R // 128), -(-C // 4), 512), np.uint8)
    for r in range(R):
        for c in range(C):
            t[r // 128, c // 4, (r % 32) * 16 + (r % 128 // 32) * 4 + c % 4] = scales[r, c]
    return t


def fp4_quantize(x, gscale=None):
    """formats.fp4_quantize of x / gscale (float32 division)."""
    u = np.asarray(x, np.float32)
    return formats.fp4_quantize(u if gscale is None else (u / np.float32(gscale)).astype(np.float32))


def fp4_linear(xc, xs, wc, ws, gx=1.0, gw=1.0):
    """(the product, the same sum over magnitudes) in float64."""
    x, w = formats.fp4_dequantize(xc, xs), formats.fp4_dequantize(wc, ws)
    g = float(np.float32(gx)) * float(np.float32(gw))
    return g * (x @ w.T), abs(g) * (np.abs(x) @ np.abs(w).T)
