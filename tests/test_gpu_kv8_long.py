"""Attention over the paged 8-bit cache at up to 2^20 tokens, in float32, against 64 bits: what a long stream loses must not
grow with its length.  All sequences have the same few pages over and over, and there are as many (sequence, key head)
pairs as spans of the work, so that a span holds one whole stream (a stream that is cut has its parts summed apart)."""
import numpy as np
import pytest
import torch

from fp4_compressed_sparse_02_gb300 import csa2
from kv8_utils import DEV, bf16, gpu
from oracle.formats import e4m3_encode, e4m3_value

pytestmark = pytest.mark.gpu
D, KINDS = 64, 41
# (key heads, query heads a key head, new tokens, max_new): 19 sequences; streams of 8 rows, of 16, tiles of 64, 128 and 256 rows
FORMS = {"8 rows": (64, 1, 1, 1), "16 rows": (64, 12, 1, 1), "64 rows": (8, 8, 3, 3), "128 rows": (8, 16, 6, 6), "256 rows": (8, 8, 3, 100)}


def step(form, n, lead, sink_value, seed=0):
    """19 sequences of n tokens whose first token leads the others by about `lead` nats and has values `sink_value`; the
    others' values lie in 0.5 .. 5.  Yields (error of out / |out|, error of lse, the logits' error bound, sum of values /
    (sum of weights x |out|), the largest weight being 1), for every row of the first and the last sequence."""
    H, G, new, hint = FORMS[form]
    S = 19
    r = np.random.default_rng(seed)
    u = np.where(r.random(D) < 0.5, -1.0, 1.0)
    k = e4m3_encode(r.standard_normal((KINDS, H, 64, D))).astype(np.uint8)
    v = e4m3_encode(np.abs(r.standard_normal((KINDS, H, 64, D))) + 0.5).astype(np.uint8)
    k[0, :, 0], v[0, :, 0] = e4m3_encode(8 * u), e4m3_encode(np.full(D, sink_value))
    table = np.concatenate(([0], r.integers(1, KINDS, -(-n // 64) - 1))).astype(np.int32)
    ones = np.ones((KINDS, H), np.float32)
    # q . k_sink / sqrt(D) = lead on average: all elements of q are of one size, which two E4M3 numbers hold exactly
    q = bf16(u * (lead / 64) * (1 + 0.27 * r.standard_normal((S * new, H * G, D))))
    cache = csa2.Kv8Cache(gpu(k), gpu(v), gpu(ones), gpu(ones), gpu(table)[None].expand(S, -1).contiguous())
    csa2.device_error()
    out, lse = csa2.kv8_attn(cache, gpu(q, torch.bfloat16), gpu(np.arange(S + 1, dtype=np.int32) * new),
                             gpu(np.full(S, n, np.int32)), max_new=hint, out_dtype=torch.float32)
    assert csa2.device_error() == 0
    kd, vd, pages = gpu(e4m3_value(k)), gpu(e4m3_value(v)), gpu(table).long()
    for t in [*range(new), *range((S - 1) * new, S * new)]:
        seen = n - new + t % new + 1
        times = torch.zeros((KINDS, 64), dtype=torch.float64, device=DEV)     # how often the row sees each token
        times += torch.bincount(pages[:seen // 64], minlength=KINDS)[:, None]
        if seen % 64:
            times[pages[seen // 64], :seen % 64] += 1
        x = torch.einsum("hgd,phtd->hgpt", gpu(q[t].reshape(H, G, D).astype(np.float64)), kd) * D ** -0.5
        top = x.amax((2, 3), keepdim=True)
        p = torch.exp(x - top) * times
        z = p.sum((2, 3))
        want = torch.einsum("hgpt,phtd->hgd", p, vd) / z[..., None]
        got = out[t].reshape(H, G, D).double()
        # D + 8 roundings of a logit's sum
        e = (D + 8) * 2.0 ** -24 * float((gpu(np.abs(q[t]).reshape(H, G, D).astype(np.float64)).sum(-1).amax() * 8) * D ** -0.5)
        values = torch.einsum("pt,phtd->hd", times, vd)[:, None] / (z[..., None] * want)
        yield (got - want) / want, lse[t].reshape(H, G).double() - (top[..., 0, 0] + z.log()), e, values


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("lead", [17, 18, 20])
def test_sum_of_small_weights_beside_a_large_one(form, lead):
    """The logarithm of the sum.  A sum of sums: at most 2^10 terms one after the other at either level, each half a step of
    float32 (2^-24) off, relative to the whole; 2^-16 for the exponentials, the logarithm and the merging, 2^-21 for
    the result's own size."""
    for _, err, e, _ in step(form, (1 << 20) - 5, lead, 0.0):
        assert float(err.abs().max()) <= e + 2 * 2.0 ** -14 + 2.0 ** -16 + 2.0 ** -21 * (lead + 2), float(err.abs().max())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n", [(1 << 14) - 3, 1 << 15, (1 << 15) + 130, 1 << 16, (1 << 16) + 1, (1 << 17) + 300, (1 << 20) - 5])
def test_sums_of_many_values_of_one_sign(form, n):
    """The output where nothing cancels: weights in fp16 (2^-11), 2^-14 for the exponentials, the logits twice, the sum as
    above.  Tiles: the tensor core cuts sums off rather than rounding them, at most a unit of 2^-23 for each of eight products a step,
    of 256 steps: 2^-12.  Streams: up to 2^15 additions, each half a step off either way: six standard deviations of
    their sum, 6 x 2^7.5 x 2^-24 / sqrt(3) < 2^-14."""
    for err, _, e, _ in step(form, n, 2, 1.0):
        assert float(err.abs().max()) <= 2.0 ** -11 + 2.0 ** -14 + 2 * e + 2 * 2.0 ** -14 + 2.0 ** -12, (float(err.mean()), float(err.abs().max()))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n", [1 << 12, (1 << 20) - 5])
@pytest.mark.parametrize("lead", [12, 15, 17, 18, 20, 22])
def test_values_of_small_weights_beside_a_large_one(form, n, lead):
    """The first token has the largest weight by far and values of zero: the output is the others' alone.  The bound is that of
    the sums above, and 2^-40 (tiles 2^-36) of the largest weight for each other one, where fp16 ends."""
    least = 2.0 ** -40 if form in ("8 rows", "16 rows") else 2.0 ** -36
    for err, _, e, values in step(form, n, lead, 0.0):
        bound = 2.0 ** -11 + 2.0 ** -14 + 2 * e + 2 * 2.0 ** -14 + 2.0 ** -12 + least * values
        assert bool((err.abs() <= bound).all()), (float(err.abs().max()), float((err.abs() / bound).max()))
