"""Decode attention's error against that of its output's own rounding.

The root mean square of y - (float64 result) is compared with the rounding of that
result to fp16, which no kernel can avoid.  What the kernel's arithmetic adds is
independent of it, so an addition of up to 0.4 of it leaves the sum within
sqrt(1 + 0.4^2) < 1.1 of the rounding alone.
"""
import numpy as np
import pytest
import torch

from int4_linear_b200 import fq
from oracle import kv_oracle as KO
from tests.test_kv_gpu import attn_case, run_attn

pytestmark = pytest.mark.gpu

HEADS = [(8, 2), (12, 2), (32, 2)]   # up to 4, up to 8, more query heads per key-value head


def error_over_rounding(y, ref):
    """rms(y - ref) over rms(fp16(ref) - ref)."""
    d = y.cpu().numpy().astype(np.float64).reshape(ref.shape) - ref
    r = ref.astype(np.float16).astype(np.float64) - ref
    assert np.isfinite(d).all()
    return np.sqrt((d ** 2).mean() / (r ** 2).mean())


@pytest.mark.parametrize("hq,h", HEADS)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("outlier", [1, 30, 100])
def test_queries_with_an_outlier_channel(hq, h, page, outlier):
    """A query channel `outlier` times the others' size, which the keys hardly use.  Values of at least 2^-11 of a
    head's largest enter exactly, smaller ones within 2^-22 of it (evenly spread: rms 2^-22 / sqrt(3)).  With codes of rms
    sqrt((8^2 + ... + 7^2) / 16) = 4.64, K scales of rms 0.25, scale 128^-0.5 and a largest value of at most 4.5 x 100, all
    128 channels among the smaller ones, a score is off by 450 2^-22 / sqrt(3) sqrt(128) 4.64 0.25 / sqrt(128) = 7.2e-5
    (rms), each weight by that much of itself, and the output of independent values by that much of its own size: 0.35 of
    the rounding of fp16 numbers (2^-11 / sqrt(3) of the power of two below them, i.e. over 0.73 of 2^-11 / sqrt(3) =
    2.05e-4 of them).  The float32 roundings of a score are below 2^-21 of its terms."""
    q, lens, table, pool = attn_case(31, [1000, 77, 4000], hq, h, page)
    q[..., 6] *= np.float16(outlier)
    if outlier > 1:
        kq, _, _, _ = KO.views(pool)
        kq[..., 3] &= 0xF0                       # channel 6: code 0
    ref = KO.attention(q, lens, table, pool, 128 ** -0.5)[0]
    assert error_over_rounding(run_attn(q, lens, table, pool), ref) <= 1.1


@pytest.mark.parametrize("hq,h", HEADS)
def test_scores_that_spread_widely(hq, h):
    """Ordinary heads whose scores have a standard deviation of about 14.  Queries: 54 2^-22 / sqrt(3) of at most
    4.64 0.25 sqrt(128) / sqrt(128) each, 9e-6; a score of up to 90 (in powers of two) is rounded three times and once
    less its reference, 4 x 90 x 2^-24 / sqrt(3) = 1.3e-5: below 0.1 of the output's rounding."""
    q, lens, table, pool = attn_case(32, [2000, 300, 5000], hq, h, 32, qstd=12.0)
    ref = KO.attention(q, lens, table, pool, 128 ** -0.5)[0]
    assert error_over_rounding(run_attn(q, lens, table, pool), ref) <= 1.1


@pytest.mark.parametrize("hq,h", [(32, 8), (64, 8), (128, 8)])
def test_long_parts_have_no_bias(hq, h):
    """512 requests of 131072 tokens and 8 heads: some 227 thousand tokens (up to 8 query heads; twice that with more) for
    each of the GPU's warps.  All tables name the same 64 pages again and again, so that the result is that of one round of
    them.  Values are positive, so cutting sums off instead of rounding them would make every output smaller.
    The mean of a request's outputs, relative to theirs: n = 14188 (twice that) rounded additions of a softmax
    sum in each of the 8 lanes that share a head, 2^-24 / sqrt(3) each (rms), the same in every round of 512 different ones,
    are n 2^-24 / (sqrt(3) sqrt(512)) of a lane's sum and that over sqrt(8 hq) in the mean (an output's own sums take half as many,
    and 128 outputs a head: less than a sixth of it); the outputs' roundings are 2^-11 / sqrt(3) at most over
    sqrt(128 hq).  Four times both."""
    page, pages, r, n = 128, 64, 512, 131072
    q, lens, table, pool = attn_case(33, [pages * page], hq, h, page)
    _, vq, _, _ = KO.views(pool)
    vq &= 0x77                                   # codes 0 to 7
    ref = KO.attention(q, lens, table, pool, 128 ** -0.5)[0]
    period = table[0, :pages]
    long_table = np.tile(period, (r, n // (pages * page)))
    y = run_attn(np.repeat(q, r, 0), np.full(r, n, np.int32), long_table, pool)
    y = y.cpu().numpy().astype(np.float64).reshape(r, hq, 128)
    bias = (y - ref).mean((1, 2)) / ref.mean()
    adds = 14188 * (2 if hq > 64 else 1)
    sums = adds * 2.0 ** -24 * np.sqrt(512 / 3) / 512 / np.sqrt(8 * hq) * 7 / 6
    assert np.abs(bias).max() <= 4 * (sums + 2.0 ** -11 / np.sqrt(3) / np.sqrt(128 * hq))


def large_value_scale(hq, h, page, at, log2_ratio):
    """A case whose requests hold one token, number `at`, with a V scale of 2^15, 2^log2_ratio times the most that the others
    have, and a score some 85 below them (query channel 6 is 30, and only that token's key uses it): its weight times its
    scale is 2^-107, nothing beside theirs."""
    q, lens, table, pool = attn_case(34, [40, 700, 33], hq, h, page)
    q[..., 6] = 30
    kq, _, ks, vs = KO.views(pool)
    kq[..., 3] &= 0xF0
    vs *= np.float16(2.0 ** (13 - log2_ratio))   # from 0.05 .. 0.4 to below 2^(15 - log2_ratio)
    for i, n in enumerate(lens):
        t = at % n
        pg, off = table[i, t // page], t % page
        kq[pg, :, off] = 0
        kq[pg, :, off, 3] = 8                    # code -8
        ks[pg, :, off] = 4.0
        vs[pg, :, off] = 2.0 ** 15
    return q, lens, table, pool


@pytest.mark.parametrize("hq,h", HEADS)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("at", [0, 20, -1])
@pytest.mark.parametrize("log2_ratio", [14, 18, 20, 23])
def test_one_large_value_scale_without_weight(hq, h, page, at, log2_ratio):
    """The weights of the other tokens are within 2^-22 of themselves, or 2^-33 of the largest p times (v scale)."""
    q, lens, table, pool = large_value_scale(hq, h, page, at, log2_ratio)
    ref = KO.attention(q, lens, table, pool, 128 ** -0.5)[0]
    assert np.sqrt((ref ** 2).mean()) > 2.0 ** -13   # fp16's normal range
    assert error_over_rounding(run_attn(q, lens, table, pool), ref) <= 1.1


def gaussian_case(seed, lens, hq, h, page):
    """Keys and values as fq_kv_write caches Gaussian ones, some key channels three times the others; queries of
    standard deviation 1.5: scores of some 1.8."""
    g = np.random.Generator(np.random.PCG64([seed, hq, h, page]))
    q, lens, table, pool = attn_case(seed, lens, hq, h, page)
    n = sum(lens)
    x = g.standard_normal((2, n, h, 128)).astype(np.float32)
    x[0, ..., ::16] *= 3
    slots = [table[i, t // page] * page + t % page for i, m in enumerate(lens) for t in range(m)]
    KO.store(pool, *KO.quant_rows(x[0]), *KO.quant_rows(x[1]), np.array(slots))
    return (q.astype(np.float32) * 1.5).astype(np.float16), lens, table, pool


@pytest.mark.parametrize("hq,h", HEADS)
@pytest.mark.parametrize("page", [16, 64])
def test_ordinary_heads(hq, h, page):
    """A turn's at most 68 terms are cut off at 2^-23 of the largest one, at most 8 times the largest weight: sqrt(68 / 3)
    2^-23 8 = 4.6e-6 of that weight (rms).  An output of values of rms 2.3 or more (the codes of Gaussian vectors, whose
    largest is 7) is at least 2.3 times the root of the weights' squares, so the cuts are 2e-6 of it.  Four float32
    roundings of scores below 16 (in powers of two) and an exponential within 2^-22 are 1e-6 of each weight.  Together
    e = 3e-6 / 2.05e-4 = 0.015 of the output's rounding: sqrt(1 + e^2), and four standard deviations 2 e / sqrt(n) of the chance
    products of both for n >= 2048 outputs: 1.0001 + 0.0027."""
    q, lens, table, pool = gaussian_case(35, [1000, 8000], hq, h, page)
    ref = KO.attention(q, lens, table, pool, 128 ** -0.5)[0]
    assert error_over_rounding(run_attn(q, lens, table, pool), ref) <= 1.0028
