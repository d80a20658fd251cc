"""The paged INT4 cache on the GPU against the oracle.

Block tables, slots, codes, scales and what is read back are whole numbers or
single roundings: compared bit for bit.

Attention.  Per output, with p the exact weights and v the cached values:
* the queries enter as 16-bit fixed point, half a step of qmax / 65278 off each,
  and the integer sums are exact: |ds| <= scale (qmax / 65278) sum|k| <= scale (qmax / 65278) 128 * 8 ks,
  ks the largest K scale, and four float32 roundings of the score; the softmax
  then moves each weight by a factor within exp(+-2 |ds|), the output by at
  most (exp(2 |ds|) - 1) sum p|v|;
* a weight enters as two fp16 numbers (2^-22 relative), its two exponentials and
  products are float32 (16 * 2^-24 taken): (2^-22 + 2^-20) sum p|v|, and 2^-33 of the
  largest for each of n weights whose second number is subnormal: n 2^-33 max|v|;
* the codes are summed as code + 8 and 8 sum(w) is taken off, 32 tokens at a
  time in two products of 16 tokens: 2 * 17 terms of at most 16 (their weights' sum) vs
  each, the sum so far among them, cut at 2^-23 of the largest, i.e. at most 34 * 16 * 2^-23 vs
  in all (all weights sum to 1), vs the largest V scale; the
  float32 sums over n tokens add n 2^-24 sum p|v| at most;
* the output's own rounding: 2^-11 |y|, and 2^-25 below fp16's normal range.
On top of these worst cases the roundings of the output are independent, so the
root mean square of the error stays under 2^-11 of the root mean square of y (it
is at most 2^-11 / sqrt(3) of it), plus the score's error with its 128 terms
taken as independent.
"""
import numpy as np
import pytest
import torch

from int4_linear_b200 import fq
from oracle import kv_oracle as KO

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rng(*seed):
    return np.random.Generator(np.random.PCG64(list(seed)))


# ---------------------------------------------------------------- block tables and slots

def _plan_case(seed, r, page, max_pages, prompts, new_hi, spare):
    g = rng(seed, r, page)
    lens = g.integers(0, page * max_pages, r).astype(np.int32)
    new = np.ones(r, np.int32)
    if prompts:
        who = g.permutation(r)[:prompts]
        new[who] = g.integers(0, new_hi + 1, prompts)
    held = -(-lens // page)
    need = int((-(-(lens + new) // page) - held).sum())
    ids = g.permutation(int(held.sum()) + max(need, 0) + 8).astype(np.int32)
    table = np.full((r, max_pages), -7, np.int32)
    o = 0
    for i in range(r):
        table[i, :held[i]] = ids[o:o + held[i]]
        o += held[i]
    free = np.concatenate([[-9, -9], ids[o:o + max(0, need + spare)]]).astype(np.int32)
    return lens, new, table, free


@pytest.mark.parametrize("r,page,max_pages,prompts,new_hi,spare", [
    (1, 16, 4, 0, 0, 3), (1, 128, 3, 1, 300, 2), (5, 16, 8, 2, 90, 0), (33, 32, 9, 5, 200, 4),
    (33, 32, 9, 12, 200, -3), (64, 16, 64, 0, 0, 1), (64, 16, 64, 0, 0, -4), (1023, 64, 20, 40, 700, 2),
    (1024, 64, 20, 40, 700, -50), (1025, 16, 30, 3, 17, 9), (2100, 16, 30, 30, 400, 1), (16384, 16, 5, 200, 70, -100)])
@pytest.mark.parametrize("cut", [0, 11])
def test_plan(r, page, max_pages, prompts, new_hi, spare, cut):
    lens, new, table, free = _plan_case(7, r, page, max_pages, prompts, new_hi, spare)
    total = int(new.sum())
    max_tokens = max(0, total - cut) if cut else total + 13
    want_table = table.copy()
    out, start, slots, used = KO.plan(lens, new, want_table, free, 2, page, max_tokens)
    t = dev(table)
    g_len, g_start, g_slots, g_used = fq.fq_kv_plan(dev(lens), dev(new), t, dev(free),
                                                    torch.full((1,), 2, dtype=torch.int32, device="cuda"), page,
                                                    max_tokens)
    assert np.array_equal(g_len.cpu().numpy(), out)
    assert np.array_equal(g_start.cpu().numpy(), start)
    assert np.array_equal(g_slots.cpu().numpy(), slots)
    assert np.array_equal(t.cpu().numpy(), want_table)
    assert int(g_used) == int(used[0])


def test_plan_steps_in_place_and_captured():
    """Ten decode steps with lens and pages_used updated in place, the call captured once and replayed."""
    page, r, max_pages = 16, 37, 6
    lens, new, table, free = _plan_case(3, r, page, 3, 0, 0, 60)
    table = np.concatenate([table, np.full((r, 3), -7, np.int32)], 1)
    d = dict(lens=dev(lens), new=dev(new), table=dev(table), free=dev(free),
             used=torch.full((1,), 2, dtype=torch.int32, device="cuda"),
             start=torch.empty(r + 1, dtype=torch.int32, device="cuda"),
             slots=torch.empty(r, dtype=torch.int32, device="cuda"))

    def step():
        fq.fq_kv_plan(d["lens"], d["new"], d["table"], d["free"], d["used"], page, r, lens_out=d["lens"],
                      token_start=d["start"], slots=d["slots"], pages_used_out=d["used"])

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    saved = {k: v.clone() for k, v in d.items()}
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        step()
    for k, v in saved.items():
        d[k].copy_(v)
    used = 2
    for _ in range(10):
        graph.replay()
        lens, _, slots, u = KO.plan(lens, new, table, free, used, page, r)
        used = int(u[0])
        assert np.array_equal(d["lens"].cpu().numpy(), lens)
        assert np.array_equal(d["slots"].cpu().numpy(), slots)
        assert np.array_equal(d["table"].cpu().numpy(), table)
        assert int(d["used"]) == used


def test_plan_without_free_pages_and_negative_counts():
    """No free list at all; negative counts are 0."""
    lens, new = np.array([-3, 5, 16], np.int32), np.array([0, -2, 1], np.int32)
    table = np.array([[4, 4], [5, 5], [6, 6]], np.int32)
    want = table.copy()
    out, start, slots, used = KO.plan(lens, new, want, [], 0, 16, 4)
    t = dev(table)
    res = fq.fq_kv_plan(dev(lens), dev(new), t, torch.empty(0, dtype=torch.int32, device="cuda"),
                        torch.zeros(1, dtype=torch.int32, device="cuda"), 16, 4)
    for a, b in zip(res, (out, start, slots, used)):
        assert np.array_equal(a.cpu().numpy(), b)
    assert np.array_equal(t.cpu().numpy(), want)


# ---------------------------------------------------------------- into and out of the pages

@pytest.mark.parametrize("t,h,page", [(1, 1, 16), (3, 5, 32), (7, 8, 64), (129, 3, 128), (200, 128, 16), (4097, 2, 16)])
@pytest.mark.parametrize("alpha", [1.0, 0.83])
def test_write_and_read_bits(t, h, page, alpha):
    g = rng(1, t, h)
    x = g.standard_normal((2, t, h, 128)).astype(np.float16)
    x[0, ::3] *= np.float16(2.0 ** -14)          # fp16 subnormal values and scales
    x[1, 1::4] *= np.float16(900)
    x[0, t // 2] = 0                             # a head vector of zeros
    x[1, t // 2, 0] = np.float16(2.0 ** -24)     # its scale rounds to zero
    # quotients on a tie: scale 1 exactly, values k + 1/2
    if alpha == 1.0:
        x[0, -1] = ((np.arange(128) % 15) - 7).astype(np.float16) / 2
        x[0, -1, :, 0] = 7
    pages = -(-t // page) + 3
    slots = g.permutation(pages * page)[:t].astype(np.int32)
    if t > 2:
        slots[t // 3] = -1
        slots[t // 3 + 1] = pages * page
    pool = g.integers(0, 256, (pages, h, page * 132)).astype(np.uint8)   # what was there stays
    want = pool.copy()
    kq, ks = KO.quant_rows(x[0], alpha)
    vq, vs = KO.quant_rows(x[1], np.float32(0.9) * np.float32(alpha))
    KO.store(want, kq, ks, vq, vs, slots)
    cache = fq.KVCache(dev(pool))
    # rows of one wider buffer, as slices of a projection's output
    buf = torch.zeros(t, 2 * h * 128 + 24, dtype=torch.float16, device="cuda")
    buf[:, 8:8 + h * 128] = dev(x[0].reshape(t, -1))
    buf[:, 16 + h * 128:16 + 2 * h * 128] = dev(x[1].reshape(t, -1))
    sl = dev(slots)
    fq.fq_kv_write(buf[:, 8:8 + h * 128], buf[:, 16 + h * 128:16 + 2 * h * 128], sl, cache, alpha,
                   float(np.float32(0.9) * np.float32(alpha)))
    assert np.array_equal(cache.pool.cpu().numpy(), want)
    k, v = fq.fq_kv_read(cache, sl)
    ok = (slots >= 0) & (slots < pages * page)
    for got, q, s in ((k, kq, ks), (v, vq, vs)):
        ref = np.where(ok[:, None, None], q.astype(np.float32) * s.astype(np.float32)[..., None], 0).astype(np.float16)
        got = got.cpu().numpy()
        assert np.array_equal(got, ref)


@pytest.mark.parametrize("t,h", [(9001, 5), (20011, 3), (700, 127)])
def test_many_head_vectors(t, h):
    """Several turns of every thread, whose tokens and heads step on by other than whole tokens: written, read
    and stored again."""
    g = rng(14, t, h)
    page = 32
    x = g.standard_normal((2, t, h, 128)).astype(np.float16)
    pages = -(-t // page) + 1
    slots = g.permutation(pages * page)[:t].astype(np.int32)
    kq, ks = KO.quant_rows(x[0], 1.0)
    vq, vs = KO.quant_rows(x[1], 1.0)
    want = KO.empty_pool(pages, h, page)
    KO.store(want, kq, ks, vq, vs, slots)
    cache, sl = fq.kv_cache(pages, h, page), dev(slots)
    fq.fq_kv_write(dev(x[0]), dev(x[1]), sl, cache)
    assert np.array_equal(cache.pool.cpu().numpy(), want)
    for got, q, s in zip(fq.fq_kv_read(cache, sl), (kq, vq), (ks, vs)):
        assert np.array_equal(got.cpu().numpy(), (q.astype(np.float32) * s.astype(np.float32)[..., None]).astype(np.float16))
    views = [v.permute(0, 2, 1, 3) if v.dim() == 4 else v.permute(0, 2, 1) for v in cache.views()]
    rows = [v.reshape(pages * page, h, -1)[sl.long()] for v in views]
    again = fq.kv_cache(pages, h, page)
    fq.fq_kv_store(rows[0].reshape(t, h * 64), rows[2].reshape(t, h), rows[1].reshape(t, h * 64), rows[3].reshape(t, h),
                   sl, again)
    assert torch.equal(again.pool, cache.pool)


def test_store_of_transformed_codes():
    """fq_quant_kv's codes through P_h, then fq_kv_store: the pages hold the same bytes."""
    g = rng(4)
    t, h, page = 37, 4, 32
    p = np.linalg.qr(g.standard_normal((128, 128)))[0].astype(np.float32)
    x = dev(g.standard_normal((2, t, h, 128)).astype(np.float16))
    kq, ks = fq.fq_quant_kv(x[0].contiguous(), dev(p))
    vq, vs = fq.fq_quant_kv(x[1].contiguous(), dev(p.T))
    slots = g.permutation(4 * page)[:t].astype(np.int32)
    slots[5] = -1
    cache = fq.kv_cache(4, h, page)
    fq.fq_kv_store(kq, ks, vq, vs, dev(slots), cache)
    want = KO.empty_pool(4, h, page)
    from oracle import fq_oracle as O
    un = lambda q: O.unpack_int4(q.cpu().numpy().reshape(-1, 64)).reshape(t, h, 128)
    KO.store(want, un(kq), ks.cpu().numpy(), un(vq), vs.cpu().numpy(), slots)
    assert np.array_equal(cache.pool.cpu().numpy(), want)
    a, b = cache.views()[0], KO.views(want)[0]
    assert np.array_equal(a.cpu().numpy(), b)


# ---------------------------------------------------------------- attention

def make_pool(g, pages, heads, page, spread=1.0):
    pool = np.zeros((pages, heads, page * 132), np.uint8)
    n = page
    pool[:, :, :128 * n] = g.integers(0, 256, (pages, heads, 128 * n))
    ks = (g.uniform(0.05, 0.4, (pages, heads, n))).astype(np.float16)
    vs = (g.uniform(0.05, 0.4, (pages, heads, n)) * spread ** g.uniform(-1, 1, (pages, heads, n))).astype(np.float16)
    pool[:, :, 128 * n:130 * n] = ks.view(np.uint8)
    pool[:, :, 130 * n:] = vs.view(np.uint8)
    return pool


def attn_case(seed, lens, hq, h, page, spread=1.0, extra_pages=2, qstd=1.0):
    g = rng(seed, len(lens), hq, h, page)
    held = [-(-max(n, 0) // page) for n in lens]
    pages = sum(held) + extra_pages
    pool = make_pool(g, pages, h, page, spread)
    ids = g.permutation(pages).astype(np.int32)
    max_pages = max(max(held), 1) + 1
    table = np.full((len(lens), max_pages), -1, np.int32)
    o = 0
    for i, c in enumerate(held):
        table[i, :c] = ids[o:o + c]
        o += c
    # NaN and Inf scales behind every last token
    _, _, ks, vs = KO.views(pool)
    for i, n in enumerate(lens):
        if n > 0 and n % page:
            pg = table[i, n // page]
            pool[pg, :, 128 * page + 2 * (n % page):130 * page] = 0xFF
            pool[pg, :, 130 * page + 2 * (n % page):] = np.tile(np.array([0x00, 0x7C], np.uint8), page - n % page)
    q = (g.standard_normal((len(lens), hq, 128)) * qstd).astype(np.float16)
    return q, np.asarray(lens, np.int32), table, pool


def check_attn(y, q, lens, table, pool, scale, window=0):
    ref, sa, sq, kmax = KO.attention(q, lens, table, pool, scale, window)
    y = y.cpu().numpy().astype(np.float64).reshape(ref.shape)
    qm, qa = np.abs(q.astype(np.float64)).max(-1), np.abs(q.astype(np.float64)).sum(-1)
    # the oracle's max|k| / 4 is at least 2 ks when a code is 8 or -8, and ks from codes of 4 on
    ks = kmax[:, None] * abs(scale)
    ds = qm / 65278 * 128 * 8 * ks + 4 * 2.0 ** -24 * 8 * qa * ks
    n = min(max(int(max(lens)), 1), table.shape[1] * (pool.shape[2] // 132))
    vs = KO.views(pool)[3].astype(np.float64)
    vmax = 8 * np.abs(vs[np.isfinite(vs)]).max()
    tol = (np.expm1(2 * ds)[..., None] + 2.0 ** -22 + 2.0 ** -20 + n * 2.0 ** -24) * sa
    tol += (n * 2.0 ** -33 + 34 * 16 * 2.0 ** -23 / 8) * vmax + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
    err = np.abs(y - ref)
    assert np.isfinite(y).all()
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3f} of the bound"
    dr = qm / 65278 / np.sqrt(3) * np.sqrt(128) * 8 * ks
    rms = np.sqrt((ref ** 2).mean()) * 2.0 ** -11 + np.sqrt(((2 * dr[..., None] * sq) ** 2).mean())
    assert np.sqrt((err ** 2).mean()) <= rms + 2.0 ** -25, (np.sqrt((err ** 2).mean()), rms)


def run_attn(q, lens, table, pool, scale=128 ** -0.5, window=0, **kw):
    y = fq.fq_kv_attn(dev(q), dev(lens), dev(table), fq.KVCache(dev(pool)), scale=scale, window=window, **kw)
    fq.fq_check_device_error()
    return y


LENS = [[1], [0], [15, 16, 17], [63, 64, 65, 0, 127, 128, 129], [1000], [300, 0, 4097, 1, 64]]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("lens", LENS)
def test_attn_lengths(lens, page):
    case = attn_case(1, lens, 8, 2, page)
    check_attn(run_attn(*case), *case, 128 ** -0.5)


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("lens", LENS)
def test_attn_lengths_with_six_queries_a_head(lens, page):
    case = attn_case(1, lens, 12, 2, page)
    check_attn(run_attn(*case), *case, 128 ** -0.5)


@pytest.mark.parametrize("hq,h", [(4, 1), (6, 1), (12, 1), (16, 4)])
@pytest.mark.parametrize("page", [16, 64])
def test_attn_long_head_layouts(hq, h, page):
    case = attn_case(12, [9001, 1, 333], hq, h, page)
    check_attn(run_attn(*case), *case, 128 ** -0.5)


@pytest.mark.parametrize("hq,h", [(4, 2), (8, 2), (16, 2), (32, 2)])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_attn_queries_that_are_not_finite(hq, h, bad):
    q, ln, table, pool = attn_case(13, [3000, 40, 0], hq, h, 32)
    good = run_attn(q, ln, table, pool)
    q[0, 1, 5] = q[1, hq - 1, 127] = q[2, 0, 0] = bad
    y = run_attn(q, ln, table, pool)
    hit = torch.zeros(3, hq, 1, dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[1, hq - 1] = True
    assert torch.equal(torch.isnan(y.view(3, hq, 128)), hit.expand(3, hq, 128))
    assert torch.equal(y.view(3, hq, 128)[~hit[..., 0]], good.view(3, hq, 128)[~hit[..., 0]])


@pytest.mark.parametrize("hq,h", [(1, 1), (2, 1), (3, 3), (5, 1), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 1),
                                  (32, 32), (24, 8), (128, 128), (71, 1), (64, 8), (36, 3)])
def test_attn_head_layouts(hq, h):
    case = attn_case(2, [200, 77, 513], hq, h, 32)
    check_attn(run_attn(*case), *case, 128 ** -0.5)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 65, 100, 1000, 5000])
@pytest.mark.parametrize("page", [16, 128])
def test_attn_window(window, page):
    lens = [1000, 64, 1, 0, 777]
    q, ln, table, pool = attn_case(3, lens, 12, 4, page)
    for i, n in enumerate(lens):                 # pages behind the window are gone
        table[i, :max(0, n - window) // page] = -1
    check_attn(run_attn(q, ln, table, pool, window=window), q, ln, table, pool, 128 ** -0.5, window)


def test_attn_long_split_over_every_sm():
    case = attn_case(4, [70001], 8, 1, 64)
    check_attn(run_attn(*case), *case, 128 ** -0.5)


def test_attn_many_short_requests():
    g = rng(5)
    lens = g.integers(0, 40, 700).tolist()
    case = attn_case(5, lens, 4, 2, 16)
    check_attn(run_attn(*case), *case, 128 ** -0.5)


@pytest.mark.parametrize("longest", [400, 9000])
@pytest.mark.parametrize("hq,h", [(2, 1), (12, 2)])
def test_attn_few_requests_among_many_empty_slots(longest, hq, h):
    """Every request and head whole on a CTA of its own, or, with a long one among them, divided."""
    g = rng(15)
    lens = np.zeros(3000, np.int64)
    lens[g.permutation(3000)[:140]] = g.integers(200, 400, 140)
    lens[g.integers(0, 3000)] = longest
    case = attn_case(15, lens.tolist(), hq, h, 32)
    check_attn(run_attn(*case), *case, 128 ** -0.5)


def test_attn_value_scales_of_every_magnitude():
    """V scales over eight decades within a request: the running reference moves."""
    case = attn_case(6, [900, 333], 8, 2, 16, spread=1e4)
    check_attn(run_attn(*case), *case, 128 ** -0.5)


@pytest.mark.parametrize("qstd,scale", [(0.0, 0.1), (20.0, 0.05), (1.0, 0.0), (1.0, -0.1), (1.0, 1.0)])
def test_attn_score_ranges(qstd, scale):
    """Equal scores, scores that leave one token, a zero and a negative scale."""
    case = attn_case(7, [500, 64], 8, 2, 32, qstd=qstd)
    check_attn(run_attn(*case, scale=scale), *case, scale)


def test_attn_growing_scores():
    """Every token's score passes the last one's: the reference moves all along."""
    q, lens, table, pool = attn_case(8, [640], 8, 1, 16)
    kq, _, ks, _ = KO.views(pool)
    for t in range(640):
        pg, off = table[0, t // 16], t % 16
        pool[pg, 0, 64 * off:64 * off + 64] = 0x77            # codes 7
        pool[pg, 0, 2048 + 2 * off:2048 + 2 * off + 2] = np.array([t / 64 + 0.01], np.float16).view(np.uint8)
    q = np.abs(q)
    check_attn(run_attn(q, lens, table, pool, scale=0.02), q, lens, table, pool, 0.02)


def test_attn_bad_table_entries_are_left_out():
    q, lens, table, pool = attn_case(9, [200, 64, 30], 4, 2, 16)
    table[0, 3], table[0, 7], table[1, :4], table[2, 0] = -1, pool.shape[0], -5, 1 << 30
    y = run_attn(q, lens, table, pool)
    check_attn(y, q, lens, table, pool, 128 ** -0.5)
    assert not y[1].any()


def test_attn_lengths_past_the_table_and_negative():
    q, lens, table, pool = attn_case(10, [64, 32, 16], 4, 2, 16)
    lens = np.array([1 << 30, -5, 16], np.int32)
    table = table[:, :4].copy()
    table[0] = [0, 1, 2, 3]
    check_attn(run_attn(q, lens, table, pool), q, lens, table, pool, 128 ** -0.5)


def test_attn_strided_queries_and_given_output():
    q, lens, table, pool = attn_case(11, [100, 200, 300], 8, 2, 16)
    buf = torch.full((3, 12 * 128), float("nan"), dtype=torch.float16, device="cuda")
    buf[:, 128:9 * 128] = dev(q.reshape(3, -1))
    y = torch.full((4, 8 * 128), 7.0, dtype=torch.float16, device="cuda")
    out = fq.fq_kv_attn(buf[:, 128:9 * 128], dev(lens), dev(table), fq.KVCache(dev(pool)), Y=y[:3])
    assert out.data_ptr() == y.data_ptr()
    check_attn(out, q, lens, table, pool, 128 ** -0.5)
    assert (y[3] == 7).all()


def test_attn_repeats_bit_for_bit_on_one_workspace():
    case = attn_case(12, [5000, 3, 0, 800], 32, 8, 64)
    args = [dev(a) for a in case[:3]] + [fq.KVCache(dev(case[3]))]
    ws = fq.fq_kv_attn_workspace(4, 32, 8)
    ws[fq.SYNC_BYTES:] = 0xA5
    first = fq.fq_kv_attn(*args, workspace=ws)
    for _ in range(20):
        assert torch.equal(fq.fq_kv_attn(*args, workspace=ws), first)
    assert not ws[:fq.SYNC_BYTES].any()
    check_attn(first, *case, 128 ** -0.5)


def test_attn_captured_follows_the_lengths_on_a_shared_workspace():
    """Two captured calls share a workspace; each replay follows the lengths it finds."""
    q, lens, table, pool = attn_case(13, [900, 900, 900], 16, 2, 32)
    dq, dl, dt, dc = dev(q), dev(lens), dev(table), fq.KVCache(dev(pool))
    ws = fq.fq_kv_attn_workspace(3, 16, 2)
    ys = [torch.empty(3, 16 * 128, dtype=torch.float16, device="cuda") for _ in range(2)]
    fq.fq_kv_attn(dq, dl, dt, dc, Y=ys[0], workspace=ws)
    graphs = []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            fq.fq_kv_attn(dq, dl, dt, dc, Y=ys[i], window=200 * i, workspace=ws)
        graphs.append(gr)
    for new in ([900, 900, 900], [1, 0, 450], [33, 899, 2]):
        ln = np.array(new, np.int32)
        dl.copy_(dev(ln))
        for i in (0, 1):
            graphs[i].replay()
        for i in (0, 1):
            check_attn(ys[i], q, ln, table, pool, 128 ** -0.5, 200 * i)


def test_attn_on_another_stream():
    case = attn_case(14, [400, 20], 8, 2, 16)
    s = torch.cuda.Stream()
    args = [dev(a) for a in case[:3]] + [fq.KVCache(dev(case[3]))]
    s.wait_stream(torch.cuda.current_stream())
    y = fq.fq_kv_attn(*args, stream=s)
    s.synchronize()
    check_attn(y, *case, 128 ** -0.5)


def test_binding_refusals():
    q, lens, table, pool = attn_case(15, [40, 20], 4, 2, 16)
    dq, dl, dt, dc = dev(q), dev(lens), dev(table), fq.KVCache(dev(pool))
    with pytest.raises(ValueError):
        fq.fq_kv_attn(dq[:1], dl, dt, dc)
    with pytest.raises(ValueError):
        fq.fq_kv_attn(dq.float(), dl, dt, dc)
    with pytest.raises(ValueError):
        fq.fq_kv_attn(dq.transpose(1, 2), dl, dt, dc)
    with pytest.raises(ValueError):
        fq.fq_kv_attn(dq, dl.long(), dt, dc)
    with pytest.raises(ValueError):
        fq.fq_kv_attn(dq, dl, dt[:1], dc)
    with pytest.raises(ValueError):
        fq.fq_kv_attn(dq, dl, dt, dc, Y=torch.empty(2, 128, dtype=torch.float16, device="cuda"))
    with pytest.raises(fq.FqError):
        fq.fq_kv_attn(dq, dl, dt, dc, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fq.FqError):
        fq.fq_kv_attn(dq[:, :3].contiguous(), dl, dt, dc)          # 3 query heads on 2 key-value heads
    with pytest.raises(ValueError):
        fq.KVCache(torch.zeros(2, 2, 100, dtype=torch.uint8, device="cuda")).as_c()


# ---------------------------------------------------------------- together

def test_decode_steps_together():
    """Prompts, then decode steps: plan -> write -> attention on the device, against
    the oracle's cache built token by token."""
    g = rng(20)
    r, h, hq, page, max_pages = 5, 2, 8, 16, 12
    prompt = np.array([3, 40, 0, 16, 77], np.int32)
    free = g.permutation(r * max_pages).astype(np.int32)
    cache = fq.kv_cache(r * max_pages, h, page)
    o_pool = KO.empty_pool(r * max_pages, h, page)
    lens = torch.zeros(r, dtype=torch.int32, device="cuda")
    table = torch.full((r, max_pages), -1, dtype=torch.int32, device="cuda")
    used = torch.zeros(1, dtype=torch.int32, device="cuda")
    o_len, o_table, o_used = np.zeros(r, np.int32), np.full((r, max_pages), -1, np.int32), 0
    ws = fq.fq_kv_attn_workspace(r, hq, h)
    dfree = dev(free)
    for step in range(12):
        new = prompt if step == 0 else np.array([1, 1, step % 2, 1, 1], np.int32)
        rows = 140 if step == 0 else r
        kv = g.standard_normal((2, rows, h, 128)).astype(np.float16)
        _, _, slots, _ = fq.fq_kv_plan(lens, dev(new), table, dfree, used, page, rows, lens_out=lens,
                                       pages_used_out=used)
        fq.fq_kv_write(dev(kv[0]), dev(kv[1]), slots, cache)
        o_len, _, o_slots, u = KO.plan(o_len, new, o_table, free, o_used, page, rows)
        o_used = int(u[0])
        KO.store(o_pool, *KO.quant_rows(kv[0]), *KO.quant_rows(kv[1]), o_slots)
        q = g.standard_normal((r, hq, 128)).astype(np.float16)
        y = fq.fq_kv_attn(dev(q), lens, table, cache, workspace=ws)
        check_attn(y, q, o_len, o_table, o_pool, 128 ** -0.5)
    assert np.array_equal(cache.pool.cpu().numpy(), o_pool)
    assert np.array_equal(table.cpu().numpy(), o_table) and np.array_equal(lens.cpu().numpy(), o_len)


@pytest.mark.parametrize("fmt", [fq.MXFP4, fq.NVFP4])
def test_layer_steps_eager_and_captured(fmt):
    """A decode layer: microscaled projection to queries, keys and values, plan, write, attention over slices of the
    projection's rows, output projection.  One captured step, replayed, against the same calls one by one, bit for bit,
    and the attention against the oracle on the cache that the step left."""
    g = rng(21, fmt)
    r, h, hq, page, max_pages, width, steps = 7, 2, 6, 32, 5, 256, 40
    wide = (hq + 2 * h) * 128
    gx = None if fmt == fq.MXFP4 else torch.full((1,), 0.01, device="cuda")
    w_in = fq.fq_mx_quant(dev((g.standard_normal((wide, width)) / 16).astype(np.float16)), fmt, gx)
    w_out = fq.fq_mx_quant(dev((g.standard_normal((width, hq * 128)) / 16).astype(np.float16)), fmt, gx)
    free = dev(g.permutation(r * max_pages).astype(np.int32))
    new = torch.ones(r, dtype=torch.int32, device="cuda")
    x = torch.zeros(r, width, dtype=torch.float16, device="cuda")
    start = g.integers(0, 30, r).astype(np.int32)
    start[2] = 0

    class State:
        def __init__(self):
            self.cache = fq.kv_cache(r * max_pages, h, page)
            self.lens, self.used = dev(start), torch.zeros(1, dtype=torch.int32, device="cuda")
            self.table = torch.full((r, max_pages), -1, dtype=torch.int32, device="cuda")
            # every request's first page, as its prompt's step would have left it
            zero = torch.zeros(r, dtype=torch.int32, device="cuda")
            fq.fq_kv_plan(zero, self.lens, self.table, free, self.used, page, 0, pages_used_out=self.used)
            fq.fq_kv_plan(zero, self.lens, self.table, free, self.used, page, 30 * r, pages_used_out=self.used)
            self.ws = fq.fq_kv_attn_workspace(r, hq, h)
            self.ws_in = fq.fq_mx_linear_workspace(r, wide, width, fmt)
            self.ws_out = fq.fq_mx_linear_workspace(r, width, hq * 128, fmt)

        def step(self):
            qkv = fq.fq_mx_linear(x, fmt, *w_in, gx, gx, workspace=self.ws_in)
            q, k, v = qkv.split([hq * 128, h * 128, h * 128], dim=1)
            _, _, slots, _ = fq.fq_kv_plan(self.lens, new, self.table, free, self.used, page, r, lens_out=self.lens,
                                           pages_used_out=self.used)
            fq.fq_kv_write(k, v, slots, self.cache)
            y = fq.fq_kv_attn(q, self.lens, self.table, self.cache, workspace=self.ws)
            return q, y, fq.fq_mx_linear(y, fmt, *w_out, gx, gx, workspace=self.ws_out)

    eager, captured = State(), State()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = captured.step()
    torch.cuda.synchronize()
    for step in range(steps):
        x.copy_(dev(g.standard_normal((r, width)).astype(np.float16)))
        q, y, z = eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((q, y, z), out)), step
        assert z.isfinite().all() and z.abs().max() > 0
    fq.fq_check_device_error()
    assert torch.equal(eager.cache.pool, captured.cache.pool) and torch.equal(eager.table, captured.table)
    lens = eager.lens.cpu().numpy()
    assert np.array_equal(lens, start + steps)
    check_attn(y, q.cpu().numpy().reshape(r, hq, 128), lens, eager.table.cpu().numpy(), eager.cache.pool.cpu().numpy(),
               128 ** -0.5)


def test_two_streams_at_once():
    """Attention and the microscaled linear on two streams, each with its own workspaces: the results of one alone."""
    g = rng(22)
    cases = [attn_case(22 + i, g.integers(1, 3000, 9).tolist(), 16, 2, 32) for i in range(2)]
    x = dev(g.standard_normal((24, 2048)).astype(np.float16))
    w = fq.fq_mx_quant(dev((g.standard_normal((1024, 2048)) / 32).astype(np.float16)), fq.MXFP4)
    args = [tuple(map(dev, c[:3])) + (fq.KVCache(dev(c[3])),) for c in cases]
    alone = [(fq.fq_kv_attn(*a), fq.fq_mx_linear(x, fq.MXFP4, *w)) for a in args]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [(fq.fq_kv_attn_workspace(9, 16, 2), fq.fq_mx_linear_workspace(24, 1024, 2048, fq.MXFP4)) for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i, (a, s, ws) in enumerate(zip(args, streams, spaces)):
            got[i].append((fq.fq_kv_attn(*a, workspace=ws[0], stream=s),
                           fq.fq_mx_linear(x, fq.MXFP4, *w, workspace=ws[1], stream=s)))
    torch.cuda.synchronize()
    fq.fq_check_device_error()
    for (y, z), outs in zip(alone, got):
        assert all(torch.equal(y, a) and torch.equal(z, b) for a, b in outs)


def test_workspace_shared_with_the_fused_linear():
    """The decode linear's one-launch form leaves a generation number in the counter block; attention
    and the block-scaled product on the same workspace are not disturbed."""
    from oracle import mx_oracle as MO
    g = rng(21)
    m, n, k = 4, 512, 1024
    qp = fq.qparams(fq.STATIC)
    scale = torch.full((k,), 0.3, device="cuda")
    w = dev(g.standard_normal((n, k)).astype(np.float16))
    wq, sw = fq.fq_quant_weight(w, fq.qparams(fq.ROW), qsm_scale=scale)
    x = dev(g.standard_normal((m, k)).astype(np.float16))
    need = max(fq.fq_linear_workspace_size(m, n, k, fq.STATIC), fq.fq_kv_attn_workspace_size(2, 8, 1),
               fq.fq_mx_linear_workspace_size(m, n, 8192, MO.MXFP4))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    case = attn_case(22, [9000, 4000], 8, 1, 64)
    args = [dev(a) for a in case[:3]] + [fq.KVCache(dev(case[3]))]
    xm = dev(g.standard_normal((m, 8192)).astype(np.float16))
    mq, ms = fq.fq_mx_quant(dev(g.standard_normal((n, 8192)).astype(np.float16)), MO.MXFP4)
    y0, z0 = fq.fq_kv_attn(*args), fq.fq_mx_linear(xm, MO.MXFP4, mq, ms)
    for _ in range(3):
        fq.fq_linear(x, qp, wq, sw, static_scale=scale, workspace=ws, fused=True)
        assert torch.equal(fq.fq_kv_attn(*args, workspace=ws), y0)
        assert torch.equal(fq.fq_mx_linear(xm, MO.MXFP4, mq, ms, workspace=ws), z0)
    check_attn(y0, *case, 128 ** -0.5)
