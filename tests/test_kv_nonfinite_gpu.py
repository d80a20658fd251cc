"""Keys and values that are not finite: their head vectors are cached with a NaN scale, and everything that reads
them shows it."""
import numpy as np
import pytest
import torch

from int4_linear_b200 import fq
from oracle import kv_oracle as KO
from tests.test_kv_gpu import dev, rng

pytestmark = pytest.mark.gpu

BAD = [np.nan, -np.nan, np.inf, -np.inf]


@pytest.mark.parametrize("t,h,page", [(1, 1, 16), (5, 3, 32), (200, 8, 64)])
@pytest.mark.parametrize("alpha", [1.0, 0.83])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -20])
def test_write_and_read(t, h, page, alpha, size):
    g = rng(51, t, h)
    x = (g.standard_normal((2, t, h, 128)) * size).astype(np.float16)
    hit = g.random((2, t, h)) < 0.3
    hit[0, 0, 0] = True
    for i, (w, a, b) in enumerate(np.argwhere(hit)):
        x[w, a, b, g.integers(0, 128)] = BAD[i % 4]
        if i % 3 == 0:                           # several in one vector
            x[w, a, b, g.integers(0, 128, 9)] = BAD[(i + 1) % 4]
    pages = -(-t // page) + 1
    slots = g.permutation(pages * page)[:t].astype(np.int32)
    rows = [KO.quant_rows(x[w], alpha) for w in range(2)]
    assert all(np.array_equal(np.isnan(s), hit[w]) and not q[hit[w]].any() for w, (q, s) in enumerate(rows))
    want = KO.empty_pool(pages, h, page)
    KO.store(want, *rows[0], *rows[1], slots)
    cache, sl = fq.kv_cache(pages, h, page), dev(slots)
    fq.fq_kv_write(dev(x[0]), dev(x[1]), sl, cache, alpha, alpha)
    pool = cache.pool.cpu().numpy()
    for kind in range(2):                        # codes beside a NaN scale have no meaning
        for p in (pool, want):
            codes, scales = KO.views(p)[kind], KO.views(p)[kind + 2]
            codes[np.isnan(scales)] = 0
    assert np.array_equal(pool, want)
    for got, bad, (q, s) in zip(fq.fq_kv_read(cache, sl), hit, rows):
        got = got.cpu().numpy()
        assert np.array_equal(np.isnan(got), np.broadcast_to(bad[..., None], got.shape))
        ref = (q[~bad].astype(np.float32) * s[~bad].astype(np.float32)[..., None]).astype(np.float16)
        assert np.array_equal(got[~bad], ref)


@pytest.mark.parametrize("hq,h", [(4, 2), (12, 2), (32, 2)])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("page", [16, 64])
def test_attention_shows_it(hq, h, which, bad, page):
    """One bad key or value of the second key-value head: the query heads that read it are NaN, the others and the other
    requests keep their bits, and so does everything once the window has left the token behind."""
    g = rng(52, hq, h)
    lens = np.array([900, 300], np.int32)
    x = g.standard_normal((2, int(lens.sum()), h, 128)).astype(np.float16)
    pages = [-(-int(n) // page) for n in lens]
    table = np.full((2, max(pages)), -1, np.int32)
    table[0, :pages[0]] = np.arange(pages[0])
    table[1, :pages[1]] = pages[0] + np.arange(pages[1])
    slots = np.concatenate([np.arange(900), pages[0] * page + np.arange(300)]).astype(np.int32)
    q = dev(g.standard_normal((2, hq, 128)).astype(np.float16))
    out = []
    for poisoned in (False, True):
        if poisoned:
            x[which, 100, 1, 77] = bad
        cache = fq.kv_cache(sum(pages), h, page)
        fq.fq_kv_write(dev(x[0]), dev(x[1]), dev(slots), cache)
        out.append([fq.fq_kv_attn(q, dev(lens), dev(table), cache, window=w).view(2, hq, 128) for w in (0, 799)])
    fq.fq_check_device_error()
    hit = torch.zeros(2, hq, 128, dtype=torch.bool, device="cuda")
    hit[0, hq // h:] = True
    good, shown = out
    assert torch.equal(torch.isnan(shown[0]), hit)
    assert torch.equal(shown[0][~hit], good[0][~hit])
    assert torch.equal(shown[1], good[1]) and shown[1].isfinite().all()


@pytest.mark.parametrize("hq,h", [(4, 1), (8, 1), (16, 1)])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("code", [0x00, 0x77, 0x88])
def test_query_whose_scores_would_be_infinite(hq, h, bad, code):
    """One infinite value times codes of one sign would give every token a score of minus infinity, i.e. no weight at
    all: the head is NaN all the same."""
    cache = fq.kv_cache(1, h, 16)
    kq, vq, ks, vs = cache.views()
    kq[:] = code
    vq[:] = 0x11
    ks[:] = vs[:] = 1
    q = torch.ones(1, hq, 128, dtype=torch.float16, device="cuda")
    q[0, 1, 17] = bad
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    y = fq.fq_kv_attn(q, one * 9, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), cache).view(hq, 128)
    hit = torch.zeros(hq, 128, dtype=torch.bool, device="cuda")
    hit[1] = True
    assert torch.equal(torch.isnan(y), hit) and (y[~hit] == 1).all()
