"""The paged INT4 cache on the host: refusals of the C ABI before any launch
(fake addresses, nothing dereferenced), workspace sizes, and the oracle's
statements against hand-worked cases."""
import ctypes

import numpy as np
import pytest

from int4_linear_b200 import fq
from oracle import fq_oracle as O
from oracle import kv_oracle as KO

A = 1 << 20


@pytest.fixture(scope="module")
def L():
    from int4_linear_b200 import build
    build.build()
    return fq.lib()


def _cache(pool=A, pages=8, page=16, heads=4):
    return fq._KVCache(pool, pages, page, heads)


BAD_CACHES = [dict(pool=None), dict(pool=A + 8), dict(pages=0), dict(page=8), dict(page=48), dict(page=256),
              dict(heads=0), dict(heads=129), dict(pages=1 << 27, page=16)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_cache_description_is_checked_everywhere(L, kw):
    c = ctypes.byref(_cache(**kw))
    assert L.fq_kv_write(A, 4096, A, 4096, 3, A, 1.0, 1.0, c, None) == fq.FQ_ERR_INVALID
    assert L.fq_kv_store(A, A, A, A, 3, A, c, None) == fq.FQ_ERR_INVALID
    assert L.fq_kv_read(c, A, 3, A, A, None) == fq.FQ_ERR_INVALID
    assert L.fq_kv_attn(A, 1024, 2, 8, A, A, 4, c, 1.0, 0, A, A, 1 << 30, None) == fq.FQ_ERR_INVALID
    assert L.fq_last_error()


def test_null_cache(L):
    assert L.fq_kv_write(A, 512, A, 512, 3, A, 1.0, 1.0, None, None) == fq.FQ_ERR_INVALID
    assert L.fq_kv_read(None, A, 3, A, A, None) == fq.FQ_ERR_INVALID


@pytest.mark.parametrize("change,msg", [
    (dict(T=0), b"T"), (dict(K=None), b"NULL"), (dict(V=A + 8), b"aligned"), (dict(slots=None), b"slots"),
    (dict(slots=A + 2), b"slots"), (dict(ldk=504), b"strides"), (dict(ldv=516), b"strides"), (dict(ak=0.0), b"alpha"),
    (dict(av=1.5), b"alpha"), (dict(ak=float("nan")), b"alpha")])
def test_kv_write_refusals(L, change, msg):
    a = dict(K=A, ldk=512, V=A, ldv=512, T=3, slots=A, ak=1.0, av=1.0)
    a.update(change)
    c = _cache()
    st = L.fq_kv_write(a["K"], a["ldk"], a["V"], a["ldv"], a["T"], a["slots"], a["ak"], a["av"], ctypes.byref(c), None)
    assert st == fq.FQ_ERR_INVALID and msg in L.fq_last_error()


def test_kv_store_and_read_refusals(L):
    c = ctypes.byref(_cache())
    for args in ((None, A, A, A, 3, A), (A + 8, A, A, A, 3, A), (A, A + 1, A, A, 3, A), (A, A, A, None, 3, A),
                 (A, A, A, A, 0, A), (A, A, A, A, 3, None)):
        assert L.fq_kv_store(*args, c, None) == fq.FQ_ERR_INVALID
    for slots, t, k, v in ((None, 3, A, A), (A, 0, A, A), (A, 3, A + 8, A), (A, 3, A, None)):
        assert L.fq_kv_read(c, slots, t, k, v, None) == fq.FQ_ERR_INVALID


@pytest.mark.parametrize("change,msg", [
    (dict(R=0), b"R"), (dict(R=16385), b"R"), (dict(Hq=6), b"Hq"), (dict(Hq=2), b"Hq"), (dict(Hq=1028), b"Hq"),
    (dict(Q=None), b"NULL"), (dict(Q=A + 8), b"aligned"), (dict(Y=A + 8), b"aligned"), (dict(ldq=1016), b"ldq"),
    (dict(ldq=1028), b"ldq"), (dict(len=None), b"len"), (dict(table=A + 2), b"block_table"),
    (dict(max_pages=0), b"max_pages"), (dict(max_pages=1 << 27), b"max_pages"), (dict(window=-1), b"window"),
    (dict(scale=float("inf")), b"scale"), (dict(scale=float("nan")), b"scale"), (dict(ws=None), b"workspace"),
    (dict(ws=A + 128), b"workspace"), (dict(wsb=-1), b"workspace")])
def test_kv_attn_refusals(L, change, msg):
    need = L.fq_kv_attn_workspace_size(2, 8, 4)
    a = dict(Q=A, ldq=1024, R=2, Hq=8, len=A, table=A, max_pages=4, scale=1.0, window=0, Y=A, ws=A, wsb=0)
    a.update(change)
    c = _cache()
    st = L.fq_kv_attn(a["Q"], a["ldq"], a["R"], a["Hq"], a["len"], a["table"], a["max_pages"], ctypes.byref(c),
                      a["scale"], a["window"], a["Y"], a["ws"], need + a["wsb"], None)
    assert st == fq.FQ_ERR_INVALID and msg in L.fq_last_error()


@pytest.mark.parametrize("scale", [65537.0, -65537.0, 3e38])
def test_kv_attn_scales_that_could_overflow_are_refused(L, scale):
    c = _cache()
    ws = L.fq_kv_attn_workspace_size(2, 8, 4)
    assert L.fq_kv_attn(A, 1024, 2, 8, A, A, 4, ctypes.byref(c), scale, 0, A, A, ws, None) == fq.FQ_ERR_INVALID
    assert b"scale" in L.fq_last_error()


def test_kv_attn_workspace_sizes(L):
    assert L.fq_kv_attn_workspace_size(1, 8, 8) == fq.SYNC_BYTES + 2 * 296 * 8 * 130 * 4
    assert L.fq_kv_attn_workspace_size(16384, 128, 8) == fq.SYNC_BYTES + 2 * 148 * 16 * 130 * 4
    for r, hq, h in ((0, 8, 8), (16385, 8, 8), (1, 7, 2), (1, 8, 0), (1, 0, 0), (1, 2048, 1)):
        assert L.fq_kv_attn_workspace_size(r, hq, h) == 0


@pytest.mark.parametrize("change,msg", [
    (dict(R=0), b"R"), (dict(R=16385), b"R"), (dict(page=24), b"page_size"), (dict(max_pages=0), b"max_pages"),
    (dict(num_free=-1), b"num_free"), (dict(max_tokens=-1), b"max_tokens"),
    (dict(max_tokens=2 ** 30 + 1), b"max_tokens"), (dict(len=None), b"NULL"),
    (dict(free=None), b"NULL"), (dict(slots=None), b"NULL"), (dict(used_out=None), b"NULL"),
    (dict(slots=A + 2), b"aligned"), (dict(table=A + 1), b"aligned")])
def test_kv_plan_refusals(L, change, msg):
    a = dict(len=A, new=A, R=3, page=16, table=A, max_pages=4, free=A, num_free=5, used=A, len_out=A, start=A,
             slots=A, max_tokens=7, used_out=A)
    a.update(change)
    st = L.fq_kv_plan(a["len"], a["new"], a["R"], a["page"], a["table"], a["max_pages"], a["free"], a["num_free"],
                      a["used"], a["len_out"], a["start"], a["slots"], a["max_tokens"], a["used_out"], None)
    assert st == fq.FQ_ERR_INVALID and msg in L.fq_last_error()


# ---------------------------------------------------------------- the oracle

def test_oracle_plan_worked():
    """Pages of 16.  Request 0: 15 + 2 tokens, one fresh page (20); 1: 16 + 1,
    one fresh page (21); 2: 3 + 4, none; 3: 0 + 40, three pages, refused (one is left);
    4: needs one, refused as well (the pages asked for passed the list); 5: 1 + 1, none."""
    table = np.full((6, 3), -1, np.int32)
    table[0, 0], table[1, 0], table[2, 0], table[4, 0], table[5, 0] = 5, 6, 7, 8, 9
    out, start, slots, used = KO.plan([15, 16, 3, 0, 16, 1], [2, 1, 4, 40, 1, 1], table, [19, 20, 21, 22], 1, 16, 60)
    assert out.tolist() == [17, 17, 7, 0, 16, 2]
    assert start.tolist() == [0, 2, 3, 7, 47, 48, 49]
    assert used.tolist() == [3]
    assert table[0].tolist() == [5, 20, -1] and table[1].tolist() == [6, 21, -1] and table[4].tolist() == [8, -1, -1]
    assert slots[:7].tolist() == [5 * 16 + 15, 20 * 16, 21 * 16, 7 * 16 + 3, 7 * 16 + 4, 7 * 16 + 5, 7 * 16 + 6]
    assert (slots[7:48] == -1).all() and slots[48] == 9 * 16 + 1 and (slots[49:] == -1).all()


def test_oracle_pool_round_trip():
    g = np.random.Generator(np.random.PCG64(3))
    pool = KO.empty_pool(5, 3, 16)
    x = g.standard_normal((7, 3, 128)).astype(np.float16)
    q, s = KO.quant_rows(x)
    assert np.abs(q).max() == 7 and np.abs(q * s[..., None].astype(np.float64) - x).max() <= float(s.max()) * 0.51
    slots = np.array([3, 79, -1, 16, 80, 17, 40], np.int32)   # 80 is past the pool's 5 * 16
    KO.store(pool, q, s, -q.clip(-7, 7), s, slots)
    k, v = KO.rows(pool, np.arange(5), 16)
    for t, sl in enumerate(slots):
        if 0 <= sl < 80:
            assert np.array_equal(k[sl], q[t] * s[t].astype(np.float64)[:, None])
            assert np.array_equal(v[sl], -k[sl])
    assert np.count_nonzero(np.abs(k).sum((1, 2))) == 5
    kq, _, ks, _ = KO.views(pool)
    assert np.array_equal(O.unpack_int4(kq[0, 1, 3][None])[0], q[0, 1]) and ks[0, 1, 3] == s[0, 1]


def test_oracle_attention_worked():
    """Two tokens whose scores differ by log 3: weights 1/4 and 3/4."""
    pool = KO.empty_pool(2, 1, 16)
    q8 = np.zeros((2, 1, 128), np.int8)
    q8[0, 0, 0], q8[1, 0, 0] = 1, 2
    v8 = np.zeros((2, 1, 128), np.int8)
    v8[0, 0, 5], v8[1, 0, 5] = 4, -8
    one = np.ones((2, 1), np.float16)
    KO.store(pool, q8, one, v8, one, np.array([16 + 0, 16 + 1]))
    q = np.zeros((1, 1, 128), np.float16)
    q[0, 0, 0] = 1
    table = np.array([[1]], np.int32)
    y = KO.attention(q, [2], table, pool, np.log(3.0))[0]
    assert abs(y[0, 0, 5] - (0.25 * 4 - 0.75 * 8)) < 1e-12 and np.count_nonzero(y) == 1
    assert abs(KO.attention(q, [2], table, pool, 1.0, window=1)[0][0, 0, 5] + 8) < 1e-12
    assert not KO.attention(q, [0], table, pool, 1.0)[0].any()
    assert not KO.attention(q, [2], np.array([[-1]], np.int32), pool, 1.0)[0].any()
