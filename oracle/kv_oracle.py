"""CPU oracle of the paged INT4 key/value cache (test infrastructure only).

Plain numpy statements of the block tables and slots of a step, of the codes
and scales of a cached head vector, of a page's bytes, and of the attention of
one new token over the cache in float64.  Shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from . import fq_oracle as O

HEAD = 128


def plan(lens, new, table, free, used, page, max_tokens):
    """(len_out, token_start, slots, used_out); `table` is updated in place."""
    lens = [max(int(x), 0) for x in lens]
    new = [max(int(x), 0) for x in new]
    slots = [-1] * max_tokens
    start, out = [0], []
    row = asked = taken = 0
    for r, (n, k) in enumerate(zip(lens, new)):
        held, want = -(-n // page), -(-(n + k) // page)
        ok = want <= table.shape[1] and row + k <= max_tokens
        if ok:
            before = asked
            asked += want - held
            ok = want == held or asked <= len(free) - used
        if ok:
            for j in range(want - held):
                table[r, held + j] = free[used + before + j]
            taken += want - held
            for i in range(k):
                p = n + i
                pg = int(table[r, p // page])
                if 0 <= pg < 2 ** 31 // page:
                    slots[row + i] = pg * page + p % page
        out.append(n + k if ok else n)
        row += k
        start.append(row)
    i32 = lambda a: np.asarray(a, np.int32)
    return i32(out), i32(start), i32(slots), i32([used + taken])


def quant_rows(x, alpha=1.0):
    """Codes int8 [..., 128] and fp16 scales [...] of head vectors x (fp16).  Vectors with an infinity or
    NaN have the NaN scale 0x7FFF (and here codes 0)."""
    v = np.asarray(x, np.float16).astype(np.float32)
    finite = np.isfinite(v).all(-1)
    v = np.where(finite[..., None], v, np.float32(0))
    amax = np.abs(v).max(-1)
    s = ((amax * np.float32(alpha)).astype(np.float32) / np.float32(7.0)).astype(np.float16)
    return (O.quantize(v, s.astype(np.float32)[..., None]).astype(np.int8),
            np.where(finite, s, np.array(0x7FFF, np.uint16).view(np.float16)))


def empty_pool(pages, heads, page):
    return np.zeros((pages, heads, page * 132), np.uint8)


def views(pool):
    """Views (K codes [P, H, page, 64], V codes, K scales, V scales) of a pool."""
    p, h, b = pool.shape
    n = b // 132
    kq = pool[:, :, :64 * n].reshape(p, h, n, 64)
    vq = pool[:, :, 64 * n:128 * n].reshape(p, h, n, 64)
    ks = pool[:, :, 128 * n:130 * n].view(np.float16)
    vs = pool[:, :, 130 * n:].view(np.float16)
    return kq, vq, ks, vs


def store(pool, kq, ks, vq, vs, slots):
    """Codes int8 [T, H, 128] and scales fp16 [T, H] to their slots (in place)."""
    n = pool.shape[2] // 132
    limit = pool.shape[0] * n
    for t, s in enumerate(slots):
        if 0 <= s < limit:
            pg, off = int(s) // n, int(s) % n
            for which, (q, sc) in enumerate(((kq, ks), (vq, vs))):
                a = 64 * n * which + 64 * off
                pool[pg, :, a:a + 64] = O.pack_int4(q[t])
                b = 128 * n + 2 * n * which + 2 * off
                pool[pg, :, b:b + 2] = sc[t][:, None].view(np.uint8)


def rows(pool, ids, page):
    """Float64 K and V [len(ids) * page, H, 128] of the pages `ids`."""
    out = []
    part = pool[np.asarray(ids, np.int64)]
    kq, vq, ks, vs = views(np.ascontiguousarray(part))
    for q, s in ((kq, ks), (vq, vs)):
        c = O.unpack_int4(q.reshape(-1, 64)).reshape(q.shape[:3] + (HEAD,)).astype(np.float64)
        with np.errstate(invalid="ignore"):       # scales of empty places may hold anything
            x = c * s.astype(np.float64)[..., None]
        out.append(x.transpose(0, 2, 1, 3).reshape(-1, pool.shape[1], HEAD))
    return out


def attention(q, lens, table, pool, scale, window=0):
    """Float64 (y [R, Hq, 128], the weights' spread sum p |v|, sqrt(sum p^2 v^2)
    and each request's largest K scale), the last three for error bounds."""
    r, hq, _ = q.shape
    h = pool.shape[1]
    page = pool.shape[2] // 132
    g = hq // h
    y, sa, sq = (np.zeros((r, hq, HEAD)) for _ in range(3))
    kmax = np.zeros(r)
    for i in range(r):
        n = min(max(int(lens[i]), 0), table.shape[1] * page)
        lo = max(0, n - window) if window > 0 else 0
        if n == lo:
            continue
        p0 = lo // page
        ids = table[i, p0:-(-n // page)]
        pos = np.arange(p0 * page, p0 * page + len(ids) * page)
        good = np.repeat((ids >= 0) & (ids < pool.shape[0]), page) & (pos >= lo) & (pos < n)
        if not good.any():
            continue
        k, v = rows(pool, np.clip(ids, 0, pool.shape[0] - 1), page)
        k, v = k[good], v[good]
        kmax[i] = np.abs(k).max() / 4 if k.size else 0.0
        for a in range(hq):
            s = (k[:, a // g] @ q[i, a].astype(np.float64)) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            vv = v[:, a // g]
            y[i, a] = w @ vv
            sa[i, a] = w @ np.abs(vv)
            sq[i, a] = np.sqrt((w * w) @ (vv * vv))
    return y, sa, sq, kmax
