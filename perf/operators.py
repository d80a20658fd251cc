"""The operators of the 4-bit decoder path, as measured workloads.

Four operators, each in its plain form (elementary torch operations) and as the
calls that a user of ``int4_linear_b200.fq`` makes:

* ``plan``      block tables and slot maps of a paged cache from request lengths
                (``fq_kv_plan``)
* ``kv_write``  keys and values into the pages as INT4 and back
                (``fq_kv_write``, ``fq_kv_read``)
* ``attn``      attention of one new token per request over the paged INT4 cache
                (``fq_kv_attn``)
* ``mx_linear`` the microscaled 4-bit floating point linear layer: activation
                quantization and the block-scaled product (``fq_mx_linear``)

Layouts: the cache pool is uint8 [pages, heads, page_size * 132]: of one page and
head, the K codes (page_size x 64 bytes, two signed nibbles each), the V codes, the
K scales (page_size fp16) and the V scales.  Microscaled codes are E2M1, two per
byte, with one scale byte per 32 (MXFP4, E8M0) or 16 (NVFP4, E4M3) values, stored
in tiles of 128 rows x 4 scales (512 bytes: row r, scale k at
(r % 32) * 16 + (r % 128 // 32) * 4 + k).
"""
from __future__ import annotations

import math

import torch

own = False

HEAD = 128
ROW_BYTES = HEAD // 2


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 64 running requests, pages of 16
        dict(name="plan_decode", op="plan", requests=64, page=16, max_len=4096, prompts=0, prompt_len=0),
        # a mixed step: 1000 running requests and 37 prompts of up to 1500 tokens
        dict(name="plan_mixed", op="plan", requests=1037, page=32, max_len=8192, prompts=37, prompt_len=1500),
        # the new tokens of 48 running requests, 8 key-value heads
        dict(name="kv_write_decode", op="kv_write", tokens=48, heads=8, page=16),
        # a prompt chunk of 16384 tokens, 8 key-value heads
        dict(name="kv_write_prompt", op="kv_write", tokens=16384, heads=8, page=64),
        # one chat request of a grouped-query model: latency counts
        dict(name="attn_single", op="attn", requests=1, q_heads=32, heads=8, page=16, min_len=1000, max_len=1000,
             window=0),
        # a ragged batch, an empty slot among it, odd lengths
        dict(name="attn_ragged", op="attn", requests=33, q_heads=40, heads=8, page=32, min_len=0, max_len=4097,
             window=0),
        # every head with its own keys and values, a sliding window
        dict(name="attn_mha_window", op="attn", requests=12, q_heads=32, heads=32, page=16, min_len=900,
             max_len=6000, window=2048),
        # long contexts of a large grouped-query model: the cache's bandwidth
        dict(name="attn_long", op="attn", requests=64, q_heads=64, heads=8, page=64, min_len=12000, max_len=16384,
             window=0),
        # query, key and value projection of one token
        dict(name="mx_linear_token", op="mx_linear", rows=1, k=4096, n=6144, fmt="mxfp4"),
        # gate and up projection of a large model, a decode batch
        dict(name="mx_linear_decode", op="mx_linear", rows=16, k=8192, n=57344, fmt="nvfp4"),
        # odd sizes: a ragged batch of prompt tokens
        dict(name="mx_linear_ragged", op="mx_linear", rows=777, k=4224, n=5000, fmt="nvfp4"),
        # gate and up projection of a prompt of 2048 tokens
        dict(name="mx_linear_prompt", op="mx_linear", rows=2048, k=4096, n=28672, fmt="mxfp4"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "kv_write", "attn", "attn", "mx_linear", "mx_linear"])
    if op == "plan":
        requests = _log_int(rng, 1, 2048)
        prompts = rng.randint(0, min(requests, 40))
        return dict(op=op, requests=requests, page=rng.choice([16, 32, 64, 128]), max_len=_log_int(rng, 64, 8192),
                    prompts=prompts, prompt_len=_log_int(rng, 1, 1500) if prompts else 0)
    if op == "kv_write":
        heads = rng.choice([1, 2, 4, 5, 8, 16, 32])
        return dict(op=op, tokens=_log_int(rng, 1, 16384 * 8 // heads if heads > 8 else 16384), heads=heads,
                    page=rng.choice([16, 32, 64, 128]))
    if op == "attn":
        heads = rng.choice([1, 2, 3, 4, 8, 16, 32])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        requests = _log_int(rng, 1, 64)
        top = min(16384, 64 * 8 * 14000 // (requests * heads))
        if heads * group > 128:
            group = 128 // heads
        max_len = _log_int(rng, 1, top)
        min_len = rng.choice([0, max_len // 2, max_len])
        return dict(op=op, requests=requests, q_heads=heads * group, heads=heads, page=rng.choice([16, 32, 64, 128]),
                    min_len=min_len, max_len=max_len, window=rng.choice([0, 0, 0, _log_int(rng, 1, max_len)]))
    rows = _log_int(rng, 1, 2048)
    k = 128 * _log_int(rng, 1, 112)
    top = min(57344, 2048 * 4096 * 28672 // (rows * k), 8192 * 57344 // k)
    return dict(op=op, rows=rows, k=k, n=8 * _log_int(rng, 1, top // 8), fmt=rng.choice(["mxfp4", "nvfp4"]))


# ---------------------------------------------------------------- inputs

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)
    return g


def _lengths(case, seed):
    """Request lengths (host integers), from the seed alone."""
    g = _gen(seed, "cpu")
    lo, hi = case["min_len"], case["max_len"]
    n = case["requests"]
    ln = torch.randint(lo, hi + 1, (n,), generator=g).tolist()
    if n > 2:
        ln[n // 3] = lo
        ln[n // 2] = hi
    return ln


def _plan_inputs(case, seed):
    g = _gen(seed, "cpu")
    n, page = case["requests"], case["page"]
    length = torch.randint(1, case["max_len"] + 1, (n,), generator=g, dtype=torch.int32)
    new = torch.ones(n, dtype=torch.int32)
    if case["prompts"]:
        who = torch.randperm(n, generator=g)[:case["prompts"]]
        length[who] = 0
        new[who] = torch.randint(1, case["prompt_len"] + 1, (case["prompts"],), generator=g, dtype=torch.int32)
    max_pages = -(-(case["max_len"] + case["prompt_len"] + 1) // page)
    held = (length + page - 1) // page
    total = int(held.sum())
    # rows of the step's batch, as a captured step has them: some are left over
    rows = n - case["prompts"] + case["prompts"] * case["prompt_len"] + 29
    ids = torch.randperm(total + n + 64 + rows // page, generator=g).to(torch.int32)
    table = torch.full((n, max_pages), -1, dtype=torch.int32)
    table[torch.arange(max_pages)[None] < held[:, None]] = ids[:total]
    return length, new, table, ids[total:].contiguous(), rows


def _quant_rows(x, alpha):
    """INT4 codes (float) and fp16 scales of head vectors x (float32 [..., 128])."""
    s = ((x.abs().amax(-1) * alpha) / 7.0).half()
    sf = s.float()[..., None]
    q = torch.where(sf == 0, torch.zeros_like(x), torch.round(x / sf))
    return q.clamp(-8, 7), s


def _pack_nibbles(q):
    u = q.to(torch.int16) & 15
    return (u[..., 0::2] | (u[..., 1::2] << 4)).to(torch.uint8)


def _fill_pool(case, pages, g):
    heads, page = case["heads"], case["page"]
    pool = torch.empty(pages, heads, page * 132, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (heads * page * HEAD))
    a, b = page * ROW_BYTES, 2 * page * ROW_BYTES
    for p0 in range(0, pages, step):
        p1 = min(pages, p0 + step)
        for which in range(2):
            x = torch.randn(p1 - p0, heads, page, HEAD, generator=g, device="cuda")
            if which == 0:
                x[..., ::16] *= 3.0
            q, s = _quant_rows(x.half().float(), 1.0)
            pool[p0:p1, :, which * a:which * a + a] = _pack_nibbles(q).view(p1 - p0, heads, -1)
            pool[p0:p1, :, b + 2 * page * which:b + 2 * page * (which + 1)] = s.view(torch.uint8)
    return pool


def _mx_block(fmt):
    return 32 if fmt == "mxfp4" else 16


def _mx_scale_to_tiles(s):
    """Scale bytes [rows, blocks] -> tiles of 128 rows x 4 blocks (rows padded with zeros)."""
    r, kb = s.shape
    rt = -(-r // 128)
    full = torch.zeros(rt * 128, kb, dtype=torch.uint8, device=s.device)
    full[:r] = s
    return full.view(rt, 4, 32, kb // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _mx_scale_from_tiles(t, r, kb):
    rt = -(-r // 128)
    return t.view(rt, kb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kb)[:r]


def _mx_scales(x, fmt, g):
    """Block scales of x float32 [rows, k]: (bytes, the float32 divisor of each block)."""
    amax = x.view(x.shape[0], -1, _mx_block(fmt)).abs().amax(-1)
    if fmt == "mxfp4":
        e = torch.frexp(amax).exponent - 3           # floor(log2 amax) - 2
        e = torch.where(amax == 0, torch.full_like(e, -127), e)
        return (e + 127).to(torch.uint8), torch.ldexp(torch.ones_like(amax), e)
    s = (amax / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    return s.view(torch.uint8), s.float() * g


def _mx_round(a):
    """Nearest E2M1 magnitude, ties to the even code."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp(max=6.0)


def _mx_quant_pack(x, fmt, g):
    """float32 [rows, k] -> (packed codes [rows, k/2], scale bytes [rows, k/block])."""
    sb, d = _mx_scales(x, fmt, g)
    xb = x.view(x.shape[0], -1, _mx_block(fmt))
    v = torch.where(d[..., None] == 0, torch.zeros_like(xb), xb / d[..., None])
    m = _mx_round(v.abs())
    code = torch.where(m < 2, m * 2, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).view(x.shape)
    return code[:, 0::2] | (code[:, 1::2] << 4), sb


def prepare(case, seed):
    op = case["op"]
    st = dict(case=case, op=op)
    if op == "plan":
        length, new, table, free, tokens = _plan_inputs(case, seed)
        st.update(length=length.cuda(), new=new.cuda(), table=table.cuda(), free=free.cuda(),
                  used=torch.zeros(1, dtype=torch.int32, device="cuda"), tokens=tokens)
        return st
    g = _gen(seed)
    if op == "kv_write":
        t, h, page = case["tokens"], case["heads"], case["page"]
        # keys and values are slices of one projection's output, as a model has them
        qkv = torch.randn(t, 3 * h * HEAD, generator=g, device="cuda")
        qkv[:, h * HEAD::37] *= 8.0
        qkv = qkv.half()
        pages = -(-t // page) * 2 + 3
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:t].to(torch.int32)
        if t > 4:
            slots[t // 2] = -1                        # a padded row of the batch
        st.update(k=qkv[:, h * HEAD:2 * h * HEAD], v=qkv[:, 2 * h * HEAD:], slots=slots,
                  pool=torch.zeros(pages, h, page * 132, dtype=torch.uint8, device="cuda"))
        if own:
            from int4_linear_b200 import fq
            st["cache"] = fq.KVCache(st["pool"])
        return st
    if op == "attn":
        ln = _lengths(case, seed)
        page, hq = case["page"], case["q_heads"]
        max_pages = max(1, -(-case["max_len"] // page))
        held = [-(-n // page) for n in ln]
        pages = sum(held) + 2
        ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((len(ln), max_pages), -1, dtype=torch.int32, device="cuda")
        o = 0
        for r, c in enumerate(held):
            table[r, :c] = ids[o:o + c]
            o += c
        q = (torch.randn(len(ln), hq, HEAD, generator=g, device="cuda") * 1.5).half()
        st.update(q=q, table=table, length=torch.tensor(ln, dtype=torch.int32, device="cuda"), host_length=ln,
                  pool=_fill_pool(case, pages, g), scale=HEAD ** -0.5)
        if own:
            from int4_linear_b200 import fq
            st["cache"] = fq.KVCache(st["pool"])
            st["ws"] = fq.fq_kv_attn_workspace(len(ln), hq, case["heads"], q.device)
        return st
    r, k, n, fmt = case["rows"], case["k"], case["n"], case["fmt"]
    x = torch.randn(r, k, generator=g, device="cuda")
    x[:, torch.randperm(k, generator=g, device="cuda")[:max(1, k // 100)]] *= 12.0   # outlier channels
    x = x.half()
    kb = k // _mx_block(fmt)
    gx = gw = None
    if fmt == "nvfp4":
        gx = torch.full((1,), 60.0 / (6 * 448), device="cuda")       # calibrated: the largest |x| seen
        gw = torch.full((1,), 0.12 / (6 * 448), device="cuda")
    wq = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
    ws = torch.empty(n, kb, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // k)
    for i in range(0, n, step):
        w = (torch.randn(min(step, n - i), k, generator=g, device="cuda") * 0.02).half().float()
        wq[i:i + step], ws[i:i + step] = _mx_quant_pack(w, fmt, gw)
    st.update(x=x, wq=wq, ws=_mx_scale_to_tiles(ws), gx=gx, gw=gw, fmt=fmt)
    if own:
        from int4_linear_b200 import fq
        st["fmt_id"] = fq.MXFP4 if fmt == "mxfp4" else fq.NVFP4
        st["workspace"] = fq.fq_mx_linear_workspace(r, n, k, st["fmt_id"], x.device)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["op"]
    if own:
        from int4_linear_b200 import fq
        if op == "plan":
            lens, start, slots, used = fq.fq_kv_plan(st["length"], st["new"], st["table"], st["free"], st["used"],
                                                     st["case"]["page"], st["tokens"])
            return st["table"], lens, start, slots, used
        if op == "kv_write":
            fq.fq_kv_write(st["k"], st["v"], st["slots"], st["cache"])
            return fq.fq_kv_read(st["cache"], st["slots"])
        if op == "attn":
            return fq.fq_kv_attn(st["q"], st["length"], st["table"], st["cache"], scale=st["scale"],
                                 window=st["case"]["window"], workspace=st["ws"])
        return fq.fq_mx_linear(st["x"], st["fmt_id"], st["wq"], st["ws"], st["gx"], st["gw"],
                               workspace=st["workspace"])
    return {"plan": _plan_plain, "kv_write": _kv_write_plain, "attn": _attn_plain, "mx_linear": _mx_plain}[op](st)


def _plan_plain(st):
    page, tokens = st["case"]["page"], st["tokens"]
    length, new, table, free = st["length"], st["new"], st["table"], st["free"]
    n, max_pages = table.shape
    after = length + new
    held = (length + page - 1) // page
    want = (after + page - 1) // page
    start = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    start[1:] = torch.cumsum(new, 0)
    fits = (want <= max_pages) & (start[1:] <= tokens)
    need = torch.where(fits, want - held, torch.zeros_like(held))
    end = torch.cumsum(need, 0).to(torch.int32)
    granted = fits & ((need == 0) | (end <= free.numel() - st["used"]))
    first = end - need + st["used"]
    j = torch.arange(max_pages, device="cuda")[None]
    fresh = granted[:, None] & (j >= held[:, None]) & (j < want[:, None])
    pick = (first[:, None] + j - held[:, None]).clamp(0, free.numel() - 1).long()
    table.copy_(torch.where(fresh, free[pick], table))
    used = st["used"] + torch.where(granted, need, torch.zeros_like(need)).sum().to(torch.int32)
    i = torch.arange(tokens, device="cuda", dtype=torch.int32)
    r = torch.searchsorted(start, i, right=True).long() - 1
    inside = r < n
    r = r.clamp(max=n - 1)
    pos = length[r] + i - start[r]
    ok = inside & granted[r]
    pid = table[r, (pos // page).clamp(0, max_pages - 1).long()]
    slots = torch.where(ok, pid * page + pos % page, torch.full_like(pos, -1))
    return table, torch.where(granted, after, length), start, slots, used


def _kv_write_plain(st):
    case = st["case"]
    t, h, page = case["tokens"], case["heads"], case["page"]
    a, b = page * ROW_BYTES, 2 * page * ROW_BYTES
    pool, slots = st["pool"], st["slots"].long()
    keep = slots >= 0
    pid, off = slots.clamp(min=0) // page, slots.clamp(min=0) % page
    out = []
    for which, x in enumerate((st["k"], st["v"])):
        q, s = _quant_rows(x.float().view(t, h, HEAD), 1.0)
        codes = pool[:, :, which * a:which * a + a].unflatten(-1, (page, ROW_BYTES))
        scales = pool[:, :, b + 2 * page * which:b + 2 * page * (which + 1)].view(torch.float16)
        kp, ko = pid[keep], off[keep]
        codes[kp, :, ko] = _pack_nibbles(q)[keep]
        scales[kp, :, ko] = s[keep]
        c = codes[pid, :, off]
        lo, hi = (c & 15).to(torch.int8), (c >> 4).to(torch.int8)
        w = torch.stack((lo, hi), -1).flatten(-2)
        w = torch.where(w > 7, w - 16, w).float() * scales[pid, :, off].float()[..., None]
        out.append(torch.where(keep[:, None, None], w, torch.zeros_like(w)).half())
    return tuple(out)


def _pool_rows(pool, ids, page, which, dtype):
    """Dequantized rows [len(ids) * page, heads, 128] of the pages `ids`."""
    a, b = page * ROW_BYTES, 2 * page * ROW_BYTES
    part = pool[ids]
    c = part[:, :, which * a:which * a + a].unflatten(-1, (page, ROW_BYTES))
    s = part[:, :, b + 2 * page * which:b + 2 * page * (which + 1)].contiguous().view(torch.float16)
    w = torch.stack(((c & 15).to(torch.int8), (c >> 4).to(torch.int8)), -1).flatten(-2)
    w = torch.where(w > 7, w - 16, w).to(dtype) * s.to(dtype)[..., None]
    return w.transpose(1, 2).flatten(0, 1)


def _attn_plain(st):
    case = st["case"]
    page, heads, hq, window = case["page"], case["heads"], case["q_heads"], case["window"]
    out = []
    for r, n in enumerate(st["host_length"]):
        if n == 0:
            out.append(torch.zeros(hq * HEAD, dtype=torch.float16, device="cuda"))
            continue
        lo = max(0, n - window) if window else 0
        p0 = lo // page
        ids = st["table"][r, p0:-(-n // page)].long()
        k = _pool_rows(st["pool"], ids, page, 0, torch.float32)[lo - p0 * page:n - p0 * page]
        v = _pool_rows(st["pool"], ids, page, 1, torch.float32)[lo - p0 * page:n - p0 * page]
        q = st["q"][r].float().view(heads, hq // heads, HEAD)
        s = torch.matmul(q, k.permute(1, 2, 0)) * st["scale"]
        s = torch.exp(s - s.amax(-1, keepdim=True))
        o = torch.matmul(s, v.transpose(0, 1)) / s.sum(-1, keepdim=True)
        out.append(o.reshape(-1).half())
    return torch.stack(out)


def _mx_unpack(codes, scale, fmt):
    """Packed codes [rows, k/2] and the block divisors [rows, k/block] -> float32 [rows, k]."""
    u = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    m = (u & 7).float()
    a = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, m * 2 - 8))
    a = torch.where(u > 7, -a, a)
    return (a.unflatten(-1, (-1, _mx_block(fmt))) * scale[..., None]).flatten(-2)


def _mx_divisor(sb, fmt):
    if fmt == "mxfp4":
        return torch.ldexp(torch.ones(sb.shape, device=sb.device), sb.int() - 127)
    return sb.view(torch.float8_e4m3fn).float()


def _mx_plain(st):
    fmt, x = st["fmt"], st["x"].float()
    r, k = x.shape
    n = st["wq"].shape[0]
    kb = k // _mx_block(fmt)
    codes, sb = _mx_quant_pack(x, fmt, st["gx"])
    xd = _mx_unpack(codes, _mx_divisor(sb, fmt), fmt)
    ws = _mx_scale_from_tiles(st["ws"], n, kb)
    y = torch.matmul(xd, _mx_unpack(st["wq"], _mx_divisor(ws, fmt), fmt).t())
    if fmt == "nvfp4":
        y = y * (st["gx"] * st["gw"])
    return y.half()


# ---------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "plan":
        length, new, table, free, tokens = _plan_inputs(case, 0)
        page = case["page"]
        fresh = int(((length + new + page - 1) // page - (length + page - 1) // page).sum())
        # lengths and counts in; lengths, offsets, fresh pages (in the free list and the
        # table) and slots out, and the table's entries that a first new token lands in
        return dict(bytes=4 * (5 * case["requests"] + 2 * fresh + tokens + 3), flops=0)
    if op == "kv_write":
        rows = 2 * case["tokens"] * case["heads"]
        return dict(bytes=rows * (2 * HEAD + ROW_BYTES + 2 + 2 * HEAD) + 4 * case["tokens"], flops=rows * HEAD * 4)
    if op == "attn":
        toks = sum(min(n, case["window"] or n) for n in _lengths(case, 0))
        return dict(bytes=int(toks * case["heads"] * 2 * (ROW_BYTES + 2) + 4 * toks / case["page"]
                              + case["requests"] * (case["q_heads"] * HEAD * 4 + 4)),
                    flops=int(toks * case["q_heads"] * HEAD * 4))
    r, k, n = case["rows"], case["k"], case["n"]
    kb = k // _mx_block(case["fmt"])
    return dict(bytes=2 * r * k + n * (k // 2 + kb) + 2 * r * n, flops=2 * r * k * n)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return _plan_exact(case, seed)
    st = prepare(case, seed)
    return {"kv_write": _kv_write_exact, "attn": _attn_exact, "mx_linear": _mx_exact}[op](st)


def _plan_exact(case, seed):
    length, new, table, free, tokens = _plan_inputs(case, seed)
    page, (n, max_pages) = case["page"], table.shape
    ln, nw, tb, fr = length.tolist(), new.tolist(), table.tolist(), free.tolist()
    slots, start, out, taken, asked, tok = [-1] * tokens, [0], [], 0, 0, 0
    for r in range(n):
        total = ln[r] + nw[r]
        want, held = -(-total // page), -(-ln[r] // page)
        ok = want <= max_pages and tok + nw[r] <= tokens
        if ok:
            asked += want - held
            ok = want == held or asked <= len(fr)
        if ok:
            first = asked - (want - held)
            for j in range(want - held):
                tb[r][held + j] = fr[first + j]
            taken += want - held
            for i in range(nw[r]):
                p = ln[r] + i
                slots[tok + i] = tb[r][p // page] * page + p % page
        out.append(total if ok else ln[r])
        tok += nw[r]
        start.append(tok)

    def dev(a):
        return torch.tensor(a, dtype=torch.int32, device="cuda")

    return dev(tb), dev(out), dev(start), dev(slots), dev([taken])


def _kv_write_exact(st):
    case = st["case"]
    t, h = case["tokens"], case["heads"]
    res = []
    for x in (st["k"], st["v"]):
        x = x.double().reshape(t, h, HEAD)
        # the scale is the fp16 rounding of a float32 quotient (alpha = 1)
        s = (x.abs().max(-1).values.float() / 7).half().double()
        ratio = (x / s[:, :, None].clamp(min=2.0 ** -30)).float().double()
        code = ratio.round().clamp(-8, 7) * (s[:, :, None] > 0)
        res.append(code * s[:, :, None] * (st["slots"] >= 0)[:, None, None])
    return tuple(res)


def _attn_exact(st):
    case = st["case"]
    page, heads, hq, window = case["page"], case["heads"], case["q_heads"], case["window"]
    y = torch.zeros(case["requests"], heads, hq // heads, HEAD, dtype=torch.float64, device="cuda")
    lut = torch.tensor([c - 16 if c > 7 else c for c in range(16)], dtype=torch.float64, device="cuda")
    a, b = page * ROW_BYTES, 2 * page * ROW_BYTES
    for r, n in enumerate(st["host_length"]):
        if not n:
            continue
        pos = torch.arange(max(0, n - window) if window else 0, n, device="cuda")
        pid, off = st["table"][r][pos // page].long(), pos % page
        for hd in range(heads):
            rows = st["pool"][:, hd]
            col = off[:, None] * ROW_BYTES + torch.arange(ROW_BYTES, device="cuda")[None]
            kv = []
            for which in range(2):
                byte = rows[pid[:, None], which * a + col].long()
                code = torch.empty(pos.numel(), HEAD, dtype=torch.float64, device="cuda")
                code[:, 0::2], code[:, 1::2] = lut[byte % 16], lut[byte // 16]
                sc = rows[:, b + 2 * page * which:b + 2 * page * (which + 1)].view(torch.float16)[pid, off]
                kv.append(code * sc.double()[:, None])
            q = st["q"][r, hd * (hq // heads):(hd + 1) * (hq // heads)].double()
            y[r, hd] = torch.softmax(q @ kv[0].t() * st["scale"], -1) @ kv[1]
    return y.reshape(case["requests"], -1)


def _mx_exact(st):
    fmt, x = st["fmt"], st["x"].double()
    blk = _mx_block(fmt)
    n, k = st["wq"].shape[0], x.shape[1]
    xb = x.reshape(x.shape[0], k // blk, blk)
    amax = xb.abs().max(-1).values
    if fmt == "mxfp4":
        # floor(log2) from the exponent bits: a logarithm may fall short at powers of two
        d = torch.exp2(((amax.view(torch.int64) >> 52) - 1023 - 2).double())
        d[amax == 0] = 2.0 ** -127
        g = 1.0
    else:
        # float32 roundings as the format's recipe has them: 6 g, the quotient, s g
        gx = st["gx"]
        s = (amax.float() / (6 * gx)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
        d, g = (s * gx).double(), gx.double() * st["gw"].double()
    v = (xb / d[..., None].clamp(min=2.0 ** -140)).float().double()
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    mid = (level[1:] + level[:-1]) / 2
    up, down = torch.bucketize(v.abs(), mid, right=True), torch.bucketize(v.abs(), mid, right=False)
    idx = torch.where(up % 2 == 0, up, down)          # a tie goes to the even code
    xd = level[idx] * torch.sign(v)
    xd = xd * (d if fmt == "mxfp4" else s.double())[..., None]
    xd = xd.reshape(x.shape)
    signed = torch.cat((level, -level))
    y = torch.empty(x.shape[0], n, dtype=torch.float64, device="cuda")
    sbytes = _mx_scale_from_tiles(st["ws"], n, k // blk)
    step = max(1, (1 << 27) // k)
    for i in range(0, n, step):
        byte = st["wq"][i:i + step].long()
        w = torch.stack((signed[byte % 16], signed[byte // 16]), -1).reshape(byte.shape[0], k // blk, blk)
        sb = sbytes[i:i + step]
        sc = torch.exp2(sb.double() - 127) if fmt == "mxfp4" else sb.view(torch.float8_e4m3fn).double()
        y[:, i:i + step] = xd @ (w * sc[..., None]).reshape(-1, k).t()
    return y * g
