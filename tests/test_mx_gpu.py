"""Microscaled 4-bit floating point on the GPU against the oracle.

Codes, scales and the values read back are single roundings of exact or
stated float32 quantities: compared bit for bit.

Product.  Each term code * code * s * s is exact in float32.  A K step of 64
terms and the running sum are added by one instruction: at most 64 terms and
the sum, each cut at 2^-23 of the largest magnitude, and K / 64 instructions;
a divided K adds at most K / 256 more float32 sums.  With B the sum of the
terms' magnitudes an output is off by at most (64 + K/64 + K/256) 2^-23 B
before its rounding to fp16 (2^-11 |y|, 2^-25 below the normal range), and two float32 products
with g_x, g_w (2^-23 |y|).  Where every sum fits 24 bits the result is compared bit for bit.
"""
import numpy as np
import pytest
import torch

from int4_linear_b200 import fq
from oracle import mx_oracle as MO

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rng(*seed):
    return np.random.Generator(np.random.PCG64(list(seed)))


def f32(v):
    return torch.full((1,), v, dtype=torch.float32, device="cuda")


FMTS = [MO.MXFP4, MO.NVFP4]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("r,k", [(1, 128), (3, 384), (127, 256), (128, 128), (129, 1152), (1000, 640), (2, 65536)])
def test_quant_bits(fmt, r, k):
    g = rng(1, r, k, fmt)
    x = (g.standard_normal((r, k)) * 2.0 ** g.uniform(-8, 6, (r, 1))).astype(np.float16)
    x[0, :32] = 0
    x[r // 2, 32:64] = np.float16(2.0 ** -24) * g.integers(0, 8, 32)       # subnormal inputs
    x[-1, 64:96] = np.array([65504, -65504, 1, -0.0] * 8, np.float16)
    # exact ties and powers of two
    x[r // 3, 96:128] = np.array([7, 0.25, -0.75, 1.25, 1.75, 2.5, 3.5, 5, 8, 4, 2, 1, 0.5, 0, -5, 6] * 2, np.float16)
    gs = None if fmt == MO.MXFP4 else np.float32(0.0173)
    code, sb = MO.quant(x, fmt, gs)
    buf = torch.full((r, k + 40), 3.0, dtype=torch.float16, device="cuda")
    buf[:, 16:16 + k] = dev(x)
    q, s = fq.fq_mx_quant(buf[:, 16:16 + k], fmt, None if gs is None else f32(gs))
    assert np.array_equal(q.cpu().numpy(), MO.pack(code))
    b = k // MO.block(fmt)
    assert np.array_equal(MO.from_tiles(s.cpu().numpy(), r, b), sb)
    back = fq.fq_mx_dequant(q, s, fmt, None if gs is None else f32(gs)).cpu().numpy()
    d = MO.scale_value(sb, fmt).astype(np.float32)
    if gs is not None:
        d = d * gs
    v = (MO.LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)).astype(np.float32) * np.repeat(d, MO.block(fmt), 1)
    assert np.array_equal(back, v.astype(np.float16))


@pytest.mark.parametrize("gs", [None, 1.0, 2.0 ** -10, 1e-6, 3.7])
def test_nvfp4_tensor_scales(gs):
    """Scales that round to zero, saturate, and the power-of-two scales whose quotients tie."""
    g = rng(2)
    x = (g.standard_normal((64, 256)) * 2.0 ** g.uniform(-12, 12, (64, 16)).repeat(16, 1)).astype(np.float16)
    code, sb = MO.quant(x, MO.NVFP4, gs)
    q, s = fq.fq_mx_quant(dev(x), MO.NVFP4, None if gs is None else f32(gs))
    assert np.array_equal(MO.from_tiles(s.cpu().numpy(), 64, 16), sb)
    assert np.array_equal(q.cpu().numpy(), MO.pack(code))


@pytest.mark.parametrize("fmt", FMTS)
def test_non_finite_blocks(fmt):
    """A block with Inf or NaN gets a NaN scale; its rows of the product are NaN, the others untouched."""
    g = rng(3)
    x = g.standard_normal((20, 256)).astype(np.float16)
    x[3, 40], x[7, 255], x[11, 0] = np.inf, np.nan, -np.inf
    code, sb = MO.quant(x, fmt)
    q, s = fq.fq_mx_quant(dev(x), fmt)
    assert np.array_equal(MO.from_tiles(s.cpu().numpy(), 20, 256 // MO.block(fmt)), sb)
    assert np.array_equal(q.cpu().numpy(), MO.pack(code))
    assert np.isnan(fq.fq_mx_dequant(q, s, fmt)[3, 32:48].cpu().numpy()).all()
    w = dev(g.standard_normal((40, 256)).astype(np.float16))
    wq, ws = fq.fq_mx_quant(w, fmt)
    y = fq.fq_mx_gemm(q, s, wq, ws, fmt).cpu().numpy()
    bad = np.isnan(y).all(1)
    assert bad.tolist() == [i in (3, 7, 11) for i in range(20)] and np.isfinite(y[~bad]).all()


def random_operand(g, r, k, fmt, spread):
    """Random codes; scales 2^+-spread (E8M0) or any E4M3 values in that range."""
    code = g.integers(0, 16, (r, k)).astype(np.uint8)
    b = k // MO.block(fmt)
    if fmt == MO.MXFP4:
        sb = g.integers(127 - spread, 128 + spread, (r, b)).astype(np.uint8)
    else:
        sb = g.integers(8 * (7 - spread), 8 * (7 + spread) + 1, (r, b)).astype(np.uint8)
    return code, sb


def upload(code, sb):
    return dev(MO.pack(code)), dev(MO.to_tiles(sb, fill=0xFF))    # NaN in the padding rows


# every token-tile width, ragged edges on all sides
SHAPES = [(1, 8, 128), (1, 136, 256), (5, 128, 384), (16, 1000, 512), (17, 256, 128), (32, 72, 640), (33, 520, 256),
          (64, 384, 1152), (65, 128, 256), (100, 264, 384), (128, 128, 128), (129, 136, 256), (255, 256, 512),
          (256, 128, 384), (300, 1032, 256), (513, 264, 128)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_exact_sums(fmt, m, n, k):
    """Codes times scales whose sums fit 24 bits: bit for bit, so a code or scale taken from
    the wrong place shows."""
    g = rng(4, m, n, k, fmt)
    if fmt == MO.MXFP4:
        xc, xs = random_operand(g, m, k, fmt, 2)
        wc, ws = random_operand(g, n, k, fmt, 2)
    else:
        # E4M3 scales 1, 1.5, 2, 3: products in quarters of quarters
        xc, wc = (g.integers(0, 16, (r, k)).astype(np.uint8) for r in (m, n))
        pick = np.array([0x38, 0x3C, 0x40, 0x44], np.uint8)
        xs, ws = (pick[g.integers(0, 4, (r, k // 16))] for r in (m, n))
    acc, _ = MO.product(xc, xs, wc, ws, fmt)
    xq, sx = upload(xc, xs)
    wq, sw = upload(wc, ws)
    y = fq.fq_mx_gemm(xq, sx, wq, sw, fmt)
    fq.fq_check_device_error()
    assert np.array_equal(y.cpu().numpy(), acc.astype(np.float16))


def check_product(y, acc, mag, k, scale=1.0):
    ref = acc * scale
    tol = (64 + k / 64 + k / 256) * 2.0 ** -23 * mag * abs(scale) + (2.0 ** -11 + 2.0 ** -23) * np.abs(ref) + 2.0 ** -25
    err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3f} of the bound"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", [(1, 6144, 4096), (3, 520, 28672), (40, 2056, 2176), (64, 4096, 1024),
                                   (200, 1544, 4224), (777, 1000, 896), (130, 128, 16384), (1500, 2048, 512)])
def test_product_wide_scales(fmt, m, n, k):
    g = rng(5, m, n, k, fmt)
    xc, xs = random_operand(g, m, k, fmt, 5)
    wc, ws = random_operand(g, n, k, fmt, 5)
    xq, sx = upload(xc, xs)
    wq, sw = upload(wc, ws)
    acc, mag = MO.product(xc, xs, wc, ws, fmt)
    scale = 2.0 ** -14
    if fmt == MO.MXFP4:
        xs -= 14
        y = fq.fq_mx_gemm(xq, dev(MO.to_tiles(xs)), wq, sw, fmt)
    else:
        gx, gw = np.float32(2.0 ** -9 * 1.1), np.float32(2.0 ** -5)
        scale = float(gx * gw)
        y = fq.fq_mx_gemm(xq, sx, wq, sw, fmt, f32(gx), f32(gw))
    fq.fq_check_device_error()
    check_product(y, acc, mag, k, scale)


# divided: few tiles of many stages, tiles in many parts, parts of three tiles; whole: several tiles a CTA
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", [(1, 8, 65536), (16, 1160, 20608), (20, 264, 16512), (32, 4096, 8320), (50, 1000, 20608),
                                   (64, 2048, 14336), (5, 20000, 8192), (33, 40000, 640), (7, 38400, 384)])
def test_product_divided_and_whole(fmt, m, n, k):
    test_product_wide_scales(fmt, m, n, k)


# pairs: a last round of whole tiles, of half tiles, with a last token tile that has one half only, ragged in it
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", [(1024, 6144, 384), (1000, 6400, 256), (850, 5000, 640), (1100, 5120, 128), (513, 6528, 384),
                                   (1536, 3328, 512), (512, 14336, 128), (700, 19000, 256)])
def test_product_last_round(fmt, m, n, k):
    test_product_wide_scales(fmt, m, n, k)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", [(1, 512, 1024), (16, 1024, 2048), (77, 512, 640), (513, 768, 1024)])
def test_linear(fmt, m, n, k):
    """Quantization and product in one call, strided rows, against the oracle's own quantization."""
    g = rng(6, m, n, k, fmt)
    x = g.standard_normal((m, k)).astype(np.float16)
    x[:, ::50] *= 10
    w = (g.standard_normal((n, k)) * 0.05).astype(np.float16)
    gx, gw = (None, None) if fmt == MO.MXFP4 else (np.float32(0.02), np.float32(1e-4))
    xc, xs = MO.quant(x, fmt, gx)
    wc, ws = MO.quant(w, fmt, gw)
    acc, mag = MO.product(xc, xs, wc, ws, fmt)
    dgx, dgw = (None, None) if gx is None else (f32(gx), f32(gw))
    wq, sw = fq.fq_mx_quant(dev(w), fmt, dgw)
    buf = torch.zeros(m, k + 64, dtype=torch.float16, device="cuda")
    buf[:, 64:] = dev(x)
    wsp = fq.fq_mx_linear_workspace(m, n, k, fmt)
    y = fq.fq_mx_linear(buf[:, 64:], fmt, wq, sw, dgx, dgw, workspace=wsp)
    check_product(y, acc, mag, k, 1.0 if gx is None else float(gx * gw))
    assert not wsp[:fq.SYNC_BYTES].any()
    for _ in range(10):
        assert torch.equal(fq.fq_mx_linear(buf[:, 64:], fmt, wq, sw, dgx, dgw, workspace=wsp), y)
    # a fresh workspace whose bytes past the counters are garbage
    wsp = torch.full_like(wsp, 0x5A)
    wsp[:fq.SYNC_BYTES] = 0
    assert torch.equal(fq.fq_mx_linear(buf[:, 64:], fmt, wq, sw, dgx, dgw, workspace=wsp), y)


def test_linear_captured_and_replayed_on_new_inputs():
    g = rng(7)
    fmt = MO.MXFP4
    w = (g.standard_normal((640, 512)) * 0.05).astype(np.float16)
    wq, sw = fq.fq_mx_quant(dev(w), fmt)
    wc, ws = MO.quant(w, fmt)
    x = torch.zeros(9, 512, dtype=torch.float16, device="cuda")
    y = torch.empty(9, 640, dtype=torch.float16, device="cuda")
    wsp = fq.fq_mx_linear_workspace(9, 640, 512, fmt)
    fq.fq_mx_linear(x, fmt, wq, sw, Y=y, workspace=wsp)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fq.fq_mx_linear(x, fmt, wq, sw, Y=y, workspace=wsp)
    for _ in range(3):
        xn = g.standard_normal((9, 512)).astype(np.float16)
        x.copy_(dev(xn))
        graph.replay()
        xc, xs = MO.quant(xn, fmt)
        acc, mag = MO.product(xc, xs, wc, ws, fmt)
        check_product(y, acc, mag, 512)


def test_rows_outside_the_output_stay():
    g = rng(8)
    fmt = MO.NVFP4
    for m in (1, 20, 140, 300):
        xq, sx = fq.fq_mx_quant(dev(g.standard_normal((m, 256)).astype(np.float16)), fmt)
        wq, sw = fq.fq_mx_quant(dev(g.standard_normal((136, 256)).astype(np.float16)), fmt)
        buf = torch.full((m + 2, 136), 5.0, dtype=torch.float16, device="cuda")
        fq.fq_mx_gemm(xq, sx, wq, sw, fmt, Y=buf[1:-1])
        assert (buf[0] == 5).all() and (buf[-1] == 5).all()


def test_output_overflows_to_infinity():
    x = torch.full((2, 128), 60000.0, dtype=torch.float16, device="cuda")
    q, s = fq.fq_mx_quant(x, MO.MXFP4)
    w = torch.ones(8, 128, dtype=torch.float16, device="cuda")
    w[1] = -1
    wq, sw = fq.fq_mx_quant(w, MO.MXFP4)
    y = fq.fq_mx_gemm(q, s, wq, sw, MO.MXFP4)
    assert torch.isposinf(y[:, 0]).all() and torch.isneginf(y[:, 1]).all()


def test_binding_refusals():
    x = torch.zeros(4, 256, dtype=torch.float16, device="cuda")
    q, s = fq.fq_mx_quant(x, MO.MXFP4)
    for bad in (x.float(), x.t(), x[0]):
        with pytest.raises(ValueError):
            fq.fq_mx_quant(bad, MO.MXFP4)
    with pytest.raises(ValueError):
        fq.fq_mx_gemm(q, s[:-1], q, s, MO.MXFP4)
    with pytest.raises(ValueError):
        fq.fq_mx_gemm(q, s, q, s, MO.NVFP4)              # scales of the other format
    with pytest.raises(ValueError):
        fq.fq_mx_linear(x[:, :128], MO.MXFP4, q, s)
    with pytest.raises(fq.FqError):
        fq.fq_mx_gemm(q, s, q, s, MO.MXFP4)              # N = 4
    with pytest.raises(fq.FqError):
        fq.fq_mx_quant(torch.zeros(4, 200, dtype=torch.float16, device="cuda"), MO.MXFP4)
