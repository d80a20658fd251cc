"""Microscaled 4-bit floating point on the host: refusals of the C ABI before
any launch (fake addresses), sizes, and the oracle against hand-worked values."""
import numpy as np
import pytest

from int4_linear_b200 import fq
from oracle import mx_oracle as MO

A = 1 << 20


@pytest.fixture(scope="module")
def L():
    from int4_linear_b200 import build
    build.build()
    return fq.lib()


@pytest.mark.parametrize("change,status,msg", [
    (dict(R=0), fq.FQ_ERR_INVALID, b"rows"), (dict(K=64), fq.FQ_ERR_INVALID, b"K"),
    (dict(K=200), fq.FQ_ERR_INVALID, b"K"), (dict(K=65536 + 128, ldx=1 << 17), fq.FQ_ERR_INVALID, b"K"),
    (dict(fmt=2), fq.FQ_ERR_UNSUPPORTED, b"format"), (dict(g=A), fq.FQ_ERR_INVALID, b"tensor scale"),
    (dict(fmt=1, g=A + 2), fq.FQ_ERR_INVALID, b"aligned"), (dict(X=None), fq.FQ_ERR_INVALID, b"NULL"),
    (dict(X=A + 8), fq.FQ_ERR_INVALID, b"aligned"), (dict(Q=A + 4), fq.FQ_ERR_INVALID, b"aligned"),
    (dict(S=None), fq.FQ_ERR_INVALID, b"NULL"), (dict(ldx=248), fq.FQ_ERR_INVALID, b"ldx"),
    (dict(ldx=260), fq.FQ_ERR_INVALID, b"ldx")])
def test_quant_refusals(L, change, status, msg):
    a = dict(X=A, ldx=256, R=3, K=256, fmt=0, g=None, Q=A, S=A)
    a.update(change)
    assert L.fq_mx_quant(a["X"], a["ldx"], a["R"], a["K"], a["fmt"], a["g"], a["Q"], a["S"], None) == status
    assert msg in L.fq_last_error()
    if "ldx" not in change:
        st = L.fq_mx_dequant(a["Q"], a["S"], a["R"], a["K"], a["fmt"], a["g"], a["X"], None)
        assert st == status and msg in L.fq_last_error()


@pytest.mark.parametrize("change,status,msg", [
    (dict(M=0), fq.FQ_ERR_INVALID, b"M"), (dict(N=12), fq.FQ_ERR_INVALID, b"N"), (dict(N=0), fq.FQ_ERR_INVALID, b"N"),
    (dict(K=192), fq.FQ_ERR_INVALID, b"K"), (dict(K=0), fq.FQ_ERR_INVALID, b"K"),
    (dict(fmt=7), fq.FQ_ERR_UNSUPPORTED, b"format"), (dict(gx=A), fq.FQ_ERR_INVALID, b"tensor scales"),
    (dict(fmt=1, gw=A + 1), fq.FQ_ERR_INVALID, b"aligned"), (dict(X=A + 8), fq.FQ_ERR_INVALID, b"aligned"),
    (dict(W=None), fq.FQ_ERR_INVALID, b"NULL"), (dict(Sw=A + 8), fq.FQ_ERR_INVALID, b"aligned"),
    (dict(Y=A + 2), fq.FQ_ERR_INVALID, b"aligned"), (dict(ws=None), fq.FQ_ERR_INVALID, b"workspace"),
    (dict(ws=A + 64), fq.FQ_ERR_INVALID, b"workspace"), (dict(wsb=-1), fq.FQ_ERR_INVALID, b"workspace")])
def test_product_and_linear_refusals(L, change, status, msg):
    a = dict(X=A, Sx=A, gx=None, W=A, Sw=A, gw=None, M=3, N=256, K=512, fmt=0, Y=A, ws=A, wsb=0)
    a.update(change)
    need = L.fq_mx_gemm_workspace_size(3, 256, 512, 0) + a["wsb"]
    st = L.fq_mx_gemm(a["X"], a["Sx"], a["gx"], a["W"], a["Sw"], a["gw"], a["M"], a["N"], a["K"], a["fmt"], a["Y"],
                      a["ws"], need, None)
    assert st == status and msg in L.fq_last_error()
    need = L.fq_mx_linear_workspace_size(3, 256, 512, 0) + a["wsb"]
    st = L.fq_mx_linear(a["X"], 512, a["M"], a["K"], a["fmt"], a["gx"], a["W"], a["Sw"], a["gw"], a["N"], a["Y"],
                        a["ws"], need, None)
    assert st == status and msg in L.fq_last_error()


@pytest.mark.parametrize("m,n", [(2 ** 31 - 1, 8), (2 ** 30 + 1, 8), (1, 2 ** 31 - 8), (1, 2 ** 30 + 8)])
def test_sizes_past_the_tile_arithmetic_are_refused(L, m, n):
    assert L.fq_mx_gemm_workspace_size(m, n, 128, 0) == 0 and L.fq_mx_linear_workspace_size(m, n, 128, 0) == 0
    assert L.fq_mx_gemm(A, A, None, A, A, None, m, n, 128, 0, A, A, 1 << 20, None) == fq.FQ_ERR_INVALID
    assert b"sizes" in L.fq_last_error()
    assert L.fq_mx_linear(A, 128, m, 128, 0, None, A, A, None, n, A, A, 1 << 20, None) == fq.FQ_ERR_INVALID
    assert b"sizes" in L.fq_last_error()


def test_sizes(L):
    assert L.fq_mx_scale_bytes(1, 128, 0) == 128 * 4 and L.fq_mx_scale_bytes(129, 256, 1) == 256 * 16
    assert L.fq_mx_scale_bytes(0, 128, 0) == 0 and L.fq_mx_scale_bytes(1, 100, 0) == 0
    assert L.fq_mx_scale_bytes(1, 128, 2) == 0
    assert L.fq_mx_gemm_workspace_size(2048, 28672, 4096, 0) == 0
    for m, n, k, fmt in ((1, 6144, 4096, 0), (64, 4096, 14336, 1), (2048, 28672, 4096, 1)):
        assert (L.fq_mx_linear_workspace_size(m, n, k, fmt) >= max(fq.SYNC_BYTES, L.fq_mx_gemm_workspace_size(m, n, k, fmt))
                + m * k // 2 + L.fq_mx_scale_bytes(m, k, fmt))
    assert L.fq_mx_gemm_workspace_size(1, 12, 128, 0) == 0 and L.fq_mx_linear_workspace_size(0, 8, 128, 0) == 0


# ---------------------------------------------------------------- the oracle

def test_oracle_mxfp4_worked():
    """amax 7: e = 2 - 2 = 0; ties go to the even code, 7 saturates at 6."""
    x = np.zeros((1, 128), np.float16)
    x[0, :12] = [7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, 0.2500001, -0.26, 4.9]
    x[0, 32:35] = [12, 5, -1]            # amax 12: e = 1, values halved
    code, sb = MO.quant(x, MO.MXFP4)
    assert sb[0].tolist() == [127, 128, 0, 0]
    assert code[0, :12].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 14, 0, 9, 6]
    assert code[0, 32:35].tolist() == [7, 4, 9]
    v = MO.values(code, sb, MO.MXFP4)
    assert v[0, 32:35].tolist() == [12, 4, -1] and v[0, 0] == 6


def test_oracle_nvfp4_worked():
    """g = 1/8, amax 3: s = e4m3(3 / 0.75) = 4, divisor 0.5; amax 2000 saturates the scale at 448."""
    x = np.zeros((1, 128), np.float16)
    x[0, :4] = [3, 1.25, -0.125, 0.4]
    x[0, 16:18] = [2000, -20]
    code, sb = MO.quant(x, MO.NVFP4, 0.125)
    assert MO.scale_value(sb, MO.NVFP4)[0, :3].tolist() == [4, 448, 0]
    assert code[0, :4].tolist() == [7, 4, 8, 2]       # 6, 2.5 -> 2, -0.25 -> -0, 0.8 -> 1
    assert code[0, 16:18].tolist() == [7, 9]          # 35.7 -> 6; -0.357 -> -0.5
    assert MO.E4M3[0b0_0001_000] == 2.0 ** -6 and MO.E4M3[1] == 2.0 ** -9 and MO.E4M3[126] == 448


def test_oracle_tiles_and_product():
    g = np.random.Generator(np.random.PCG64(0))
    sb = g.integers(0, 255, (300, 8)).astype(np.uint8)
    t = MO.to_tiles(sb)
    assert t.size == 384 * 8 and np.array_equal(MO.from_tiles(t, 300, 8), sb)
    # row 0's first four scales lie together, row 32's behind them, row 1's 16 bytes on
    assert np.array_equal(t[:4], sb[0, :4]) and np.array_equal(t[4:8], sb[32, :4]) and np.array_equal(t[16:20], sb[1, :4])
    assert np.array_equal(t[512:516], sb[0, 4:]) and np.array_equal(t[1024:1028], sb[128, :4])
    xc, xs = MO.quant(g.standard_normal((3, 128)), MO.MXFP4)
    wc, ws = MO.quant(g.standard_normal((5, 128)), MO.MXFP4)
    y, _ = MO.product(xc, xs, wc, ws, MO.MXFP4)
    def one(code, scale):
        return MO.LEVELS[code & 7] * (-1.0 if code > 7 else 1.0) * 2.0 ** (int(scale) - 127)

    ref = sum(one(xc[1, k], xs[1, k // 32]) * one(wc[4, k], ws[4, k // 32]) for k in range(128))
    assert abs(y[1, 4] - ref) < 1e-12
    assert np.array_equal(MO.unpack(MO.pack(xc)), xc)
