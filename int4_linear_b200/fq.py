"""Python binding of libfq.so (C ABI in include/fq.h).

Argument marshalling only: every function checks tensor dtypes/devices,
allocates outputs through PyTorch when the caller gives none, and calls the
C entry point of the same name on the current (or given) CUDA stream.  All
arithmetic runs in the library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass

import torch

ROW, GROUP, STATIC, ROW_ZP, STATIC_RESIDUAL = 0, 1, 2, 3, 4  # fq_gran
SYNC_BYTES = 16384  # FQ_WORKSPACE_SYNC_BYTES: leading workspace bytes kept zero between calls
GROUP_SIZE = 128
MXFP4, NVFP4 = 0, 1  # fq_mx_format
ZERO_POINT_MINMAX = -1                   # fq_qparams.zero_point: per-row min-max (asymmetric) quantizer

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfq.so")

FQ_OK, FQ_ERR_INVALID, FQ_ERR_UNSUPPORTED, FQ_ERR_CUDA, FQ_ERR_TIMEOUT = range(5)


class FqError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (status {status})")
        self.status = status


class QParams(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int), ("zero_point", ctypes.c_int), ("gran", ctypes.c_int),
                ("group_size", ctypes.c_int), ("alpha", ctypes.c_float)]


class _Transform(ctypes.Structure):
    _fields_ = [("n1", ctypes.c_int), ("n2", ctypes.c_int), ("P1", ctypes.c_void_p),
                ("P2", ctypes.c_void_p), ("c", ctypes.c_void_p)]


@dataclass
class Transform:
    """Kronecker factors (device float32) and channel scale.  For fq_quant_weight
    pass the inverses P1^-1, P2^-1 (and the same c)."""
    P1: torch.Tensor | None = None
    P2: torch.Tensor | None = None
    c: torch.Tensor | None = None

    n1: int = 0  # with P1 None and P2 given: the number of rows of the reshape (P1 = I)

    def as_c(self) -> _Transform:
        t = _Transform()
        if self.P1 is not None or self.P2 is not None:
            _check(self.P1, torch.float32, "P1")
            _check(self.P2, torch.float32, "P2")
            t.n1 = self.P1.shape[0] if self.P1 is not None else self.n1
            t.n2 = self.P2.shape[0]
            t.P1 = self.P1.data_ptr() if self.P1 is not None else None
            t.P2 = self.P2.data_ptr()
        if self.c is not None:
            _check(self.c, torch.float32, "c")
            t.c = self.c.data_ptr()
        return t


class _KVCache(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("H", ctypes.c_int)]


_HEAD_SCALE = 128 ** -0.5
KV_TOKEN_BYTES = 132  # per token and head: K and V codes (64 bytes each), two fp16 scales


class KVCache:
    """A paged INT4 key/value cache: pool uint8 [num_pages, H, page_size * 132]
    (the bytes of a page and head: see fq_kv_cache in fq.h).  Make an empty one
    with kv_cache()."""

    def __init__(self, pool: torch.Tensor):
        _check(pool, torch.uint8, "pool")
        if pool.dim() != 3 or pool.shape[2] % KV_TOKEN_BYTES:
            raise ValueError("pool must be [num_pages, H, page_size * 132]")
        self._pool = pool
        self.num_pages, self.heads = pool.shape[:2]
        self.page_size = pool.shape[2] // KV_TOKEN_BYTES
        self._c = _KVCache(pool.data_ptr(), self.num_pages, self.page_size, self.heads)
        self._ref = ctypes.byref(self._c)

    @property
    def pool(self) -> torch.Tensor:
        return self._pool

    def views(self):
        """(K codes [P, H, page, 64], V codes, K scales fp16 [P, H, page], V scales): views of the pool."""
        n = self.page_size
        parts = self._pool.split([64 * n, 64 * n, 2 * n, 2 * n], dim=-1)
        kq, vq = (x.unflatten(-1, (n, 64)) for x in parts[:2])
        ks, vs = (x.view(torch.float16) for x in parts[2:])
        return kq, vq, ks, vs


def kv_cache(num_pages: int, heads: int, page_size: int, device="cuda") -> KVCache:
    """An empty cache of num_pages pages of page_size (16, 32, 64 or 128) tokens."""
    return KVCache(torch.zeros(num_pages, heads, page_size * KV_TOKEN_BYTES, dtype=torch.uint8, device=device))


def qparams(gran: int = ROW, alpha: float = 1.0, bits: int = 4, zero_point: int = 8,
            group_size: int = GROUP_SIZE) -> QParams:
    return QParams(bits, zero_point, gran, group_size, alpha)


_lib = None


def lib():
    """Load libfq.so (raises if it was not built: there is no other code path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FqError(FQ_ERR_CUDA, f"{LIB_PATH} is missing: build it with python -m int4_linear_b200.build")
    L = ctypes.CDLL(LIB_PATH)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    ll = ctypes.c_longlong
    qp, tp, kc = ctypes.POINTER(QParams), ctypes.POINTER(_Transform), ctypes.POINTER(_KVCache)
    sigs = {
        "fq_quant_weight": [vp, i, i, qp, tp, vp, vp, vp, vp],
        "fq_quant_act": [vp, i, i, qp, tp, vp, vp, vp, vp],
        "fq_quant_act_debug": [vp, i, i, qp, tp, vp, vp, vp, vp, vp],
        "fq_w4a4_gemm": [vp, vp, vp, vp, i, i, i, i, vp, vp, sz, vp],
        "fq_w4a4_gemm_s32": [vp, vp, i, i, i, vp, vp],
        "fq_w4a4_gemm_noalloc": [vp, vp, vp, vp, i, i, i, i, vp, vp],
        "fq_linear": [vp, i, i, qp, tp, vp, vp, vp, i, vp, vp, sz, vp],
        "fq_linear_fused": [vp, i, i, qp, tp, vp, vp, vp, i, vp, vp, sz, vp],
        "fq_ternary_linear": [vp, i, i, vp, vp, vp, i, vp, vp],
        "fq_quant_kv": [vp, i, i, vp, ctypes.c_float, vp, vp, vp],
        "fq_ternary_pack": [vp, i, i, vp, vp],
        "fq_kv_plan": [vp, vp, i, i, vp, i, vp, i, vp, vp, vp, vp, i, vp, vp],
        "fq_kv_write": [vp, ll, vp, ll, i, vp, ctypes.c_float, ctypes.c_float, kc, vp],
        "fq_kv_store": [vp, vp, vp, vp, i, vp, kc, vp],
        "fq_kv_read": [kc, vp, i, vp, vp, vp],
        "fq_kv_attn": [vp, ll, i, i, vp, vp, i, kc, ctypes.c_float, i, vp, vp, sz, vp],
        "fq_mx_quant": [vp, ll, i, i, i, vp, vp, vp, vp],
        "fq_mx_dequant": [vp, vp, i, i, i, vp, vp, vp],
        "fq_mx_gemm": [vp, vp, vp, vp, vp, vp, i, i, i, i, vp, vp, sz, vp],
        "fq_mx_linear": [vp, ll, i, i, i, vp, vp, vp, vp, i, vp, vp, sz, vp],
        "fq_check_device_error": [vp],
        "fq_debug_wait_timeout": [ctypes.c_uint, vp],
    }
    for name, args in sigs.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    for name in ("fq_gemm_workspace_size", "fq_linear_workspace_size", "fq_mx_gemm_workspace_size",
                 "fq_mx_linear_workspace_size"):
        f = getattr(L, name)
        f.argtypes = [i, i, i, i]
        f.restype = sz
    L.fq_mx_scale_bytes.argtypes = [i, i, i]
    L.fq_mx_scale_bytes.restype = sz
    L.fq_kv_attn_workspace_size.argtypes = [i, i, i]
    L.fq_kv_attn_workspace_size.restype = sz
    L.fq_status_string.argtypes = [ctypes.c_int]
    L.fq_status_string.restype = ctypes.c_char_p
    L.fq_last_error.argtypes = []
    L.fq_last_error.restype = ctypes.c_char_p
    _lib = L
    return L


def _raise(status: int):
    if status != FQ_OK:
        L = lib()
        raise FqError(status, f"{L.fq_status_string(status).decode()}: {L.fq_last_error().decode()}")


_Tensor = torch.Tensor


def _check(t, dtype, name):
    if t is None:
        return
    if t.__class__ is _Tensor and t.dtype is dtype and t.is_cuda and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _p(t):
    return None if t is None else t.data_ptr()


def _s(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


_current_device = getattr(torch._C, "_cuda_getDevice", None)  # None: a torch without CUDA
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _enter(stream, *tensors):
    """The device of `tensors` (all on one) made current and, where a stream is given, that
    stream, so that what is allocated meanwhile belongs to the stream that uses it.  Returns the stream's
    handle and what the caller closes in the end: None in the usual case, the current device and stream,
    where nothing is entered."""
    if stream is None:
        dev = tensors[0].get_device()
        for t in tensors:
            if t is not None and t.get_device() != dev:
                break
        else:
            if dev == _current_device():
                return _current_stream(dev), None
    dev = -1
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if dev < 0:
                dev = d
            elif d != dev:
                raise ValueError(f"the tensors lie on cuda:{dev} and cuda:{d}, not on one device")
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        elif stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(dev))
    if stream is not None:
        stack.enter_context(torch.cuda.stream(stream))
    return _current_stream(dev), stack


def _check_shape(t, shape, name):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _check_int(value, most, name):
    """A whole number in [0, most]: what passes 32 bits would reach the library cut off."""
    if not 0 <= value <= most:
        raise ValueError(f"{name} = {value} must lie in [0, {most}]")


_INT_MAX = 2 ** 31 - 1


def _size(fn, *sizes) -> int:
    """The bytes that `fn` says for these sizes; 0, as it says for others out of range, where one passes 32 bits."""
    return fn(*sizes) if all(-_INT_MAX <= n <= _INT_MAX for n in sizes) else 0


def _check_fmt(fmt):
    if fmt != MXFP4 and fmt != NVFP4:
        raise FqError(FQ_ERR_UNSUPPORTED, f"unsupported parameters: format {fmt} is not provided")


def _check_rows(t, name, width):
    """fp16 rows of `width` values, any distance apart: [T, width] or [T, H, 128] with dense rows.
    Returns (T, the distance in elements)."""
    if t.__class__ is _Tensor and t.dtype is torch.float16 and t.is_cuda:  # the usual cases
        shape = t.shape
        n = len(shape)
        if n == 2 and shape[1] == width and shape[0] > 0:
            ld, one = t.stride()
            if one == 1:
                return shape[0], ld if shape[0] > 1 else width
        elif n == 3 and shape[2] == 128 and shape[1] * 128 == width and shape[0] > 0 and t.is_contiguous():
            return shape[0], width
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.float16:
        raise ValueError(f"{name} must be torch.float16, got {t.dtype}")
    shape, strides = t.shape, t.stride()
    if len(shape) == 2:
        n, dense = shape[1], strides[1] == 1 or shape[1] == 1
    elif len(shape) == 3:
        if shape[2] != 128:
            raise ValueError(f"{name} must be [T, heads, 128] or [T, heads * 128], got shape {tuple(shape)}")
        n = shape[1] * 128
        dense = strides[2] == 1 and (strides[1] == 128 or shape[1] == 1)
    else:
        n = dense = None
    if n != width or shape[0] < 1:
        raise ValueError(f"{name} must have rows of {width} values, got shape {tuple(shape)}")
    if not dense:
        raise ValueError(f"the rows of {name} must be contiguous")
    return shape[0], (strides[0] if shape[0] > 1 else width)


def _scales_out(gran, rows, k, dev, zero_point=8):
    if gran == ROW and zero_point == ZERO_POINT_MINMAX:
        # float32 s[rows], int32 o[rows] = 2^(b-1) - z, int32 code sums[rows]
        return torch.empty(3, rows, dtype=torch.float32, device=dev)
    if gran in (ROW, STATIC_RESIDUAL):
        return torch.empty(rows, dtype=torch.float32, device=dev)
    if gran == GROUP:
        return torch.empty(k // GROUP_SIZE, rows, dtype=torch.float16, device=dev)
    return None


def fq_quant_weight(W, qp: QParams, inv: Transform | None = None, qsm_scale=None,
                    Wq=None, s_w=None, stream=None):
    """Offline weight quantization: returns (Wq uint8 [N, K/2], s_w)."""
    _check(W, torch.float16, "W")
    _check(qsm_scale, torch.float32, "qsm_scale")
    n, k = W.shape
    Wq = torch.empty(n, k // 2, dtype=torch.uint8, device=W.device) if Wq is None else Wq
    s_w = _scales_out(qp.gran, n, k, W.device, qp.zero_point) if s_w is None else s_w
    t = inv.as_c() if inv is not None else None
    st = lib().fq_quant_weight(W.data_ptr(), n, k, ctypes.byref(qp), ctypes.byref(t) if t else None,
                               _p(qsm_scale), Wq.data_ptr(), _p(s_w), _s(stream))
    _raise(st)
    return Wq, s_w


def fq_quant_act(X, qp: QParams, t: Transform | None = None, static_scale=None,
                 Xq=None, s_x=None, stream=None):
    """Online activation quantization: returns (Xq uint8 [M, K/2], s_x or None)."""
    _check(X, torch.float16, "X")
    _check(static_scale, torch.float32, "static_scale")
    m, k = X.shape
    Xq = torch.empty(m, k // 2, dtype=torch.uint8, device=X.device) if Xq is None else Xq
    s_x = _scales_out(qp.gran, m, k, X.device, qp.zero_point) if s_x is None else s_x
    tc = t.as_c() if t is not None else None
    st = lib().fq_quant_act(X.data_ptr(), m, k, ctypes.byref(qp), ctypes.byref(tc) if tc else None,
                            _p(static_scale), Xq.data_ptr(), _p(s_x), _s(stream))
    _raise(st)
    return Xq, s_x


def fq_quant_act_debug(X, qp: QParams, t: Transform | None = None, static_scale=None, stream=None):
    """fq_quant_act that also returns the float32 transformed values: (Xq, s_x, xhat)."""
    _check(X, torch.float16, "X")
    _check(static_scale, torch.float32, "static_scale")
    m, k = X.shape
    Xq = torch.empty(m, k // 2, dtype=torch.uint8, device=X.device)
    s_x = _scales_out(qp.gran, m, k, X.device, qp.zero_point)
    xhat = torch.empty(m, k, dtype=torch.float32, device=X.device)
    tc = t.as_c() if t is not None else None
    st = lib().fq_quant_act_debug(X.data_ptr(), m, k, ctypes.byref(qp), ctypes.byref(tc) if tc else None,
                                  _p(static_scale), Xq.data_ptr(), _p(s_x), xhat.data_ptr(), _s(stream))
    _raise(st)
    return Xq, s_x, xhat


def split_zero_point_block(block):
    """The min-max quantizer's scale block -> (s float32 [R], o int32 [R] =
    2^(b-1) - z, S int32 [R] = the rows' sums of the stored codes)."""
    b = block.reshape(3, -1)
    return b[0], b[1].view(torch.int32), b[2].view(torch.int32)


def fq_gemm_workspace_size(m, n, k, gran) -> int:
    return int(lib().fq_gemm_workspace_size(m, n, k, gran))


def fq_linear_workspace_size(m, n, k, gran) -> int:
    return int(lib().fq_linear_workspace_size(m, n, k, gran))


def _workspace(nbytes, dev, ws):
    if nbytes == 0:
        return None, 0
    if ws is None:
        # zeroed: the library's counters at the start of a workspace must be 0 on first use
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
    if ws.numel() < nbytes:
        raise ValueError(f"workspace needs {nbytes} bytes")
    return ws, ws.numel()


def fq_w4a4_gemm(Xq, s_x, Wq, s_w, gran: int, Y=None, workspace=None, stream=None):
    """Y fp16 [M, N] = dequant(Xq Wq^T)."""
    _check(Xq, torch.uint8, "Xq")
    _check(Wq, torch.uint8, "Wq")
    m, k2 = Xq.shape
    n = Wq.shape[0]
    k = 2 * k2
    Y = torch.empty(m, n, dtype=torch.float16, device=Xq.device) if Y is None else Y
    _check(Y, torch.float16, "Y")
    ws, wsb = _workspace(fq_gemm_workspace_size(m, n, k, gran), Xq.device, workspace)
    st = lib().fq_w4a4_gemm(Xq.data_ptr(), _p(s_x), Wq.data_ptr(), _p(s_w), m, n, k, gran, Y.data_ptr(),
                            _p(ws), wsb, _s(stream))
    _raise(st)
    return Y


def fq_w4a4_gemm_noalloc(Xq, s_x, Wq, s_w, gran: int, Y=None, stream=None):
    """fq_w4a4_gemm without a workspace, for callers that cannot allocate device
    memory: the library's static 32 MiB scratch holds the split-K partial sums.
    Calls that overlap on the GPU share that scratch and race; keep them on one
    stream.  (Y is allocated here only when the caller passes none.)"""
    _check(Xq, torch.uint8, "Xq")
    _check(Wq, torch.uint8, "Wq")
    m, k2 = Xq.shape
    n = Wq.shape[0]
    Y = torch.empty(m, n, dtype=torch.float16, device=Xq.device) if Y is None else Y
    _check(Y, torch.float16, "Y")
    st = lib().fq_w4a4_gemm_noalloc(Xq.data_ptr(), _p(s_x), Wq.data_ptr(), _p(s_w), m, n, 2 * k2, gran,
                                    Y.data_ptr(), _s(stream))
    _raise(st)
    return Y


def fq_w4a4_gemm_s32(Xq, Wq, acc=None, stream=None):
    """The exact int32 accumulators [M, N]."""
    _check(Xq, torch.uint8, "Xq")
    _check(Wq, torch.uint8, "Wq")
    m, k2 = Xq.shape
    n = Wq.shape[0]
    acc = torch.empty(m, n, dtype=torch.int32, device=Xq.device) if acc is None else acc
    _check(acc, torch.int32, "acc")
    st = lib().fq_w4a4_gemm_s32(Xq.data_ptr(), Wq.data_ptr(), m, n, 2 * k2, acc.data_ptr(), _s(stream))
    _raise(st)
    return acc


def fq_linear(X, qp: QParams, Wq, s_w, t: Transform | None = None, static_scale=None,
              Y=None, workspace=None, stream=None, fused=False):
    """Y fp16 [M, N] = dequant(Q(X P) Q(P^-1 W^T)), quantization + GEMM on one
    stream (fused=True: fq_linear_fused, one launch at decode sizes)."""
    _check(X, torch.float16, "X")
    _check(Wq, torch.uint8, "Wq")
    _check(static_scale, torch.float32, "static_scale")
    m, k = X.shape
    n = Wq.shape[0]
    Y = torch.empty(m, n, dtype=torch.float16, device=X.device) if Y is None else Y
    _check(Y, torch.float16, "Y")
    gran = ROW_ZP if qp.zero_point == ZERO_POINT_MINMAX else qp.gran
    ws, wsb = _workspace(fq_linear_workspace_size(m, n, k, gran), X.device, workspace)
    tc = t.as_c() if t is not None else None
    fn = lib().fq_linear_fused if fused else lib().fq_linear
    st = fn(X.data_ptr(), m, k, ctypes.byref(qp), ctypes.byref(tc) if tc else None,
                         _p(static_scale), Wq.data_ptr(), _p(s_w), n, Y.data_ptr(), _p(ws), wsb,
                         _s(stream))
    _raise(st)
    return Y


def fq_quant_kv(KV, P_h, alpha: float = 1.0, Q=None, scales=None, stream=None):
    """INT4 key/value cache: KV fp16 [T, H, 128] (or [T, H * 128]) with the
    per-head transform P_h [128, 128] -> (Q uint8 [T, H * 64], scales fp16 [T, H])."""
    _check(KV, torch.float16, "KV")
    _check(P_h, torch.float32, "P_h")
    t = KV.shape[0]
    h = KV[0].numel() // 128
    Q = torch.empty(t, h * 64, dtype=torch.uint8, device=KV.device) if Q is None else Q
    scales = torch.empty(t, h, dtype=torch.float16, device=KV.device) if scales is None else scales
    _raise(lib().fq_quant_kv(KV.data_ptr(), t, h, P_h.data_ptr(), alpha, Q.data_ptr(), scales.data_ptr(),
                             _s(stream)))
    return Q, scales


def fq_kv_plan(lens, new_tokens, block_table, free_pages, pages_used, page_size: int, max_tokens: int,
               lens_out=None, token_start=None, slots=None, pages_used_out=None, stream=None):
    """Block tables and slots of one step from the request lengths: lens, new_tokens int32 [R],
    block_table int32 [R, max_pages] (updated in place), free_pages int32 [F], pages_used int32 [1].
    Returns (lens_out [R], token_start [R + 1], slots [max_tokens], pages_used_out [1])."""
    i32 = torch.int32
    _check(lens, i32, "lens")
    _check(new_tokens, i32, "new_tokens")
    _check(block_table, i32, "block_table")
    _check(free_pages, i32, "free_pages")
    _check(pages_used, i32, "pages_used")
    r = lens.numel()
    table_shape = block_table.shape
    if lens.dim() != 1 or len(table_shape) != 2 or table_shape[0] != r:
        raise ValueError(f"lens must be [R] and block_table [R, max_pages], got {tuple(lens.shape)} and "
                         f"{tuple(table_shape)}")
    _check_shape(new_tokens, (r,), "new_tokens")
    _check_shape(pages_used, (1,), "pages_used")
    max_pages, num_free = table_shape[1], free_pages.numel()
    if not (0 <= page_size <= _INT_MAX and 0 <= max_tokens <= 1 << 30 and max_pages <= _INT_MAX and num_free <= _INT_MAX):
        _check_int(page_size, _INT_MAX, "page_size")
        _check_int(max_tokens, 1 << 30, "max_tokens")
        _check_int(max_pages, _INT_MAX, "max_pages")
        _check_int(num_free, _INT_MAX, "the number of free pages")
    s, entered = _enter(stream, lens, new_tokens, block_table, free_pages, pages_used, lens_out, token_start, slots,
                        pages_used_out)
    try:
        if lens_out is None and token_start is None and slots is None and pages_used_out is None:
            # one allocation for the four
            lens_out, token_start, slots, pages_used_out = torch.unsafe_split_with_sizes(
                lens.new_empty(2 * r + 2 + max_tokens), [r, r + 1, max_tokens, 1])
        else:
            sizes = (r, r + 1, max_tokens, 1)
            given = (lens_out, token_start, slots, pages_used_out)
            for t, n, name in zip(given, sizes, ("lens_out", "token_start", "slots", "pages_used_out")):
                if t is not None:
                    _check(t, i32, name)
                    _check_shape(t, (n,), name)
            lens_out, token_start, slots, pages_used_out = (
                lens.new_empty(n) if t is None else t for t, n in zip(given, sizes))
        _raise(lib().fq_kv_plan(lens.data_ptr(), new_tokens.data_ptr(), r, page_size, block_table.data_ptr(),
                                max_pages, free_pages.data_ptr() or None, num_free,
                                pages_used.data_ptr(), lens_out.data_ptr(), token_start.data_ptr(),
                                slots.data_ptr() or None, max_tokens, pages_used_out.data_ptr(), s))
    finally:
        if entered is not None:
            entered.close()
    return lens_out, token_start, slots, pages_used_out


def _check_slots(slots, t):
    _check(slots, torch.int32, "slots")
    _check_shape(slots, (t,), "slots")


def fq_kv_write(K, V, slots, cache: KVCache, alpha_k: float = 1.0, alpha_v: float = 1.0, stream=None):
    """New keys and values (fp16 [T, H, 128] or [T, H * 128], rows any distance apart) into the
    cache's slots (int32 [T], -1: skipped) as INT4."""
    width = cache.heads * 128
    t, ldk = _check_rows(K, "K", width)
    tv, ldv = _check_rows(V, "V", width)
    if tv != t:
        raise ValueError(f"K has {t} rows, V {tv}")
    _check_slots(slots, t)
    s, entered = _enter(stream, K, V, slots, cache.pool)
    try:
        _raise(lib().fq_kv_write(K.data_ptr(), ldk, V.data_ptr(), ldv, t, slots.data_ptr(), alpha_k, alpha_v,
                                 cache._ref, s))
    finally:
        if entered is not None:
            entered.close()


def fq_kv_store(Kq, Ks, Vq, Vs, slots, cache: KVCache, stream=None):
    """Codes and scales that fq_quant_kv returned (uint8 [T, H * 64], fp16 [T, H]) into the cache's slots."""
    h = cache.heads
    t = slots.shape[0]
    for x, dt, w, name in ((Kq, torch.uint8, h * 64, "Kq"), (Ks, torch.float16, h, "Ks"),
                           (Vq, torch.uint8, h * 64, "Vq"), (Vs, torch.float16, h, "Vs")):
        _check(x, dt, name)
        _check_shape(x, (t, w), name)
    _check_slots(slots, t)
    s, entered = _enter(stream, Kq, Ks, Vq, Vs, slots, cache.pool)
    try:
        _raise(lib().fq_kv_store(Kq.data_ptr(), Ks.data_ptr(), Vq.data_ptr(), Vs.data_ptr(), t, slots.data_ptr(),
                                 cache._ref, s))
    finally:
        if entered is not None:
            entered.close()


def fq_kv_read(cache: KVCache, slots, K=None, V=None, stream=None):
    """The cached tokens of `slots` (int32 [T]) as fp16 (K, V), each [T, H, 128]; zeros where a slot is no place."""
    t = slots.numel()
    _check_slots(slots, t)
    shape = (t, cache.heads, 128)
    s, entered = _enter(stream, slots, cache.pool, K, V)
    try:
        if K is None:
            K = slots.new_empty(t, cache.heads, 128, dtype=torch.float16)
        else:
            _check(K, torch.float16, "K")
            _check_shape(K, shape, "K")
        if V is None:
            V = torch.empty_like(K)
        else:
            _check(V, torch.float16, "V")
            _check_shape(V, shape, "V")
        _raise(lib().fq_kv_read(cache._ref, slots.data_ptr(), t, K.data_ptr(), V.data_ptr(), s))
    finally:
        if entered is not None:
            entered.close()
    return K, V


def fq_kv_attn_workspace_size(R: int, Hq: int, H: int) -> int:
    return _size(lib().fq_kv_attn_workspace_size, R, Hq, H)


def fq_kv_attn_workspace(R: int, Hq: int, H: int, device="cuda"):
    """A zeroed workspace for fq_kv_attn.  Calls that may overlap on the GPU need one each."""
    with torch.cuda.device(device):
        return torch.zeros(fq_kv_attn_workspace_size(R, Hq, H), dtype=torch.uint8, device=device)


def fq_kv_attn(Q, lens, block_table, cache: KVCache, scale: float | None = None, window: int = 0, Y=None,
               workspace=None, stream=None):
    """Attention of one new token per request over the paged cache: Q fp16 [R, Hq, 128] or
    [R, Hq * 128] (rows any distance apart), lens int32 [R], block_table int32 [R, max_pages];
    scale defaults to 128^-0.5, window > 0 keeps the last `window` tokens.  Returns Y fp16 [R, Hq * 128]."""
    _check(lens, torch.int32, "lens")
    _check(block_table, torch.int32, "block_table")
    r = lens.numel()
    table_shape, q_shape = block_table.shape, Q.shape
    if lens.dim() != 1 or len(table_shape) != 2 or table_shape[0] != r:
        raise ValueError(f"lens must be [R] and block_table [R, max_pages], got {tuple(lens.shape)} and "
                         f"{tuple(table_shape)}")
    width = q_shape[-1] * (q_shape[1] if len(q_shape) == 3 else 1) if len(q_shape) > 1 else 0
    rows, ldq = _check_rows(Q, "Q", width)
    if rows != r or width < 128 or width % 128:
        raise ValueError(f"Q must have {r} rows of Hq * 128 values, got shape {tuple(q_shape)}")
    if not (0 <= window <= _INT_MAX and table_shape[1] <= _INT_MAX):
        _check_int(window, _INT_MAX, "window")
        _check_int(table_shape[1], _INT_MAX, "max_pages")
    hq = width // 128
    s, entered = _enter(stream, Q, lens, block_table, cache.pool, Y, workspace)
    try:
        if Y is None:
            Y = Q.new_empty(r, width)  # sizes one by one: a tuple costs 0.4 us more
        else:
            _check(Y, torch.float16, "Y")
            if Y.numel() != r * width:
                raise ValueError(f"Y must hold {r} x {width} values, got shape {tuple(Y.shape)}")
        if workspace is None:
            workspace = fq_kv_attn_workspace(r, hq, cache.heads, Q.device)
        else:
            _check(workspace, torch.uint8, "workspace")
        _raise(lib().fq_kv_attn(Q.data_ptr(), ldq, r, hq, lens.data_ptr(), block_table.data_ptr(), table_shape[1],
                                cache._ref, _HEAD_SCALE if scale is None else scale, window, Y.data_ptr(),
                                workspace.data_ptr(), workspace.numel(), s))
    finally:
        if entered is not None:
            entered.close()
    return Y


def fq_mx_scale_bytes(rows: int, k: int, fmt: int) -> int:
    """Bytes of the tiled scales of a [rows, K] tensor, padding included."""
    return _size(lib().fq_mx_scale_bytes, rows, k, fmt)


_MX_NAMES = {"X": ("Xq", "Sx"), "W": ("Wq", "Sw")}


def _check_mx(Q, S, fmt, name):
    """(rows, K) of microscaled codes Q [rows, K/2] with their tiled scales S."""
    _check_fmt(fmt)
    codes, scales = _MX_NAMES[name]
    _check(Q, torch.uint8, codes)
    _check(S, torch.uint8, scales)
    shape = Q.shape
    if len(shape) != 2:
        raise ValueError(f"{codes} must be [rows, K/2]")
    rows, k = shape[0], 2 * shape[1]
    need = (rows + 127) // 128 * 128 * (k // (16 if fmt == NVFP4 else 32))
    if S.numel() != need:
        raise ValueError(f"{scales} must hold {need} bytes, got {S.numel()}")
    return rows, k


def _check_x(X, name):
    if not isinstance(X, torch.Tensor) or len(X.shape) != 2:
        raise ValueError(f"{name} must be a CUDA tensor [rows, K]")
    k = X.shape[1]
    r, ldx = _check_rows(X, name, k)
    return r, k, ldx


def fq_mx_quant(X, fmt: int, g=None, Q=None, S=None, stream=None):
    """fp16 [R, K] (rows any distance apart) to microscaled 4-bit codes: (Q uint8 [R, K/2], S uint8, the
    tiled scales).  fmt MXFP4 or NVFP4 (g: its float32 [1] tensor scale on the device, None: 1)."""
    _check_fmt(fmt)
    r, k, ldx = _check_x(X, "X")
    _check_g(g, "g")
    s, entered = _enter(stream, X, g, Q, S)
    try:
        if Q is None:
            Q = X.new_empty(r, k // 2, dtype=torch.uint8)
        if S is None:
            S = X.new_empty(fq_mx_scale_bytes(r, k, fmt), dtype=torch.uint8)
        elif k % 128 == 0:
            _check_mx(Q, S, fmt, "X")
        _check(Q, torch.uint8, "Q")
        _check_shape(Q, (r, k // 2), "Q")
        _raise(lib().fq_mx_quant(X.data_ptr(), ldx, r, k, fmt, _p(g), Q.data_ptr(), S.data_ptr() or None, s))
    finally:
        if entered is not None:
            entered.close()
    return Q, S


def fq_mx_dequant(Q, S, fmt: int, g=None, X=None, stream=None):
    """Microscaled codes back to fp16 [R, K]."""
    r, k = _check_mx(Q, S, fmt, "X")
    _check_g(g, "g")
    s, entered = _enter(stream, Q, S, g, X)
    try:
        if X is None:
            X = Q.new_empty(r, k, dtype=torch.float16)
        else:
            _check(X, torch.float16, "X")
            _check_shape(X, (r, k), "X")
        _raise(lib().fq_mx_dequant(Q.data_ptr(), S.data_ptr(), r, k, fmt, _p(g), X.data_ptr(), s))
    finally:
        if entered is not None:
            entered.close()
    return X


def fq_mx_gemm_workspace_size(m: int, n: int, k: int, fmt: int) -> int:
    return _size(lib().fq_mx_gemm_workspace_size, m, n, k, fmt)


def fq_mx_linear_workspace_size(m: int, n: int, k: int, fmt: int) -> int:
    return _size(lib().fq_mx_linear_workspace_size, m, n, k, fmt)


def fq_mx_linear_workspace(m: int, n: int, k: int, fmt: int, device="cuda"):
    """A zeroed workspace for fq_mx_linear.  Calls that may overlap on the GPU need one each."""
    with torch.cuda.device(device):
        return torch.zeros(fq_mx_linear_workspace_size(m, n, k, fmt), dtype=torch.uint8, device=device)


def _check_g(g, name):
    if g is not None:
        _check(g, torch.float32, name)
        if g.numel() != 1:
            raise ValueError(f"{name} must hold one value, got shape {tuple(g.shape)}")


def _mx_out(like, Y, m, n):
    if Y is None:
        return like.new_empty(m, n, dtype=torch.float16)
    _check(Y, torch.float16, "Y")
    _check_shape(Y, (m, n), "Y")
    return Y


def fq_mx_gemm(Xq, Sx, Wq, Sw, fmt: int, g_x=None, g_w=None, Y=None, workspace=None, stream=None):
    """Y fp16 [M, N] = the block-scaled product of microscaled activations and weights
    (codes and scales as fq_mx_quant returns them), times g_x g_w."""
    m, k = _check_mx(Xq, Sx, fmt, "X")
    n, kw = _check_mx(Wq, Sw, fmt, "W")
    if kw != k:
        raise ValueError(f"Xq has K = {k}, Wq {kw}")
    _check_g(g_x, "g_x")
    _check_g(g_w, "g_w")
    if workspace is not None:
        _check(workspace, torch.uint8, "workspace")
    s, entered = _enter(stream, Xq, Sx, Wq, Sw, g_x, g_w, Y, workspace)
    try:
        Y = _mx_out(Xq, Y, m, n)
        ws, wsb = _workspace(fq_mx_gemm_workspace_size(m, n, k, fmt), Xq.device, workspace)
        _raise(lib().fq_mx_gemm(Xq.data_ptr(), Sx.data_ptr(), _p(g_x), Wq.data_ptr(), Sw.data_ptr(), _p(g_w), m, n, k,
                                fmt, Y.data_ptr(), _p(ws), wsb, s))
    finally:
        if entered is not None:
            entered.close()
    return Y


def fq_mx_linear(X, fmt: int, Wq, Sw, g_x=None, g_w=None, Y=None, workspace=None, stream=None):
    """Y fp16 [M, N]: X fp16 [M, K] (rows any distance apart) quantized to microscaled 4-bit,
    times the microscaled weights Wq [N, K/2], Sw, on one stream."""
    m, k, ldx = _check_x(X, "X")
    n, kw = _check_mx(Wq, Sw, fmt, "W")
    if kw != k:
        raise ValueError(f"X has K = {k}, Wq {kw}")
    _check_g(g_x, "g_x")
    _check_g(g_w, "g_w")
    s, entered = _enter(stream, X, Wq, Sw, g_x, g_w, Y, workspace)
    try:
        Y = _mx_out(X, Y, m, n)
        if workspace is None:
            workspace = fq_mx_linear_workspace(m, n, k, fmt, X.device)
        else:
            _check(workspace, torch.uint8, "workspace")
        _raise(lib().fq_mx_linear(X.data_ptr(), ldx, m, k, fmt, _p(g_x), Wq.data_ptr(), Sw.data_ptr(), _p(g_w), n,
                                  Y.data_ptr(), workspace.data_ptr(), workspace.numel(), s))
    finally:
        if entered is not None:
            entered.close()
    return Y


def fq_ternary_pack(T, Tq=None, stream=None):
    """int8 T [N, K] in {-1, 0, 1} -> packed 2-bit codes uint8 [N, K/4]."""
    _check(T, torch.int8, "T")
    n, k = T.shape
    Tq = torch.empty(n, k // 4, dtype=torch.uint8, device=T.device) if Tq is None else Tq
    _raise(lib().fq_ternary_pack(T.data_ptr(), n, k, Tq.data_ptr(), _s(stream)))
    return Tq


def fq_ternary_linear(X, Tq, alpha, mu, Y=None, stream=None):
    """Y fp16 [M, N] = X (alpha T + mu)^T for packed ternary codes Tq [N, K/4]
    and per-(row, 128-block) alpha, mu float32 [N, K/128]."""
    _check(X, torch.float16, "X")
    _check(Tq, torch.uint8, "Tq")
    _check(alpha, torch.float32, "alpha")
    _check(mu, torch.float32, "mu")
    m, k = X.shape
    n = Tq.shape[0]
    Y = torch.empty(m, n, dtype=torch.float16, device=X.device) if Y is None else Y
    _check(Y, torch.float16, "Y")
    _raise(lib().fq_ternary_linear(X.data_ptr(), m, k, Tq.data_ptr(), alpha.data_ptr(), mu.data_ptr(), n,
                                   Y.data_ptr(), _s(stream)))
    return Y


def fq_check_device_error(stream=None):
    _raise(lib().fq_check_device_error(_s(stream)))


def fq_debug_wait_timeout(limit_us: int, stream=None):
    _raise(lib().fq_debug_wait_timeout(limit_us, _s(stream)))
