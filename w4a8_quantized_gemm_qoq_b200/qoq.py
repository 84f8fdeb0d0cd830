"""ctypes binding of libqoq.so (the C ABI in include/qoq.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. PyTorch supplies device memory and the current stream. There is no
CPU fallback: if the library is missing or no CUDA device is present the calls
raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqoq.so")

QOQ_OK = 0
QOQ_ERR_TIMEOUT = 7
STATUS = {0: "QOQ_OK", 1: "QOQ_ERR_INVALID_ARG", 2: "QOQ_ERR_UNSUPPORTED", 3: "QOQ_ERR_ALIGNMENT",
          4: "QOQ_ERR_WORKSPACE", 5: "QOQ_ERR_BAD_BLOB", 6: "QOQ_ERR_CUDA", 7: "QOQ_ERR_TIMEOUT"}
TILE = 128
GROUP = 128
WORKSPACE_CONTROL_BYTES = 1280   # status word + per-tile arrival counters (include/qoq.h)

_lib = None


class QoQError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__("%s failed: %s (%d)" % (fn, STATUS.get(code, "?"), code))
        self.code = code


def lib() -> ctypes.CDLL:
    """Open libqoq.so (built in-tree by w4a8_quantized_gemm_qoq_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libqoq.so is not built (%s); run python -m w4a8_quantized_gemm_qoq_b200.build"
                              % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)
        L.qoq_quantize_act_per_token.argtypes = [vp, i64, i64, vp, vp, vp, vp]
        L.qoq_quantize_weights.argtypes = [vp, i64, i64, i32, vp, sz, vp]
        L.qoq_rmsnorm_quant.argtypes = [vp, vp, i64, i64, ctypes.c_float, vp, vp, vp, vp]
        L.qoq_silu_mul_quant.argtypes = [vp, i64, i64, vp, vp, vp, vp]
        L.qoq_w4a8_gemm.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp, vp, sz, vp]
        L.qoq_gemm_fp16_out.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, vp, vp, sz, vp]
        L.qoq_gemm_fp16_out_saturating.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp, vp, sz, vp]
        L.qoq_gemm_fp16_out_saturating.restype = ctypes.c_int
        L.qoq_w4a8_linear.argtypes = [vp, vp, i64, i64, i64, i32, vp, vp, sz, vp]
        L.qoq_w4a8_linear.restype = ctypes.c_int
        L.qoq_kv4_cache_write.argtypes = [vp, i64, i64, i64, i64, i64, i64, vp, vp, vp, vp]
        L.qoq_kv4_cache_write.restype = ctypes.c_int
        L.qoq_kv4_decode_attention.argtypes = [vp] * 8 + [i64] * 5 + [vp, vp, sz, vp]
        L.qoq_kv4_decode_attention.restype = ctypes.c_int
        L.qoq_kv4_pages_assign.argtypes = [vp, vp, i64, i64, vp, vp, i64, vp, i64, i64] + [vp] * 7
        L.qoq_kv4_pages_release.argtypes = [vp, i64, i64, vp, vp, i64, vp, vp, i64, vp, vp]
        L.qoq_kv4_paged_write.argtypes = [vp, i64, vp, i64, vp] + [i64] * 5 + [vp] * 5
        L.qoq_kv4_paged_read.argtypes = [vp] + [i64] * 5 + [vp] * 7
        L.qoq_kv4_paged_attention.argtypes = [vp, i64, vp, vp, vp, vp, vp, i64, vp, vp] + [i64] * 10 + \
            [vp, i64, vp, sz, vp]
        for f in (L.qoq_kv4_pages_assign, L.qoq_kv4_pages_release, L.qoq_kv4_paged_write, L.qoq_kv4_paged_read,
                  L.qoq_kv4_paged_attention):
            f.restype = ctypes.c_int
        L.qoq_plan.argtypes = [i64, i64, i64, vp, vp]
        L.qoq_plan.restype = ctypes.c_int
        L.qoq_watchdog_selftest.argtypes = [vp, i64, vp]
        L.qoq_watchdog_selftest.restype = ctypes.c_int
        L.qoq_status_string.argtypes = [ctypes.c_int]
        L.qoq_status_string.restype = ctypes.c_char_p
        for f in (L.qoq_quantize_act_per_token, L.qoq_quantize_weights, L.qoq_w4a8_gemm, L.qoq_gemm_fp16_out):
            f.restype = ctypes.c_int
        _lib = L
    return _lib


def _check(fn, code):
    if code != QOQ_OK:
        raise QoQError(fn, code)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _cuda_tensor(t, dtype, name):
    import torch
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


# ------------------------------------------------------------------ sizes

def blob_bytes(N: int, K: int, group_size: int = GROUP) -> int:
    n = ctypes.c_size_t(0)
    _check("qoq_quantize_weights", lib().qoq_quantize_weights(None, N, K, group_size, None, ctypes.byref(n), None))
    return n.value


def workspace_bytes(M: int, N: int, K: int, group_size: int = GROUP) -> int:
    n = ctypes.c_size_t(0)
    _check("qoq_gemm_fp16_out", lib().qoq_gemm_fp16_out(None, None, None, None, M, N, K, group_size, None, None,
                                                        ctypes.byref(n), None))
    return n.value


def linear_workspace_bytes(M: int, N: int, K: int, group_size: int = GROUP) -> int:
    n = ctypes.c_size_t(0)
    _check("qoq_w4a8_linear", lib().qoq_w4a8_linear(None, None, M, N, K, group_size, None, None, ctypes.byref(n),
                                                    None))
    return n.value


def plan(M: int, N: int, K: int):
    """(token tile, kernels qoq_w4a8_linear launches) for an M x N x K problem."""
    tok, nl = ctypes.c_int32(0), ctypes.c_int32(0)
    _check("qoq_plan", lib().qoq_plan(M, N, K, ctypes.byref(tok), ctypes.byref(nl)))
    return tok.value, nl.value


# ------------------------------------------------------------------ calls

def quantize_act_per_token(X, X8=None, s_x=None, rowsum=None, stream=None):
    """X [M][K] fp16 -> (X8 int8 [M][K], s_x fp16 [M], rowsum int32 [M])."""
    import torch
    X = _cuda_tensor(X, torch.float16, "X")
    M, K = X.shape
    X8 = torch.empty((M, K), dtype=torch.int8, device=X.device) if X8 is None else X8
    s_x = torch.empty((M,), dtype=torch.float16, device=X.device) if s_x is None else s_x
    rowsum = torch.empty((M,), dtype=torch.int32, device=X.device) if rowsum is None else rowsum
    _check("qoq_quantize_act_per_token",
           lib().qoq_quantize_act_per_token(_ptr(X), M, K, _ptr(X8), _ptr(s_x), _ptr(rowsum), _stream(stream)))
    return X8, s_x, rowsum


def rmsnorm_quant(X, gamma, eps: float, X8=None, s_x=None, rowsum=None, stream=None):
    """Fused RMSNorm + per-token INT8 quantisation: X [M][K] fp16, gamma [K]
    fp16 -> (X8 int8 [M][K], s_x fp16 [M], rowsum int32 [M])."""
    import torch
    X = _cuda_tensor(X, torch.float16, "X")
    gamma = _cuda_tensor(gamma, torch.float16, "gamma")
    M, K = X.shape
    if tuple(gamma.shape) != (K,):
        raise ValueError("gamma must have shape (%d,)" % K)
    X8 = torch.empty((M, K), dtype=torch.int8, device=X.device) if X8 is None else X8
    s_x = torch.empty((M,), dtype=torch.float16, device=X.device) if s_x is None else s_x
    rowsum = torch.empty((M,), dtype=torch.int32, device=X.device) if rowsum is None else rowsum
    _check("qoq_rmsnorm_quant", lib().qoq_rmsnorm_quant(_ptr(X), _ptr(gamma), M, K, float(eps), _ptr(X8),
                                                        _ptr(s_x), _ptr(rowsum), _stream(stream)))
    return X8, s_x, rowsum


def silu_mul_quant(GU, X8=None, s_x=None, rowsum=None, stream=None):
    """Fused SiLU(gate) * up + per-token INT8 quantisation: GU [M][2I] fp16
    (gate | up) -> (X8 int8 [M][I], s_x fp16 [M], rowsum int32 [M])."""
    import torch
    GU = _cuda_tensor(GU, torch.float16, "GU")
    M, I2 = GU.shape
    if I2 % 2:
        raise ValueError("GU must have an even number of columns (gate | up)")
    I = I2 // 2
    X8 = torch.empty((M, I), dtype=torch.int8, device=GU.device) if X8 is None else X8
    s_x = torch.empty((M,), dtype=torch.float16, device=GU.device) if s_x is None else s_x
    rowsum = torch.empty((M,), dtype=torch.int32, device=GU.device) if rowsum is None else rowsum
    _check("qoq_silu_mul_quant", lib().qoq_silu_mul_quant(_ptr(GU), M, I, _ptr(X8), _ptr(s_x), _ptr(rowsum),
                                                          _stream(stream)))
    return X8, s_x, rowsum


def quantize_weights(W, group_size: int = GROUP, blob=None, stream=None):
    """W [N][K] fp16 -> packed blob (uint8 tensor) in compute order."""
    import torch
    W = _cuda_tensor(W, torch.float16, "W")
    N, K = W.shape
    need = blob_bytes(N, K, group_size)
    blob = torch.empty((need,), dtype=torch.uint8, device=W.device) if blob is None else blob
    n = ctypes.c_size_t(blob.numel())
    _check("qoq_quantize_weights",
           lib().qoq_quantize_weights(_ptr(W), N, K, group_size, _ptr(blob), ctypes.byref(n), _stream(stream)))
    return blob


class Workspace:
    """Zero-filled device workspace for the GEMM calls. Its leading control
    bytes (the device status word, then per-tile arrival counters) are left zero by
    every call that completes; the rest is scratch."""

    def __init__(self, nbytes: int, device="cuda"):
        import torch
        self.buf = torch.zeros((nbytes + 15) // 16 * 16, dtype=torch.uint8, device=device)

    @classmethod
    def for_shape(cls, M, N, K, group_size=GROUP, device="cuda"):
        return cls(workspace_bytes(M, N, K, group_size), device)

    @classmethod
    def for_linear(cls, M, N, K, group_size=GROUP, device="cuda"):
        """Workspace of qoq_w4a8_linear (GEMM scratch plus the quantised activations)."""
        return cls(linear_workspace_bytes(M, N, K, group_size), device)

    def status(self) -> int:
        return int(self.buf[:4].view(dtype=__import__("torch").int32).item())

    def timeout_site(self):
        """(wait site, block index, detail) recorded with QOQ_ERR_TIMEOUT."""
        import torch
        w = self.buf[:16].view(dtype=torch.int32).tolist()
        return tuple(w[1:4])

    def control_clear(self) -> bool:
        return not bool(self.buf[:WORKSPACE_CONTROL_BYTES].any().item())

    def reset(self):
        self.buf.zero_()


def watchdog_selftest(limit_ns=50_000_000, stream=None):
    """Run the device bounded-wait self-test; returns the 32 status words
    (the mbarrier wait's record at [0:4], the flag wait's at [8:12])."""
    import torch
    status = torch.zeros(32, dtype=torch.int32, device="cuda")
    _check("qoq_watchdog_selftest", lib().qoq_watchdog_selftest(_ptr(status), int(limit_ns), _stream(stream)))
    torch.cuda.synchronize()
    return status.cpu().tolist()


def w4a8_gemm(X8, blob, N, K, group_size=GROUP, rowsum=None, ws=None, acc=None, stream=None):
    """Exact INT32 GEMM: acc [M][N]."""
    import torch
    X8 = _cuda_tensor(X8, torch.int8, "X8")
    M = X8.shape[0]
    ws = ws or Workspace.for_shape(M, N, K, group_size, X8.device)
    acc = torch.empty((M, N), dtype=torch.int32, device=X8.device) if acc is None else acc
    n = ctypes.c_size_t(ws.buf.numel())
    _check("qoq_w4a8_gemm", lib().qoq_w4a8_gemm(_ptr(X8), _ptr(rowsum), _ptr(blob), M, N, K, group_size, _ptr(acc),
                                                _ptr(ws.buf), ctypes.byref(n), _stream(stream)))
    return acc


def gemm_fp16_out(X8, s_x, blob, N, K, group_size=GROUP, rowsum=None, ws=None, Y=None, stream=None):
    """W4A8 GEMM with fused FP16 epilogue: Y [M][N] fp16."""
    import torch
    X8 = _cuda_tensor(X8, torch.int8, "X8")
    M = X8.shape[0]
    ws = ws or Workspace.for_shape(M, N, K, group_size, X8.device)
    Y = torch.empty((M, N), dtype=torch.float16, device=X8.device) if Y is None else Y
    n = ctypes.c_size_t(ws.buf.numel())
    _check("qoq_gemm_fp16_out", lib().qoq_gemm_fp16_out(_ptr(X8), _ptr(s_x), _ptr(rowsum), _ptr(blob), M, N, K,
                                                        group_size, _ptr(Y), _ptr(ws.buf), ctypes.byref(n),
                                                        _stream(stream)))
    return Y


def gemm_fp16_out_saturating(X8, s_x, blob, N, K, ws=None, Y=None, stream=None):
    """The same GEMM with a saturating weight decode (the protective-range
    ablation; group_size 128; M <= 16, or M > 512 with N / 128 even)."""
    import torch
    X8 = _cuda_tensor(X8, torch.int8, "X8")
    M = X8.shape[0]
    ws = ws or Workspace.for_shape(M, N, K, GROUP, X8.device)
    Y = torch.empty((M, N), dtype=torch.float16, device=X8.device) if Y is None else Y
    n = ctypes.c_size_t(ws.buf.numel())
    _check("qoq_gemm_fp16_out_saturating",
           lib().qoq_gemm_fp16_out_saturating(_ptr(X8), _ptr(s_x), _ptr(blob), M, N, K, GROUP, _ptr(Y),
                                              _ptr(ws.buf), ctypes.byref(n), _stream(stream)))
    return Y


def linear(X, blob, N, K, group_size=GROUP, ws=None, Y=None, stream=None):
    """The whole hot path in one call (qoq_w4a8_linear): per-token
    quantisation of X [M][K] fp16, then the W4A8 GEMM with the FP16 epilogue;
    two launches, or one for token tiles of at most 64 tokens when
    QOQ_FORCE_CONFIG holds fuse=1 (plan() reports which). Y [M][N] fp16."""
    import torch
    X = _cuda_tensor(X, torch.float16, "X")
    M = X.shape[0]
    if X.shape[1] != K:
        raise ValueError("X must have K = %d columns" % K)
    ws = ws or Workspace.for_linear(M, N, K, group_size, X.device)
    Y = torch.empty((M, N), dtype=torch.float16, device=X.device) if Y is None else Y
    n = ctypes.c_size_t(ws.buf.numel())
    _check("qoq_w4a8_linear", lib().qoq_w4a8_linear(_ptr(X), _ptr(blob), M, N, K, group_size, _ptr(Y), _ptr(ws.buf),
                                                    ctypes.byref(n), _stream(stream)))
    return Y


# ------------------------------------------------------------------ KV4

class KV4Cache:
    """A per-head, dynamic, asymmetric 4-bit cache of one tensor (K or V):
    codes uint8 [B][Hkv][max_tokens][D/2], scales and zeros FP16
    [B][Hkv][max_tokens] (include/qoq.h, qoq_kv4_cache_write)."""

    def __init__(self, B, Hkv, max_tokens, D, device="cuda"):
        import torch
        self.B, self.Hkv, self.T, self.D = B, Hkv, max_tokens, D
        self.codes = torch.zeros((B, Hkv, max_tokens, D // 2), dtype=torch.uint8, device=device)
        self.scales = torch.zeros((B, Hkv, max_tokens), dtype=torch.float16, device=device)
        self.zeros = torch.zeros((B, Hkv, max_tokens), dtype=torch.float16, device=device)

    def write(self, src, t0=0, stream=None):
        """Quantise src [B][Hkv][n][D] FP16 into slots t0 .. t0 + n - 1."""
        import torch
        src = _cuda_tensor(src, torch.float16, "src")
        B, H, n, D = src.shape
        if (B, H, D) != (self.B, self.Hkv, self.D):
            raise ValueError("src shape %s does not match the cache" % (tuple(src.shape),))
        _check("qoq_kv4_cache_write", lib().qoq_kv4_cache_write(_ptr(src), B, H, self.T, t0, n, D, _ptr(self.codes),
                                                                _ptr(self.scales), _ptr(self.zeros),
                                                                _stream(stream)))
        return self


def kv4_workspace_bytes(B, Hq, Hkv, max_tokens, D) -> int:
    n = ctypes.c_size_t(0)
    _check("qoq_kv4_decode_attention", lib().qoq_kv4_decode_attention(*([None] * 8), B, Hq, Hkv, max_tokens, D, None,
                                                                      None, ctypes.byref(n), None))
    return n.value


def kv4_decode_attention(q, kcache, vcache, seq_lens=None, ws=None, out=None, stream=None):
    """q [B][Hq][D] FP16 against the KV4 caches -> out [B][Hq][D] FP16."""
    import torch
    q = _cuda_tensor(q, torch.float16, "q")
    B, Hq, D = q.shape
    if seq_lens is not None:
        seq_lens = _cuda_tensor(seq_lens, torch.int32, "seq_lens")
    ws = ws or Workspace(kv4_workspace_bytes(B, Hq, kcache.Hkv, kcache.T, D), q.device)
    out = torch.empty((B, Hq, D), dtype=torch.float16, device=q.device) if out is None else out
    n = ctypes.c_size_t(ws.buf.numel())
    _check("qoq_kv4_decode_attention", lib().qoq_kv4_decode_attention(
        _ptr(q), _ptr(kcache.codes), _ptr(kcache.scales), _ptr(kcache.zeros), _ptr(vcache.codes),
        _ptr(vcache.scales), _ptr(vcache.zeros), _ptr(seq_lens), B, Hq, kcache.Hkv, kcache.T, D, _ptr(out),
        _ptr(ws.buf), ctypes.byref(n), _stream(stream)))
    return out


# ------------------------------------------------------------------ paged KV4
#
# A serving step makes these calls for every layer, so their checks are kept
# short: one test of what a correct argument has, and the reason only where it
# fails; pointers of the buffers that an object owns are kept with it, and what
# is needed of torch in names of this module from the first object on.

_vp, _i64 = ctypes.c_void_p, ctypes.c_int64
_Tensor = _int32 = _float16 = _empty_like = _get_device = _current_stream = None


def _bind_torch():
    global _Tensor, _int32, _float16, _empty_like, _get_device, _current_stream
    if _Tensor is None:
        import torch
        _int32, _float16, _empty_like = torch.int32, torch.float16, torch.empty_like
        _get_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        _Tensor = torch.Tensor


def _device_scope(device):
    """Launches go to the tensors' device: entered only when it is not current."""
    import torch
    return torch.cuda.device(device)


def _raw_stream(stream, index):
    """The stream to launch on: the given one, or the device's current one."""
    return _vp(_current_stream(index) if stream is None else stream.cuda_stream)


def _stream_scope(stream):
    """Allocations belong to the stream that uses them."""
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _empty_fp16(like, shape, stream):
    """An FP16 tensor beside `like`, which is one too."""
    if stream is None:
        return like.new_empty(shape)
    with _stream_scope(stream):
        return like.new_empty(shape)


def _i32(t, shape, device, name):
    """Pointer of an int32 CUDA tensor of this shape on this device."""
    if not (isinstance(t, _Tensor) and t.dtype is _int32 and t.shape == shape and t.device == device and
            t.is_contiguous()):
        _cuda_tensor(t, _int32, name)
        if t.shape != shape:
            raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    return _vp(t.data_ptr())


def _rows(t, heads, D, device, name):
    """Pointer, row stride (in elements) and rows of FP16 [N][heads][D] with
    dense heads and any row stride; heads None: any number of them."""
    if isinstance(t, _Tensor) and t.dtype is _float16 and t.device == device and t.dim() == 3:
        n, h, d = t.shape
        if d == D and (heads is None or h == heads):
            s0, s1, s2 = t.stride()
            if s2 == 1 and (s1 == D or h == 1) or n == 0:
                return _vp(t.data_ptr()), s0 if n > 1 else h * D, n
            raise ValueError("the heads of a row of %s must be dense" % name)
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype is not _float16:
        raise TypeError("%s must be %s, got %s" % (name, _float16, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    raise ValueError("%s must have shape [N][%s][%d], got %s" % (name, "heads" if heads is None else heads, D,
                                                                  tuple(t.shape)))


class PagedStep:
    """What one step of up to max_tokens rows needs of the page tables
    (include/qoq.h, qoq_kv4_pages_assign): q_start [B + 1], and positions and
    slots [max_tokens], -1 past the step's rows. The buffers stay the same
    ones, so that a captured step can refer to them."""

    def __init__(self, B, max_tokens, device="cuda"):
        import torch
        _bind_torch()
        self._q_start = torch.zeros((B + 1,), dtype=torch.int32, device=device)
        self._positions = torch.full((max_tokens,), -1, dtype=torch.int32, device=device)
        self._slots = torch.full((max_tokens,), -1, dtype=torch.int32, device=device)
        self._ptrs = tuple(_vp(t.data_ptr()) for t in (self._q_start, self._positions, self._slots))
        self.B, self.max_tokens, self.device = B, max_tokens, self._q_start.device

    q_start = property(lambda self: self._q_start)
    positions = property(lambda self: self._positions)
    slots = property(lambda self: self._slots)


class PageTable:
    """Pages of B requests, kept on the GPU: cached lengths, block table, and
    the stack of free pages (include/qoq.h, "Paged KV4 cache"). One table
    serves the caches of every layer."""

    def __init__(self, B, max_pages, n_pages, page_size=64, device="cuda"):
        import torch
        i32 = dict(dtype=torch.int32, device=device)
        self._set(torch.zeros((B,), **i32), torch.full((B, max_pages), -1, **i32), torch.arange(n_pages, **i32),
                  torch.full((1,), n_pages, **i32), page_size)

    @classmethod
    def of(cls, seq_lens, block_table, free_pages, free_count, page_size):
        """A table over buffers the caller already holds (not copied)."""
        self = cls.__new__(cls)
        self._set(seq_lens, block_table, free_pages, free_count, page_size)
        return self

    def _set(self, seq_lens, block_table, free_pages, free_count, page_size):
        import torch
        _bind_torch()
        _cuda_tensor(seq_lens, torch.int32, "seq_lens")
        if seq_lens.dim() != 1 or block_table.dim() != 2 or free_pages.dim() != 1:
            raise ValueError("seq_lens [B], block_table [B][max_pages] and free_pages [n_pages] are expected")
        B, device = seq_lens.shape[0], seq_lens.device
        self.B, self.device, self.page_size = B, device, int(page_size)
        self._seq_lens, self._block_table, self._free_pages, self._free_count = \
            seq_lens, block_table, free_pages, free_count
        self.status_words = torch.zeros((4,), dtype=torch.int32, device=device)
        self._seq = _i32(seq_lens, (B,), device, "seq_lens")
        self._table = _i32(block_table, (B, block_table.shape[1]), device, "block_table")
        self._free = _i32(free_pages, free_pages.shape, device, "free_pages")
        self._count = _i32(free_count, (1,), device, "free_count")
        self._status = _vp(self.status_words.data_ptr())
        self._sizes = _i64(B), _i64(self.page_size), _i64(free_pages.shape[0]), _i64(block_table.shape[1])

    seq_lens = property(lambda self: self._seq_lens)
    block_table = property(lambda self: self._block_table)
    free_pages = property(lambda self: self._free_pages)
    free_count = property(lambda self: self._free_count)

    def assign(self, new_lens, step, kv_lens=None, free_left=None, stream=None):
        """Begin a step in which new_lens[b] tokens join request b: fills
        `step` and enters the pages taken. The lengths and the free count
        are updated in place, unless kv_lens [B] and free_left [1] are given
        to take the new ones. Returns `step`."""
        device = self.device
        if _get_device() != device.index:
            with _device_scope(device):
                return self.assign(new_lens, step, kv_lens, free_left, stream)
        B, page_size, n_pages, max_pages = self._sizes
        if step.B != self.B or step.device != device:
            raise ValueError("the step is for %d requests on %s, the table for %d on %s"
                             % (step.B, step.device, self.B, device))
        q_start, positions, slots = step._ptrs
        code = lib().qoq_kv4_pages_assign(
            self._seq, _i32(new_lens, (self.B,), device, "new_lens"), B, page_size, self._free, self._count, n_pages,
            self._table, max_pages, step.max_tokens,
            self._seq if kv_lens is None else _i32(kv_lens, (self.B,), device, "kv_lens"), q_start, positions, slots,
            self._count if free_left is None else _i32(free_left, (1,), device, "free_left"), self._status,
            _raw_stream(stream, device.index))
        if code:
            _check("qoq_kv4_pages_assign", code)
        return step

    def release(self, leave, stream=None):
        """End the requests b with leave[b] != 0 (int32 [B]): their pages are
        free again, their lengths 0."""
        device = self.device
        if _get_device() != device.index:
            with _device_scope(device):
                return self.release(leave, stream)
        B, page_size, n_pages, max_pages = self._sizes
        code = lib().qoq_kv4_pages_release(_i32(leave, (self.B,), device, "leave"), B, page_size, self._seq, self._table,
                                           max_pages, self._free, self._count, n_pages, self._status,
                                           _raw_stream(stream, device.index))
        if code:
            _check("qoq_kv4_pages_release", code)

    def status(self) -> int:
        """The first refused step's status code (synchronises), 0 if none was."""
        return int(self.status_words[0].item())


class PagedKV4Cache:
    """One layer's paged 4-bit cache of K and V (include/qoq.h, "Paged KV4
    cache"): codes uint8 [n_pages][Hkv][page_size][D/2] and params FP16
    [n_pages][Hkv][page_size][2] (scale, zero) of each."""

    def __init__(self, n_pages, Hkv, page_size, D, device="cuda"):
        import torch
        u8 = dict(dtype=torch.uint8, device=device)
        f16 = dict(dtype=torch.float16, device=device)
        self._set(torch.zeros((n_pages, Hkv, page_size, D // 2), **u8),
                  torch.zeros((n_pages, Hkv, page_size, 2), **f16),
                  torch.zeros((n_pages, Hkv, page_size, D // 2), **u8),
                  torch.zeros((n_pages, Hkv, page_size, 2), **f16))

    @classmethod
    def of(cls, k_codes, k_params, v_codes, v_params):
        """A cache over buffers the caller already holds (not copied)."""
        self = cls.__new__(cls)
        self._set(k_codes, k_params, v_codes, v_params)
        return self

    def _set(self, k_codes, k_params, v_codes, v_params):
        import torch
        _bind_torch()
        for t, name in ((k_codes, "k_codes"), (v_codes, "v_codes")):
            _cuda_tensor(t, torch.uint8, name)
        for t, name in ((k_params, "k_params"), (v_params, "v_params")):
            _cuda_tensor(t, torch.float16, name)
        if k_codes.dim() != 4:
            raise ValueError("k_codes must have shape [n_pages][Hkv][page_size][D/2]")
        n, h, P, db = k_codes.shape
        if v_codes.shape != (n, h, P, db) or k_params.shape != (n, h, P, 2) or v_params.shape != (n, h, P, 2):
            raise ValueError("the shapes of codes and params do not match")
        if len({t.device for t in (k_codes, k_params, v_codes, v_params)}) != 1:
            raise ValueError("codes and params must be on one device")
        self.n_pages, self.Hkv, self.page_size, self.D, self.device = n, h, P, 2 * db, k_codes.device
        self._tensors = k_codes, k_params, v_codes, v_params
        self._ptrs = tuple(_vp(t.data_ptr()) for t in self._tensors)
        self._sizes = _i64(h), _i64(2 * db), _i64(n), _i64(P)

    k_codes = property(lambda self: self._tensors[0])
    k_params = property(lambda self: self._tensors[1])
    v_codes = property(lambda self: self._tensors[2])
    v_params = property(lambda self: self._tensors[3])

    def write(self, k, v, slots, stream=None):
        """Quantise rows k, v [N][Hkv][D] FP16 (any row stride) into
        slots [N] int32; rows with a slot outside the cache are skipped."""
        device = self.device
        if _get_device() != device.index:
            with _device_scope(device):
                return self.write(k, v, slots, stream)
        kp, ks, N = _rows(k, self.Hkv, self.D, device, "k")
        vp, vs, n = _rows(v, self.Hkv, self.D, device, "v")
        if n != N:
            raise ValueError("k has %d rows, v %d" % (N, n))
        code = lib().qoq_kv4_paged_write(kp, ks, vp, vs, _i32(slots, (N,), device, "slots"), N, *self._sizes,
                                         *self._ptrs, _raw_stream(stream, device.index))
        if code:
            _check("qoq_kv4_paged_write", code)
        return self

    def read(self, slots, k=None, v=None, stream=None):
        """The cached K and V of slots [N] as FP16 [N][Hkv][D] each (a sequence
        moved elsewhere, or handed to a dense kernel); 0 outside the cache."""
        device = self.device
        if _get_device() != device.index:
            with _device_scope(device):
                return self.read(slots, k, v, stream)
        N = slots.shape[0]
        sp = _i32(slots, (N,), device, "slots")
        shape = (N, self.Hkv, self.D)
        for t, name in ((k, "k"), (v, "v")):
            if t is not None:
                _cuda_tensor(t, _float16, name)
                if t.shape != shape or t.device != device:
                    raise ValueError("%s must have shape %s on %s" % (name, shape, device))
        k = _empty_fp16(self._tensors[1], shape, stream) if k is None else k
        if v is None:
            v = _empty_like(k) if stream is None else _empty_fp16(k, shape, stream)
        code = lib().qoq_kv4_paged_read(sp, N, *self._sizes, *self._ptrs, _vp(k.data_ptr()), _vp(v.data_ptr()),
                                        _raw_stream(stream, device.index))
        if code:
            _check("qoq_kv4_paged_read", code)
        return k, v


def kv4_paged_workspace_bytes(B, N, Hq, Hkv, D, max_new) -> int:
    n = ctypes.c_size_t(0)
    _check("qoq_kv4_paged_attention", lib().qoq_kv4_paged_attention(
        None, 0, None, None, None, None, None, 0, None, None, B, N, max_new, Hq, Hkv, D, 0, 0, 0, 0, None, 0, None,
        ctypes.byref(n), None))
    return n.value


def kv4_paged_attention(q, cache, block_table, q_start, kv_lens, max_new, window=0, sinks=0, ws=None, out=None,
                        stream=None):
    """q [N][Hq][D] FP16 (any row stride): rows q_start[b] .. q_start[b + 1] - 1
    are request b's latest tokens, attending to the kv_lens[b] tokens that
    block_table [B][max_pages] holds of it, causally, and with window > 0 only
    to the latest `window` of them and the first `sinks`. max_new bounds the
    rows per request (1 for a decode step). Returns out [N][Hq][D] FP16."""
    device = cache.device
    if _get_device() != device.index:
        with _device_scope(device):
            return kv4_paged_attention(q, cache, block_table, q_start, kv_lens, max_new, window, sinks, ws, out, stream)
    Hkv, D, n_pages, page_size = cache._sizes
    qp, qs, N = _rows(q, None, cache.D, device, "q")
    Hq = q.shape[1]
    B, max_pages = block_table.shape
    if ws is None:
        with _stream_scope(stream):
            ws = Workspace(kv4_paged_workspace_bytes(B, N, Hq, cache.Hkv, cache.D, max_new), device)
    if out is None:
        out = _empty_fp16(q, (N, Hq, cache.D), stream)
    op, os_, n = _rows(out, Hq, cache.D, device, "out")
    if n != N or ws.buf.device != device:
        raise ValueError("out must have q's shape, and the workspace its device")
    n = ctypes.c_size_t(ws.buf.numel())
    code = lib().qoq_kv4_paged_attention(
        qp, qs, *cache._ptrs, _i32(block_table, (B, max_pages), device, "block_table"), max_pages,
        _i32(q_start, (B + 1,), device, "q_start"), _i32(kv_lens, (B,), device, "kv_lens"), B, N, max_new, Hq, Hkv, D,
        n_pages, page_size, window, sinks, op, os_, _vp(ws.buf.data_ptr()), ctypes.byref(n),
        _raw_stream(stream, device.index))
    if code:
        _check("qoq_kv4_paged_attention", code)
    return out
