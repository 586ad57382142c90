"""Python binding of libbonsai (include/bonsai.h): argument marshalling only.

Every function has the name of the C entry point it calls and forwards raw
device pointers, sizes and the CUDA stream; all computation happens in the CUDA
kernels.  Tensors are torch CUDA tensors (torch is used for device memory and
streams only); plain integers are accepted as device pointers too, except for cache pools and
page tables, whose shapes the binding reads.

Importing this module fails loudly if libbonsai.so has not been built: there is
no CPU fallback.  Build with ``python -m ternary_weight_02_b200.build``.  The entry points
that a decode step calls per layer go through a small extension module that the same build
makes, or through ctypes (1 to 2 us more of host time a call) where it cannot be loaded.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libbonsai.so")

BONSAI_FMT_PTQ1_0 = 1
BONSAI_FMT_PQ2_0 = 2
BONSAI_FMT_Q1_0 = 3
BONSAI_FMT_PQ2_0_G64 = 4  # PQ2_0 codes, one FP16 scale per 64 weights

BONSAI_OK = 0
BONSAI_ERR_NULL = -1
BONSAI_ERR_SHAPE = -2
BONSAI_ERR_FMT = -3
BONSAI_ERR_ALIGN = -4
BONSAI_ERR_CUDA = -5
BONSAI_ERR_ARCH = -6
BONSAI_ERR_NOMEM = -7
BONSAI_ERR_ALGO = -8
BONSAI_ERR_TOO_LARGE = -9
BONSAI_ERR_ARG = -10

BONSAI_DEVICE_GEMV_COPY_TIMEOUT = 1
BONSAI_DEVICE_GEMV_PIECE_TIMEOUT = 2
BONSAI_DEVICE_GEMM_TIMEOUT = 4
BONSAI_DEVICE_SKINNY_TIMEOUT = 8
BONSAI_DEVICE_CACHE_RANGE = 16
BONSAI_DEVICE_ATTENTION_TIMEOUT = 32

BONSAI_ALGO_AUTO = 0
BONSAI_ALGO_SIMPLE = 1
BONSAI_ALGO_GEMV = 2
BONSAI_ALGO_SKINNY = 3
BONSAI_ALGO_GEMM = 4
BONSAI_ALGO_IMMA = 5

BONSAI_ACT_NONE = 0
BONSAI_ACT_RELU = 1
BONSAI_ACT_SILU = 2
BONSAI_ACT_GELU = 3
BONSAI_ACT_GELU_TANH = 4

BONSAI_ROPE_HALF = 0
BONSAI_ROPE_INTERLEAVED = 1

BONSAI_ROPE_PLAIN = 0
BONSAI_ROPE_LINEAR = 1
BONSAI_ROPE_NTK = 2
BONSAI_ROPE_YARN = 3
BONSAI_ROPE_BANDS = 4

BONSAI_KV_F16 = 0
BONSAI_KV_E4M3 = 1

FORMATS = {"ptq1": BONSAI_FMT_PTQ1_0, "pq2": BONSAI_FMT_PQ2_0, "q1": BONSAI_FMT_Q1_0,
           "pq2g64": BONSAI_FMT_PQ2_0_G64}

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libbonsai.so is missing at {LIB_PATH}; build it with "
        "`python -m ternary_weight_02_b200.build` (there is no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)
_i64, _int, _p = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
_f32, _f64 = ctypes.c_float, ctypes.c_double

_SIGS = {
    "bonsai_version": (_int, []),
    "bonsai_status_string": (ctypes.c_char_p, [_int]),
    "bonsai_check_device": (_int, []),
    "bonsai_packed_bytes": (_i64, [_int, _i64, _i64]),
    "bonsai_pack_ptq1": (_int, [_p, _p, _i64, _i64, _p]),
    "bonsai_pack_pq2": (_int, [_p, _p, _i64, _i64, _p]),
    "bonsai_pack_q1": (_int, [_p, _p, _i64, _i64, _p]),
    "bonsai_unpack": (_int, [_int, _p, _p, _i64, _i64, _p]),
    "bonsai_hadamard128": (_int, [_p, _p, _i64, _i64, _p]),
    "bonsai_ternary_linear": (_int, [_p, _p, _p, _p, _i64, _i64, _i64, _int, _p]),
    "bonsai_ternary_linear_algo": (_int, [_p, _p, _p, _p, _i64, _i64, _i64, _int, _int, _int, _p]),
    "bonsai_ternary_linear_noalloc": (_int, [_p, _p, _p, _p, _i64, _i64, _i64, _int, _p]),
    "bonsai_launch_count": (_int, [_i64, _i64, _i64, _int, _int, _int]),
    "bonsai_swiglu": (_int, [_p, _p, _i64, _i64, _p]),
    "bonsai_ternary_linear_swiglu": (_int, [_p, _p, _p, _p, _i64, _i64, _i64, _int, _p]),
    "bonsai_ternary_linear_epilogue": (_int, [_p] * 6 + [_i64] * 3 + [_int] * 4 + [_p]),
    "bonsai_rope_frequencies": (_int, [_p, _p, _i64, _f64, _int] + [_f64] * 4),
    "bonsai_rope": (_int, [_p] * 4 + [_i64] * 6 + [_f32, _int, _p]),
    "bonsai_rope_append": (_int, [_p] * 9 + [_i64] * 9 + [_f32, _int, _int, _p]),
    "bonsai_paged_attention": (_int, [_p] * 9 + [_i64] * 10 + [_f32, _int, _p]),
    "bonsai_reserve": (_int, [_i64, _i64, _i64]),
    "bonsai_device_status": (_int, [_p, ctypes.POINTER(ctypes.c_uint32), _int]),
    "bonsai_debug_force_timeouts": (_int, [_int]),
    "bonsai_shutdown": (None, []),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


try:
    from . import _bonsai_call as _call  # the per-layer entry points without ctypes' conversions
except ImportError:
    _call = _lib  # the same functions of libbonsai.so


class BonsaiError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {bonsai_status_string(status)} (status {status})")


def raw():
    """The ctypes handle of libbonsai.so."""
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor arguments must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:  # the current stream's handle, without a Stream object (3 us of a call's host time)
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _stream_on(stream, dev: int):
    """_stream() where the current device's index is known."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(dev)
    return _stream(stream)


def _check(rc: int, where: str) -> int:
    if rc != BONSAI_OK:
        raise BonsaiError(rc, where)
    return rc


def bonsai_version() -> int:
    return _lib.bonsai_version()


def bonsai_status_string(status: int) -> str:
    return _lib.bonsai_status_string(status).decode()


def bonsai_check_device() -> int:
    return _lib.bonsai_check_device()


def bonsai_packed_bytes(fmt: int, N: int, K: int) -> int:
    v = _lib.bonsai_packed_bytes(fmt, N, K)
    if v < 0:
        raise BonsaiError(int(v), "bonsai_packed_bytes")
    return int(v)


def bonsai_pack_ptq1(trits, packed, N: int, K: int, stream=None) -> None:
    _check(_lib.bonsai_pack_ptq1(_ptr(trits), _ptr(packed), N, K, _stream(stream)), "bonsai_pack_ptq1")


def bonsai_pack_pq2(trits, packed, N: int, K: int, stream=None) -> None:
    _check(_lib.bonsai_pack_pq2(_ptr(trits), _ptr(packed), N, K, _stream(stream)), "bonsai_pack_pq2")


def bonsai_pack_q1(trits, packed, N: int, K: int, stream=None) -> None:
    _check(_lib.bonsai_pack_q1(_ptr(trits), _ptr(packed), N, K, _stream(stream)), "bonsai_pack_q1")


def bonsai_unpack(fmt: int, packed, trits, N: int, K: int, stream=None) -> None:
    _check(_lib.bonsai_unpack(fmt, _ptr(packed), _ptr(trits), N, K, _stream(stream)), "bonsai_unpack")


def bonsai_hadamard128(x, x_out, M: int, K: int, stream=None) -> None:
    _check(_lib.bonsai_hadamard128(_ptr(x), _ptr(x_out), M, K, _stream(stream)), "bonsai_hadamard128")


def bonsai_ternary_linear(x, packed, scales, y, M: int, N: int, K: int, fmt: int,
                          stream=None) -> None:
    _check(_call.bonsai_ternary_linear(_ptr(x), _ptr(packed), _ptr(scales), _ptr(y), M, N, K, fmt,
                                      _stream(stream)), "bonsai_ternary_linear")


def bonsai_ternary_linear_algo(x, packed, scales, y, M: int, N: int, K: int, fmt: int, algo: int,
                               split_k: int = 0, stream=None) -> None:
    _check(_lib.bonsai_ternary_linear_algo(_ptr(x), _ptr(packed), _ptr(scales), _ptr(y), M, N, K,
                                           fmt, algo, split_k, _stream(stream)),
           "bonsai_ternary_linear_algo")


def bonsai_ternary_linear_noalloc(x, packed, scales, y, M: int, N: int, K: int, fmt: int,
                                  stream=None) -> None:
    """Batch-1 layer on the library's fixed device scratch: allocates nothing."""
    _check(_lib.bonsai_ternary_linear_noalloc(_ptr(x), _ptr(packed), _ptr(scales), _ptr(y), M, N, K,
                                              fmt, _stream(stream)), "bonsai_ternary_linear_noalloc")


def bonsai_launch_count(M: int, N: int, K: int, fmt: int, algo: int = BONSAI_ALGO_AUTO,
                        split_k: int = 0) -> int:
    n = _lib.bonsai_launch_count(M, N, K, fmt, algo, split_k)
    if n < 0:
        raise BonsaiError(n, "bonsai_launch_count")
    return n


def bonsai_reserve(M: int, N: int, K: int) -> None:
    _check(_lib.bonsai_reserve(M, N, K), "bonsai_reserve")


def bonsai_device_status(stream=None, clear: bool = False) -> int:
    """The calling device's status bits (BONSAI_DEVICE_*), after synchronising `stream`."""
    bits = ctypes.c_uint32(0)
    _check(_lib.bonsai_device_status(_stream(stream), ctypes.byref(bits), 1 if clear else 0),
           "bonsai_device_status")
    return int(bits.value)


def bonsai_debug_force_timeouts(enable: bool) -> None:
    """Test hook: cross-CTA waits give up (NaN outputs, status bits) while enabled."""
    _check(_lib.bonsai_debug_force_timeouts(1 if enable else 0), "bonsai_debug_force_timeouts")


def bonsai_shutdown() -> None:
    _lib.bonsai_shutdown()


# ---------------------------------------------------------------- conveniences

def bonsai_swiglu(y, h, M: int, F: int, stream=None) -> None:
    _check(_lib.bonsai_swiglu(_ptr(y), _ptr(h), M, F, _stream(stream)), "bonsai_swiglu")


def bonsai_ternary_linear_swiglu(x, packed, scales, h, M: int, F: int, K: int, fmt: int, stream=None) -> None:
    _check(_call.bonsai_ternary_linear_swiglu(_ptr(x), _ptr(packed), _ptr(scales), _ptr(h), M, F, K, fmt,
                                             _stream(stream)), "bonsai_ternary_linear_swiglu")


# bytes of a packed 128-weight group, and its scales
_GROUP_BYTES = {BONSAI_FMT_PTQ1_0: (26, 1), BONSAI_FMT_PQ2_0: (32, 1), BONSAI_FMT_Q1_0: (16, 1),
                BONSAI_FMT_PQ2_0_G64: (32, 2)}


def _dev(t, dtype, numel: int, dev: int):
    """Device pointer of a contiguous tensor on device `dev`, with the type and at least the size
    the call reads or writes.  None and plain device pointers pass as they are."""
    if t is None or type(t) is int:
        return t
    if t.get_device() == dev and t.dtype is dtype and t.is_contiguous() and t.numel() >= numel:
        return t.data_ptr()
    if t.get_device() != dev:
        raise ValueError("tensor arguments must be CUDA tensors on the current device")
    if t.dtype is not dtype:
        raise ValueError(f"a tensor argument is {t.dtype} where {dtype} is expected")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    raise ValueError(f"a tensor argument has {t.numel()} elements where the call takes {numel}")


def _rows(t, rows: int, width: int, ld, dev: int):
    """(pointer, row stride) of a matrix of heads: `rows` rows of `width` FP16 elements, at the row
    stride given or the tensor's own (a contiguous tensor, or a matrix with contiguous rows)."""
    if t is None or type(t) is int:
        return t, width if ld is None else ld
    import torch
    if t.is_contiguous():
        if ld is None:  # a matrix's rows may be wider, or more, than the call takes
            n = t.numel()
            if t.dim() == 2 and t.shape[1] >= width:
                # (one row of a wider matrix counts as contiguous: its stride is the matrix's, unless it
                # is one that no rows can have)
                ld = t.stride(0)
                if ld < width or ld & 7:
                    ld = t.shape[1]
            elif n == rows * width or rows == 0:
                ld = width
            elif t.dim() > 1 and t.shape[0] == rows and n > rows * width:
                ld = n // rows
            else:
                raise ValueError("a tensor of heads that is no matrix holds the rows of the call, or the call is given "
                                 "their stride")
        return _dev(t, torch.float16, (rows - 1) * ld + width if rows > 0 else 0, dev), ld
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("a strided tensor of heads is a matrix with contiguous rows")
    if ld is None:
        ld = t.stride(0)
    if t.shape[0] < rows or t.shape[1] < width or t.stride(0) != ld:
        raise ValueError("a strided tensor of heads is smaller than the call takes")
    if t.get_device() != dev or t.dtype is not torch.float16:
        raise ValueError("tensor arguments must be float16 CUDA tensors on the current device")
    return t.data_ptr(), ld


def bonsai_ternary_linear_epilogue(x, packed, scales, bias, residual, y, M: int, N: int, K: int, fmt: int,
                                   act: int = BONSAI_ACT_NONE, algo: int = BONSAI_ALGO_AUTO, split_k: int = 0,
                                   stream=None) -> None:
    """y = act(x' . Wdeq^T + bias) + residual; bias and residual may be None, residual may be y."""
    import torch
    dev, f16 = torch.cuda.current_device(), torch.float16
    plane, groups = _GROUP_BYTES.get(fmt, (0, 0))
    _check(_call.bonsai_ternary_linear_epilogue(
        _dev(x, f16, M * K, dev), _dev(packed, torch.uint8, N * (K // 128) * plane, dev),
        _dev(scales, f16, N * (K // 128) * groups, dev), _dev(bias, f16, N, dev),
        _dev(residual, f16, M * N, dev), _dev(y, f16, M * N, dev), M, N, K, fmt, act, algo, split_k, _stream_on(stream, dev)),
        "bonsai_ternary_linear_epilogue")


def bonsai_rope_frequencies(R: int, base: float, scaling: int = BONSAI_ROPE_PLAIN, factor: float = 1.0,
                            original: float = 0.0, low: float = 1.0, high: float = 32.0):
    """(freqs, magnitude): R/2 frequencies in radians per position (an FP64 CPU tensor, to be
    moved to the device) and the factor on rotated values."""
    import torch
    freqs = torch.empty(max(R, 0) // 2, dtype=torch.float64)
    magnitude = ctypes.c_double(0.0)
    _check(_lib.bonsai_rope_frequencies(freqs.data_ptr() or None, ctypes.byref(magnitude), R, base, scaling, factor,
                                        original, low, high), "bonsai_rope_frequencies")
    return freqs, magnitude.value


def bonsai_rope(x, out, freqs, positions, T: int, H: int, D: int, R: int, layout: int = BONSAI_ROPE_HALF,
                magnitude: float = 1.0, ld_x=None, ld_out=None, stream=None) -> None:
    """Rotates T rows of H heads of D elements; x and out may be row-strided matrices, out may be x."""
    import torch
    dev = torch.cuda.current_device()
    xp, ld_x = _rows(x, T, H * D, ld_x, dev)
    op, ld_out = _rows(out, T, H * D, ld_out, dev)
    _check(_call.bonsai_rope(xp, op, _dev(freqs, torch.float64, R // 2, dev), _dev(positions, torch.int32, T, dev), T, H, D,
                            R, ld_x, ld_out, magnitude, layout, _stream_on(stream, dev)), "bonsai_rope")


def _pools(k_cache, v_cache, k_scale, v_scale, dev: int):
    """Pointers of a pair of cache pools and their scales, and (pages, Hkv, page_size, D, kv_type)."""
    import torch
    kind, shape = k_cache.dtype, k_cache.shape
    if kind is not torch.float16 and kind is not torch.float8_e4m3fn:
        raise ValueError("a cache holds float16 or float8_e4m3fn values")
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache are two pools of the same shape: pages x Hkv x page_size x D")
    pages, Hkv, page_size, D = shape
    f32 = torch.float32
    return ((_dev(k_cache, kind, 0, dev), _dev(v_cache, kind, 0, dev), _dev(k_scale, f32, Hkv, dev),
             _dev(v_scale, f32, Hkv, dev)),
            (pages, Hkv, page_size, D, BONSAI_KV_F16 if kind is torch.float16 else BONSAI_KV_E4M3))


def bonsai_rope_append(qkv, q_out, k_cache, v_cache, k_scale, v_scale, freqs, positions, slots, T: int, Hq: int,
                       R: int, layout: int = BONSAI_ROPE_HALF, magnitude: float = 1.0, ld_qkv=None, ld_q=None,
                       stream=None) -> None:
    """Rotates the query heads into q_out and the key heads, with the value heads, into the cache pools
    (pages x Hkv x page_size x D tensors, float16 or float8_e4m3fn with FP32 scales per head)."""
    import torch
    dev = torch.cuda.current_device()
    ptrs, (pages, Hkv, page_size, D, kind) = _pools(k_cache, v_cache, k_scale, v_scale, dev)
    xp, ld_qkv = _rows(qkv, T, (Hq + 2 * Hkv) * D, ld_qkv, dev)
    qp, ld_q = _rows(q_out, T, Hq * D, ld_q, dev)
    _check(_call.bonsai_rope_append(xp, qp, *ptrs, _dev(freqs, torch.float64, R // 2, dev),
                                   _dev(positions, torch.int32, T, dev), _dev(slots, torch.int64, T, dev), T, Hq, Hkv, D,
                                   R, ld_qkv, ld_q, pages, page_size, magnitude, layout, kind, _stream_on(stream, dev)),
           "bonsai_rope_append")


def bonsai_paged_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, lengths, out, B: int, Hq: int,
                           window: int = 0, scale=None, lse=None, ld_q=None, ld_out=None, stream=None) -> None:
    """Attention of one new token per sequence over the cache pools; scale defaults to 1/sqrt(D).
    page_table is a B x max_pages int32 matrix, lengths B int32 values, lse an optional B x Hq FP32 output."""
    import torch
    dev, i32 = torch.cuda.current_device(), torch.int32
    ptrs, (pages, Hkv, page_size, D, kind) = _pools(k_cache, v_cache, k_scale, v_scale, dev)
    qp, ld_q = _rows(q, B, Hq * D, ld_q, dev)
    op, ld_out = _rows(out, B, Hq * D, ld_out, dev)
    width = page_table.shape[-1]
    _check(_call.bonsai_paged_attention(qp, *ptrs, _dev(page_table, i32, B * width, dev), _dev(lengths, i32, B, dev), op,
                                       _dev(lse, torch.float32, B * Hq, dev), B, Hq, Hkv, D, ld_q, ld_out, pages,
                                       page_size, width, window, D ** -0.5 if scale is None else scale, kind,
                                       _stream_on(stream, dev)), "bonsai_paged_attention")


def pack(fmt: int, trits, stream=None):
    """Packs an N x K int8 CUDA tensor of trits; returns the uint8 plane (N x bytes/row)."""
    import torch
    N, K = trits.shape
    out = torch.empty(bonsai_packed_bytes(fmt, N, K), dtype=torch.uint8, device=trits.device)
    fn = {BONSAI_FMT_PTQ1_0: bonsai_pack_ptq1, BONSAI_FMT_PQ2_0: bonsai_pack_pq2,
          BONSAI_FMT_Q1_0: bonsai_pack_q1, BONSAI_FMT_PQ2_0_G64: bonsai_pack_pq2}[fmt]
    fn(trits, out, N, K, stream)
    return out.view(N, -1) if N else out


def ternary_linear(x, packed, scales, N: int, fmt: int, algo: int = BONSAI_ALGO_AUTO,
                   split_k: int = 0, stream=None):
    """y = x' . Wdeq^T for an M x K FP16 CUDA tensor x; returns a new M x N FP16 tensor."""
    import torch
    M, K = x.shape
    y = torch.empty((M, N), dtype=torch.float16, device=x.device)
    bonsai_ternary_linear_algo(x, packed, scales, y, M, N, K, fmt, algo, split_k, stream)
    return y
