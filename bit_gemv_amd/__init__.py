"""Python binding of librfp2 (ROCmFP2 GEMV / GEMM for MI355X).

Argument marshalling only: every function here has the name and argument
order of the C entry point declared in include/rfp2.h, takes torch tensors
that live on the GPU, checks that each tensor has the dtype, layout and size
the call will touch (so that no kernel reads or writes outside a buffer), and
passes raw device pointers plus the current HIP stream to the library.  All
computation happens in the library's HIP kernels; there is no fallback path:
if librfp2.so is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "librfp2.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "rfp2.h")

KV_F16, KV_I8 = 0, 1
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ATTN_MAX_NEW = 8

RFP2_OK, RFP2_E_NULL, RFP2_E_SHAPE, RFP2_E_ALIGN, RFP2_E_LAUNCH = 0, -1, -2, -3, -4
GEMV_MAX_M = 8

_lib = None

_c_i64 = ctypes.c_int64
_c_p = ctypes.c_void_p
_c_f64 = ctypes.c_double


class _KvCacheStruct(ctypes.Structure):
    """rfp2_kv_cache of include/rfp2.h."""
    _fields_ = [("k", _c_p), ("v", _c_p), ("k_scale", _c_p), ("v_scale", _c_p),
                ("page_table", _c_p), ("seqs", _c_i64), ("max_pages", _c_i64),
                ("pages", _c_i64), ("page_size", _c_i64), ("kv_heads", _c_i64),
                ("head_dim", _c_i64), ("format", ctypes.c_int32)]


_c_cache = ctypes.POINTER(_KvCacheStruct)
_SIGNATURES = {
    "rfp2_abi_version": ([], ctypes.c_int),
    "rfp2_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "rfp2_quantize_acts": ([_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p], ctypes.c_int),
    "rfp2_quantize_weights": ([_c_p, _c_i64, _c_i64, _c_p, _c_p], ctypes.c_int),
    "rfp2_quantize_weights_imatrix": ([_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p], ctypes.c_int),
    "rfp2_gemv": ([_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_p, _c_p], ctypes.c_int),
    "rfp2_gemm": ([_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_p, _c_p], ctypes.c_int),
    "rfp2_gemm_f16": ([_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_p, _c_p], ctypes.c_int),
    "rfp2_moe_gemv": ([_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_i64, _c_p, _c_p, _c_p,
                       _c_p, _c_p], ctypes.c_int),
    "rfp2_moe_gemv_tokens": ([_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_i64, _c_i64, _c_p, _c_p,
                              _c_p, _c_p, _c_p], ctypes.c_int),
    "rfp2_moe_sort": ([_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p], ctypes.c_int),
    "rfp2_moe_gemm_workspace_bytes": ([_c_i64, _c_i64, _c_i64], ctypes.c_size_t),
    "rfp2_moe_gemm": ([_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p,
                       _c_p, _c_p, ctypes.c_size_t, _c_p], ctypes.c_int),
    "rfp2_moe_gemm_noalloc": ([_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_i64, _c_i64, _c_p, _c_p,
                               _c_p, _c_p, _c_p], ctypes.c_int),
    "rfp2_rope_freqs": ([_c_i64, _c_f64, _c_f64, _c_f64, _c_f64, _c_f64, _c_p, _c_p],
                        ctypes.c_int),
    "rfp2_rope": ([_c_p, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i64, ctypes.c_int,
                   _c_f64, _c_p, _c_i64, _c_p], ctypes.c_int),
    "rfp2_kv_write": ([_c_cache, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p],
                      ctypes.c_int),
    "rfp2_rope_kv_write": ([_c_cache, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64,
                            _c_p, _c_p, _c_p, _c_i64, ctypes.c_int, _c_f64, _c_p, _c_i64, _c_p,
                            _c_p], ctypes.c_int),
    "rfp2_kv_read": ([_c_cache, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p],
                     ctypes.c_int),
    "rfp2_paged_attn_workspace_bytes": ([_c_cache, _c_i64, _c_i64, _c_i64], ctypes.c_size_t),
    "rfp2_paged_attn": ([_c_cache, _c_p, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, ctypes.c_float,
                         _c_i64, _c_p, _c_p, _c_p, ctypes.c_size_t, _c_p], ctypes.c_int),
    "rfp2_read_ceiling": ([_c_p, _c_i64, ctypes.c_uint32, _c_p, _c_p], ctypes.c_int),
    "rfp2_quant_gemv": ([_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p], ctypes.c_int),
    "rfp2_quant_moe_gemv": ([_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_i64, _c_p, _c_p, _c_p,
                             _c_p, _c_p, _c_p], ctypes.c_int),
    "rfp2_debug_decode": ([_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p], ctypes.c_int),
    "rfp2_debug_half_dots": ([_c_p, _c_i64, _c_i64, _c_p, _c_i64, _c_p, _c_p], ctypes.c_int),
    "rfp2_debug_half_sums_mf": ([_c_p, _c_i64, _c_i64, _c_p, _c_i64, _c_p, _c_p], ctypes.c_int),
    "rfp2_debug_decode_f16": ([_c_p, _c_i64, _c_i64, ctypes.c_int, _c_p, _c_p], ctypes.c_int),
    "rfp2_debug_decode_i8": ([_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p], ctypes.c_int),
}


class Rfp2Error(RuntimeError):
    def __init__(self, call: str, status: int):
        self.status = status
        super().__init__(f"{call}: status {status}: {rfp2_status_string(status)}")


def lib() -> ctypes.CDLL:
    """The loaded librfp2.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -c 'import "
                "__graft_entry__ as g; g.build()'` (ROCm hipcc, gfx950)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def header_symbols() -> list[str]:
    """Names of the functions declared in include/rfp2.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:[\w\s\*]+?)\b(rfp2_\w+)\s*\(", text, re.M)))


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
def _stream(stream):
    import torch
    if stream is None:
        # the handle without a Stream object around it: 0.3 us against 2.9, in every call
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t, dtype, numel: int, name: str):
    """Device pointer of `t` after checking what the call will touch."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, the call needs {numel}")
    return t.data_ptr()


def _check(call: str, status: int):
    if status != RFP2_OK:
        raise Rfp2Error(call, status)


def _blocks(K: int) -> int:
    return K // 32


# ---------------------------------------------------------------------------
# entry points (same names and argument order as the C ABI)
# ---------------------------------------------------------------------------
def rfp2_abi_version() -> int:
    return lib().rfp2_abi_version()


def rfp2_status_string(status: int) -> str:
    return lib().rfp2_status_string(int(status)).decode()


def rfp2_quantize_acts(a, M: int, K: int, q, d, stream=None) -> None:
    import torch
    _check("rfp2_quantize_acts", lib().rfp2_quantize_acts(
        _ptr(a, torch.float32, M * K, "a"), M, K, _ptr(q, torch.int8, M * K, "q"),
        _ptr(d, torch.float32, M * _blocks(K), "d"), _stream(stream)))


def rfp2_quantize_weights(x, N: int, K: int, w, stream=None) -> None:
    import torch
    _check("rfp2_quantize_weights", lib().rfp2_quantize_weights(
        _ptr(x, torch.float32, N * K, "x"), N, K,
        _ptr(w, torch.uint8, N * _blocks(K) * 10, "w"), _stream(stream)))


def rfp2_quantize_weights_imatrix(x, N: int, K: int, importance, w, stream=None) -> None:
    import torch
    _check("rfp2_quantize_weights_imatrix", lib().rfp2_quantize_weights_imatrix(
        _ptr(x, torch.float32, N * K, "x"), N, K,
        _ptr(importance, torch.float32, K, "importance"),
        _ptr(w, torch.uint8, N * _blocks(K) * 10, "w"), _stream(stream)))


def rfp2_gemv(w, N: int, K: int, q, d, M: int, y, stream=None) -> None:
    import torch
    _check("rfp2_gemv", lib().rfp2_gemv(
        _ptr(w, torch.uint8, N * _blocks(K) * 10, "w"), N, K,
        _ptr(q, torch.int8, M * K, "q"), _ptr(d, torch.float32, M * _blocks(K), "d"), M,
        _ptr(y, torch.float32, M * N, "y"), _stream(stream)))


def rfp2_gemm(w, N: int, K: int, q, d, M: int, y, stream=None) -> None:
    import torch
    _check("rfp2_gemm", lib().rfp2_gemm(
        _ptr(w, torch.uint8, N * _blocks(K) * 10, "w"), N, K,
        _ptr(q, torch.int8, M * K, "q"), _ptr(d, torch.float32, M * _blocks(K), "d"), M,
        _ptr(y, torch.float32, M * N, "y"), _stream(stream)))


def rfp2_gemm_f16(w, N: int, K: int, q, d, M: int, y, stream=None) -> None:
    import torch
    _check("rfp2_gemm_f16", lib().rfp2_gemm_f16(
        _ptr(w, torch.uint8, N * _blocks(K) * 10, "w"), N, K,
        _ptr(q, torch.int8, M * K, "q"), _ptr(d, torch.float32, M * _blocks(K), "d"), M,
        _ptr(y, torch.float32, M * N, "y"), _stream(stream)))


def rfp2_moe_gemv(w, E: int, N: int, K: int, ids, top_k: int, q, d, y, err=None,
                  stream=None) -> None:
    import torch
    errp = None if err is None else _ptr(err, torch.int32, 1, "err")
    _check("rfp2_moe_gemv", lib().rfp2_moe_gemv(
        _ptr(w, torch.uint8, E * N * _blocks(K) * 10, "w"), E, N, K,
        _ptr(ids, torch.int32, top_k, "ids"), top_k,
        _ptr(q, torch.int8, K, "q"), _ptr(d, torch.float32, _blocks(K), "d"),
        _ptr(y, torch.float32, top_k * N, "y"), errp, _stream(stream)))


def rfp2_moe_gemv_tokens(w, E: int, N: int, K: int, ids, T: int, top_k: int, q, d, y,
                         err=None, stream=None) -> None:
    import torch
    errp = None if err is None else _ptr(err, torch.int32, 1, "err")
    _check("rfp2_moe_gemv_tokens", lib().rfp2_moe_gemv_tokens(
        _ptr(w, torch.uint8, E * N * _blocks(K) * 10, "w"), E, N, K,
        _ptr(ids, torch.int32, T * top_k, "ids"), T, top_k,
        _ptr(q, torch.int8, T * K, "q"), _ptr(d, torch.float32, T * _blocks(K), "d"),
        _ptr(y, torch.float32, T * top_k * N, "y"), errp, _stream(stream)))


def rfp2_moe_sort(ids, S: int, E: int, offsets, order, err=None, stream=None) -> None:
    import torch
    errp = None if err is None else _ptr(err, torch.int32, 1, "err")
    _check("rfp2_moe_sort", lib().rfp2_moe_sort(
        _ptr(ids, torch.int32, S, "ids"), S, E, _ptr(offsets, torch.int32, E + 1, "offsets"),
        _ptr(order, torch.int32, S, "order"), errp, _stream(stream)))


def rfp2_moe_gemm_workspace_bytes(E: int, T: int, top_k: int) -> int:
    return int(lib().rfp2_moe_gemm_workspace_bytes(E, T, top_k))


def rfp2_moe_gemm(w, E: int, N: int, K: int, ids, T: int, top_k: int, q, d, y, err=None,
                  workspace=None, stream=None) -> None:
    """workspace: a uint8 GPU tensor of at least rfp2_moe_gemm_workspace_bytes
    bytes; when None, one is allocated for this call."""
    import torch
    need = rfp2_moe_gemm_workspace_bytes(E, T, top_k)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=y.device)
    errp = None if err is None else _ptr(err, torch.int32, 1, "err")
    _check("rfp2_moe_gemm", lib().rfp2_moe_gemm(
        _ptr(w, torch.uint8, E * N * _blocks(K) * 10, "w"), E, N, K,
        _ptr(ids, torch.int32, T * top_k, "ids"), T, top_k,
        _ptr(q, torch.int8, T * K, "q"), _ptr(d, torch.float32, T * _blocks(K), "d"),
        _ptr(y, torch.float32, T * top_k * N, "y"), errp,
        _ptr(workspace, torch.uint8, need, "workspace"), workspace.numel(), _stream(stream)))


READ_CEILING_OUTPUTS = 524288


MOE_GEMM_NOALLOC_MAX_BYTES = 1 << 20


def rfp2_moe_gemm_noalloc(w, E: int, N: int, K: int, ids, T: int, top_k: int, q, d, y,
                          err=None, stream=None) -> None:
    import torch
    errp = None if err is None else _ptr(err, torch.int32, 1, "err")
    _check("rfp2_moe_gemm_noalloc", lib().rfp2_moe_gemm_noalloc(
        _ptr(w, torch.uint8, E * N * _blocks(K) * 10, "w"), E, N, K,
        _ptr(ids, torch.int32, T * top_k, "ids"), T, top_k,
        _ptr(q, torch.int8, T * K, "q"), _ptr(d, torch.float32, T * _blocks(K), "d"),
        _ptr(y, torch.float32, T * top_k * N, "y"), errp, _stream(stream)))


def read_ceiling_threads(nbytes: int) -> int:
    """Threads of the read helper's grid for nbytes (256 per workgroup)."""
    return 256 * min(2048, max(1, -(-(nbytes // 16) // 256)))


def rfp2_read_ceiling(buf, nbytes: int, out, magic: int = 0x9E3779B9, stream=None) -> None:
    """Measurement helper: read nbytes of buf with plain 16-byte loads; a
    thread whose XOR of what it read equals `magic` writes it to out[thread]."""
    import torch
    _check("rfp2_read_ceiling", lib().rfp2_read_ceiling(
        _ptr(buf, torch.uint8, nbytes, "buf"), nbytes, int(magic) & 0xFFFFFFFF,
        _ptr(out, torch.int32, read_ceiling_threads(nbytes), "out"), _stream(stream)))


def rfp2_quant_gemv(w, N: int, K: int, a, q, d, y, stream=None) -> None:
    import torch
    _check("rfp2_quant_gemv", lib().rfp2_quant_gemv(
        _ptr(w, torch.uint8, N * _blocks(K) * 10, "w"), N, K,
        _ptr(a, torch.float32, K, "a"), _ptr(q, torch.int8, K, "q"),
        _ptr(d, torch.float32, _blocks(K), "d"), _ptr(y, torch.float32, N, "y"),
        _stream(stream)))


def rfp2_quant_moe_gemv(w, E: int, N: int, K: int, ids, top_k: int, a, q, d, y, err=None,
                        stream=None) -> None:
    import torch
    errp = None if err is None else _ptr(err, torch.int32, 1, "err")
    _check("rfp2_quant_moe_gemv", lib().rfp2_quant_moe_gemv(
        _ptr(w, torch.uint8, E * N * _blocks(K) * 10, "w"), E, N, K,
        _ptr(ids, torch.int32, top_k, "ids"), top_k,
        _ptr(a, torch.float32, K, "a"), _ptr(q, torch.int8, K, "q"),
        _ptr(d, torch.float32, _blocks(K), "d"),
        _ptr(y, torch.float32, top_k * N, "y"), errp, _stream(stream)))


class KvCache:
    """The rfp2_kv_cache of a set of tensors (kept alive by this object):

      k [pages, kv_heads, page_size, head_dim] and v [pages, kv_heads,
      page_size/8, head_dim, 8], both float16 (KV_F16) or int8 (KV_I8);
      k_scale, v_scale [pages, kv_heads, page_size/8, head_dim/32, 8] float32
      for int8, None for float16; page_table [seqs, max_pages] int32.

    All contiguous, on one GPU.  The tensors' contents may change between
    calls (the page table's too); their shapes are checked here, once."""

    def __init__(self, k, v, k_scale, v_scale, page_table):
        import torch
        if not isinstance(k, torch.Tensor) or k.dtype not in (torch.float16, torch.int8):
            raise TypeError("k must be a float16 or int8 torch tensor")
        if k.dim() != 4:
            raise ValueError("k must be [pages, kv_heads, page_size, head_dim]")
        pages, heads, size, dim = k.shape
        i8 = k.dtype == torch.int8
        if size % 8 or dim % 32:
            raise ValueError("page_size must be a multiple of 8 and head_dim of 32")

        def check(t, dtype, shape, name):
            p = _ptr(t, dtype, 0, name)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must have shape {shape} (got {tuple(t.shape)})")
            if t.device != k.device:
                raise ValueError(f"{name} must be on {k.device} like k (got {t.device})")
            return p

        scale_shape = (pages, heads, size // 8, dim // 32, 8)
        kp = check(k, k.dtype, (pages, heads, size, dim), "k")
        vp = check(v, k.dtype, (pages, heads, size // 8, dim, 8), "v")
        if i8:
            ksp = check(k_scale, torch.float32, scale_shape, "k_scale")
            vsp = check(v_scale, torch.float32, scale_shape, "v_scale")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a float16 cache has no scales")
        else:
            ksp = vsp = None
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be a [seqs, max_pages] torch tensor")
        tp = check(page_table, torch.int32, tuple(page_table.shape), "page_table")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.page_table = page_table
        self.device, self.kv_heads, self.head_dim = k.device, heads, dim
        self.seqs, self.page_size = page_table.shape[0], size
        self.format = KV_I8 if i8 else KV_F16
        self._struct = _KvCacheStruct(kp, vp, ksp, vsp, tp, page_table.shape[0],
                                      page_table.shape[1], pages, size, heads, dim, self.format)

    @classmethod
    def allocate(cls, format: int, pages: int, page_size: int, kv_heads: int, head_dim: int,
                 page_table):
        """A cache of new, zeroed memory (on the page table's GPU) behind a page table."""
        import torch
        if format not in (KV_F16, KV_I8):
            raise ValueError("format must be KV_F16 or KV_I8")
        dt = torch.int8 if format == KV_I8 else torch.float16

        def zeros(*shape, dtype=dt):
            return torch.zeros(shape, dtype=dtype, device=page_table.device)

        s = [zeros(pages, kv_heads, page_size // 8, head_dim // 32, 8, dtype=torch.float32)
             for _ in range(2)] if format == KV_I8 else [None, None]
        return cls(zeros(pages, kv_heads, page_size, head_dim),
                   zeros(pages, kv_heads, page_size // 8, head_dim, 8), *s, page_table)


def _cache_ref(cache):
    if not isinstance(cache, KvCache):
        raise TypeError("cache must be a KvCache")
    return ctypes.byref(cache._struct)


def _rows(t, T: int, width: int, name: str):
    """(device pointer, elements between rows) of a float32 tensor whose first
    dimension counts T or more rows of `width` or more values, contiguous in a
    row (so a slice of a product's columns will do)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU (got {t.device})")
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be torch.float32 (got {t.dtype})")
    shape = t.shape
    if len(shape) < 2 or shape[0] < T:
        raise ValueError(f"{name} must have {T} or more rows (shape {tuple(shape)})")
    stride, *inner = t.stride()
    row = 1
    for n, s in zip(shape[:0:-1], reversed(inner)):
        if s != row and n != 1:
            row = -1
            break
        row *= n
    if row < width:
        raise ValueError(f"a row of {name} must be {width} or more contiguous values")
    return t.data_ptr(), stride if T > 1 else width


def rfp2_rope_freqs(rot: int, base: float, factor: float, orig_len: float, low_turns: float,
                    high_turns: float, freqs, stream=None) -> None:
    import torch
    _check("rfp2_rope_freqs", lib().rfp2_rope_freqs(
        rot, base, factor, orig_len, low_turns, high_turns,
        _ptr(freqs, torch.float64, rot // 2, "freqs"), _stream(stream)))


def rfp2_rope(x, T: int, H: int, D: int, pos, freqs, rot: int, style: int, mscale: float, y,
              stream=None) -> None:
    """x, y: T rows of H * D values ([T, H, D] or [T, H * D]); rows may lie
    apart.  y may be x."""
    import torch
    xp, xs = _rows(x, T, H * D, "x")
    yp, ys = _rows(y, T, H * D, "y")
    _check("rfp2_rope", lib().rfp2_rope(
        xp, T, H, D, xs, _ptr(pos, torch.int32, T, "pos"),
        _ptr(freqs, torch.float64, rot // 2, "freqs"), rot, style, mscale, yp, ys,
        _stream(stream)))


def rfp2_kv_write(cache, k, v, T: int, seq, pos, err=None, stream=None) -> None:
    import torch
    ref = _cache_ref(cache)
    row = cache.kv_heads * cache.head_dim
    kp, ks = _rows(k, T, row, "k")
    vp, vs = _rows(v, T, row, "v")
    errp = None if err is None else _ptr(err, torch.int32, 1, "err")
    _check("rfp2_kv_write", lib().rfp2_kv_write(
        ref, kp, vp, T, ks, vs, _ptr(seq, torch.int32, T, "seq"),
        _ptr(pos, torch.int32, T, "pos"), errp, _stream(stream)))


def rfp2_rope_kv_write(cache, q, k, v, T: int, H: int, seq, pos, freqs, rot: int, style: int,
                       mscale: float, q_out, err=None, stream=None) -> None:
    """q, q_out: T rows of H heads (both None with H == 0: keys alone)."""
    import torch
    ref = _cache_ref(cache)
    row = cache.kv_heads * cache.head_dim
    qp, qs, op, os_ = None, 0, None, 0
    if H:
        qp, qs = _rows(q, T, H * cache.head_dim, "q")
        op, os_ = _rows(q_out, T, H * cache.head_dim, "q_out")
    kp, ks = _rows(k, T, row, "k")
    vp, vs = _rows(v, T, row, "v")
    errp = None if err is None else _ptr(err, torch.int32, 1, "err")
    _check("rfp2_rope_kv_write", lib().rfp2_rope_kv_write(
        ref, qp, kp, vp, T, H, qs, ks, vs, _ptr(seq, torch.int32, T, "seq"),
        _ptr(pos, torch.int32, T, "pos"), _ptr(freqs, torch.float64, rot // 2, "freqs"), rot,
        style, mscale, op, os_, errp, _stream(stream)))


def rfp2_kv_read(cache, T: int, seq, pos, k, v, err=None, stream=None) -> None:
    import torch
    ref = _cache_ref(cache)
    row = cache.kv_heads * cache.head_dim
    kp, ks = _rows(k, T, row, "k")
    vp, vs = _rows(v, T, row, "v")
    errp = None if err is None else _ptr(err, torch.int32, 1, "err")
    _check("rfp2_kv_read", lib().rfp2_kv_read(
        ref, T, _ptr(seq, torch.int32, T, "seq"),
        _ptr(pos, torch.int32, T, "pos"), kp, vp, ks, vs, errp, _stream(stream)))


def rfp2_paged_attn_workspace_bytes(cache, B: int, new_tokens: int, H: int) -> int:
    return int(lib().rfp2_paged_attn_workspace_bytes(_cache_ref(cache), B, new_tokens, H))


def rfp2_paged_attn(cache, q, B: int, new_tokens: int, H: int, lens, scale: float, y,
                    window: int = 0, err=None, workspace=None, stream=None) -> None:
    """q: [B, new_tokens, ...] or [B * new_tokens, ...], H * D contiguous values
    a row, the rows evenly spaced (a buffer of more sequences is passed as q[:B]);
    y: [B, new_tokens, H, D], contiguous.
    workspace: a uint8 GPU tensor of at least rfp2_paged_attn_workspace_bytes
    bytes; when None, one is allocated for this call (on the current stream
    only: a call on another stream brings its own)."""
    import torch
    ref = _cache_ref(cache)
    rows, width = B * new_tokens, H * cache.head_dim
    if isinstance(q, torch.Tensor) and q.dim() > 2 and q.shape[1] == new_tokens:
        if q.shape[0] == B:
            if B > 1 and new_tokens > 1 and q.stride(0) != new_tokens * q.stride(1):
                raise ValueError("the rows of q must be evenly spaced")
            q = q[:, 0] if new_tokens == 1 else q[0] if B == 1 else q.view(rows, *q.shape[2:])
        elif q.shape[0] > B and new_tokens > 1 and q[0, 0].numel() >= width:
            raise ValueError(f"q holds {q.shape[0]} sequences, not {B}: pass q[:{B}]")
    qp, qs = _rows(q, rows, width, "q")
    if workspace is None:
        if stream is not None:
            raise ValueError("a call on a stream of its own needs a workspace")
        need = rfp2_paged_attn_workspace_bytes(cache, B, new_tokens, H)
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=y.device)
    errp = None if err is None else _ptr(err, torch.int32, 1, "err")
    _check("rfp2_paged_attn", lib().rfp2_paged_attn(
        ref, qp, B, new_tokens, H, qs, _ptr(lens, torch.int32, B, "lens"), scale,
        window, _ptr(y, torch.float32, rows * width, "y"), errp,
        _ptr(workspace, torch.uint8, 0, "workspace"), workspace.numel(), _stream(stream)))


def rfp2_debug_decode(w, N: int, K: int, codes_out, scales_out, stream=None) -> None:
    import torch
    _check("rfp2_debug_decode", lib().rfp2_debug_decode(
        _ptr(w, torch.uint8, N * _blocks(K) * 10, "w"), N, K,
        _ptr(codes_out, torch.int8, N * K, "codes_out"),
        _ptr(scales_out, torch.float32, N * K // 16, "scales_out"), _stream(stream)))


def rfp2_debug_half_dots(w, N: int, K: int, q, M: int, sums_out, stream=None) -> None:
    import torch
    _check("rfp2_debug_half_dots", lib().rfp2_debug_half_dots(
        _ptr(w, torch.uint8, N * _blocks(K) * 10, "w"), N, K,
        _ptr(q, torch.int8, M * K, "q"), M,
        _ptr(sums_out, torch.int32, M * N * _blocks(K) * 2, "sums_out"), _stream(stream)))


def rfp2_debug_half_sums_mf(w, N: int, K: int, q, M: int, sums_out, stream=None) -> None:
    import torch
    _check("rfp2_debug_half_sums_mf", lib().rfp2_debug_half_sums_mf(
        _ptr(w, torch.uint8, N * _blocks(K) * 10, "w"), N, K,
        _ptr(q, torch.int8, M * K, "q"), M,
        _ptr(sums_out, torch.int32, M * N * _blocks(K) * 2, "sums_out"), _stream(stream)))


def rfp2_debug_decode_f16(w, N: int, K: int, form: int, h_out, stream=None) -> None:
    """h_out: int16 tensor [N, K] receiving IEEE half-precision bit patterns."""
    import torch
    _check("rfp2_debug_decode_f16", lib().rfp2_debug_decode_f16(
        _ptr(w, torch.uint8, N * _blocks(K) * 10, "w"), N, K, int(form),
        _ptr(h_out, torch.int16, N * K, "h_out"), _stream(stream)))


def rfp2_debug_decode_i8(w, N: int, K: int, wa_out, wb_out, scales_out, stream=None) -> None:
    """wa_out, wb_out: int8 [N, K]; scales_out: fp32 [N, K/32, 6]."""
    import torch
    _check("rfp2_debug_decode_i8", lib().rfp2_debug_decode_i8(
        _ptr(w, torch.uint8, N * _blocks(K) * 10, "w"), N, K,
        _ptr(wa_out, torch.int8, N * K, "wa_out"),
        _ptr(wb_out, torch.int8, N * K, "wb_out"),
        _ptr(scales_out, torch.float32, N * _blocks(K) * 6, "scales_out"), _stream(stream)))
