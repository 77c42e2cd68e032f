"""Python binding of libiq (include/iq.h): ctypes argument marshalling only.

Every step of the path runs in the library's CUDA kernels.  PyTorch supplies
device memory and the current stream.  There is no fallback: if the library
has not been built, or the device is not sm_103, the calls raise.
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

from .build import LIB_PATH

LATENT_DIM = 1536
N_HEADS = 64
HEAD_DIM = 128
Q_DIM = 8192
SMALL_M_MAX = 128

_STATUS = {0: "IQ_OK", -1: "IQ_ERR_ARG", -2: "IQ_ERR_ALIGN", -3: "IQ_ERR_SHAPE", -4: "IQ_ERR_ARCH",
           -5: "IQ_ERR_CUDA", -6: "IQ_ERR_WORKSPACE", -7: "IQ_ERR_TIMEOUT"}

# Every symbol include/iq.h declares, with (restype, argtypes).
_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_LL = ctypes.c_longlong
SIGNATURES = {
    "iq_status_str": (ctypes.c_char_p, [_I]),
    "iq_device_status": (_I, [ctypes.POINTER(ctypes.c_uint32), _I]),
    "iq_set_wait_timeout_ns": (None, [ctypes.c_uint64]),
    "iq_selftest_workspace": (_SZ, []),
    "iq_selftest_wait_timeout": (_I, [_P, _SZ, ctypes.c_uint64, ctypes.POINTER(ctypes.c_uint32), _P]),
    "iq_debug_fail_next_setups": (None, [_I]),
    "iq_debug_e2m1_codes": (_I, [_P, ctypes.c_longlong, _P, _P]),
    "iq_fp8_scale_words": (_SZ, [_I, _I]),
    "iq_fp8_quant_1x128_ue8m0": (_I, [_P, _I, _I, _I, _P, _I, _P, _P]),
    "iq_prepare_q_workspace": (_SZ, [_I]),
    "iq_prepare_q": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "iq_prepare_q_debug": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "iq_gemm_rope_hadamard_fp4": (_I, [_P, _P, _I, _P, _P, _P, _P, _P, _P, _P]),
    "iq_prepare_q_static": (_I, [_P, _I, _P, _P, _P, _P, _P, _P]),
    "iq_set_small_m_threshold": (_I, [_I]),
    "iq_small_m_threshold": (_I, []),
    "iq_set_gemm_tiling": (None, [_I, _I]),
    "iq_set_quant_fusion": (_I, [_I]),
    "iq_debug_delay_quant_ns": (None, [ctypes.c_uint64]),
    "iq_fp4_scale_bytes": (_SZ, [_I]),
    "iq_prepare_q_ex": (_I, [_P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _SZ, _P]),
    "iq_prepare_q_host_workspace": (_SZ, [_I, _I]),
    "iq_prepare_q_host": (_I, [_P, _I, _P, _P, _P, _I, _P, _P, _P, _SZ, _P]),
    "iq_set_host_chunk_rows": (_I, [_I]),
    "iq_host_chunk_rows": (_I, []),
    "iq_indexer_logits": (_I, [_P, _P, _I, _P, _P, _I, _P, _P, _P, ctypes.c_longlong, _P]),
    "iq_indexer_topk": (_I, [_P, ctypes.c_longlong, _I, _I, _P, _I, _P, _P]),
    "iq_kv_cache_write": (_I, [_P, _P, _P, _LL, _P, _LL, _P]),
    "iq_kv_cache_read": (_I, [_P, _P, _P, _LL, _P, _LL, _P]),
    "iq_kv_attention": (_I, [_P, _P, _P, _LL, _I, ctypes.c_float, _P, _LL, _P, _SZ, _P]),
    "iq_kv_attention_topk": (_I, [_P, _P, _P, _LL, _I, _P, _LL, _I, ctypes.c_float, _P, _LL, _P, _SZ, _P]),
    "iq_kv_attention_workspace": (_SZ, [_I, _I, _I, _I]),
}

# FP4 output variants (include/iq.h, iq_fp4_format).
FP4_FORMATS = {"mx": 0, "mx_ocp": 1, "nv": 2}

_lib = None


class IQError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {_STATUS.get(code, code)} ({status_str(code)})")
        self.code = code


def lib() -> ctypes.CDLL:
    """The loaded libiq.so.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libiq.so is not built ({LIB_PATH}); run python -m fp4_fp8_quant_gb300.build")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_str(code: int) -> str:
    try:
        return lib().iq_status_str(code).decode()
    except ImportError:
        return _STATUS.get(code, str(code))


def _check(code: int, what: str):
    if code != 0:
        raise IQError(code, what)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _require(t: torch.Tensor, name: str, dtypes, shape=None, contiguous=True):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_U8 = (torch.uint8, torch.float8_e4m3fn)


def scale_words(M: int, K: int) -> int:
    return int(lib().iq_fp8_scale_words(M, K))


def fp8_quant_1x128_ue8m0(x: torch.Tensor, y: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                          stream=None):
    """BF16 [M, K] (row stride may exceed K) -> (E4M3 codes uint8 [M, K],
    packed UE8M0 scales int32 [ceil(K/512), align4(M)])."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D tensor with unit column stride")
    _require(x, "x", (torch.bfloat16,), contiguous=False)
    M, K = x.shape
    if y is None:
        y = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((max(1, -(-K // 512)), (M + 3) // 4 * 4), dtype=torch.int32, device=x.device)
    if y.dim() != 2 or y.stride(1) != 1:
        raise ValueError("y must be a 2-D tensor with unit column stride")
    _require(y, "y", _U8, contiguous=False)
    _require(scales, "scales", (torch.int32,))
    _check(lib().iq_fp8_quant_1x128_ue8m0(_ptr(x), M, K, x.stride(0), _ptr(y), y.stride(0), _ptr(scales),
                                          _stream(stream)), "iq_fp8_quant_1x128_ue8m0")
    return y, scales


def prepare_q_workspace_bytes(M: int) -> int:
    return int(lib().iq_prepare_q_workspace(M))


def fp4_scale_bytes(fp4_format: str = "mx") -> int:
    """Scale bytes per token of an FP4 output variant (256 or 512)."""
    return int(lib().iq_fp4_scale_bytes(FP4_FORMATS[fp4_format]))


def _prepare_out(M, device, q_fp4, q_sf, fp4_format="mx"):
    sf_cols = Q_DIM // 16 if fp4_format == "nv" else Q_DIM // 32
    if q_fp4 is None:
        q_fp4 = torch.empty((M, Q_DIM // 2), dtype=torch.uint8, device=device)
    if q_sf is None:
        q_sf = torch.empty((M, sf_cols), dtype=torch.uint8, device=device)
    _require(q_fp4, "q_fp4", (torch.uint8,), (M, Q_DIM // 2))
    _require(q_sf, "q_sf", (torch.uint8,), (M, sf_cols))
    return q_fp4, q_sf


def prepare_q(latent: torch.Tensor, wq: torch.Tensor, wq_sf: torch.Tensor, positions: torch.Tensor, *,
              q_fp4: torch.Tensor | None = None, q_sf: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, q_prequant: torch.Tensor | None = None,
              debug: bool = False, fp4_format: str = "mx", stream=None):
    """Indexer-Q preparation: returns (q_fp4 uint8 [M, 4096], q_sf uint8
    [M, 256] ([M, 512] for fp4_format="nv")) and, with debug=True, also the
    float32 pre-quant Q [M, 8192].  fp4_format: "mx" (default), "mx_ocp" or
    "nv" (include/iq.h, FP4 output variants)."""
    M = latent.shape[0]
    if fp4_format not in FP4_FORMATS:
        raise ValueError(f"fp4_format must be one of {sorted(FP4_FORMATS)}")
    _require(latent, "latent", (torch.bfloat16,), (M, LATENT_DIM))
    _require(wq, "wq", _U8, (Q_DIM, LATENT_DIM))
    _require(wq_sf, "wq_sf", (torch.uint8,), (N_HEADS, LATENT_DIM // 128))
    _require(positions, "positions", (torch.int32,), (M,))
    q_fp4, q_sf = _prepare_out(M, latent.device, q_fp4, q_sf, fp4_format)
    ws_bytes = prepare_q_workspace_bytes(M)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=latent.device)
    _require(workspace, "workspace", (torch.uint8,))
    if debug and q_prequant is None:
        q_prequant = torch.empty((M, Q_DIM), dtype=torch.float32, device=latent.device)
    if fp4_format != "mx":
        if q_prequant is not None:
            _require(q_prequant, "q_prequant", (torch.float32,), (M, Q_DIM))
        _check(lib().iq_prepare_q_ex(_ptr(latent), M, _ptr(wq), _ptr(wq_sf), _ptr(positions),
                                     FP4_FORMATS[fp4_format], _ptr(q_fp4), _ptr(q_sf), _ptr(q_prequant),
                                     _ptr(workspace), workspace.numel(), _stream(stream)), "iq_prepare_q_ex")
        return (q_fp4, q_sf, q_prequant) if q_prequant is not None else (q_fp4, q_sf)
    if q_prequant is not None:
        _require(q_prequant, "q_prequant", (torch.float32,), (M, Q_DIM))
        _check(lib().iq_prepare_q_debug(_ptr(latent), M, _ptr(wq), _ptr(wq_sf), _ptr(positions), _ptr(q_fp4),
                                        _ptr(q_sf), _ptr(q_prequant), _ptr(workspace), workspace.numel(),
                                        _stream(stream)), "iq_prepare_q_debug")
        return q_fp4, q_sf, q_prequant
    _check(lib().iq_prepare_q(_ptr(latent), M, _ptr(wq), _ptr(wq_sf), _ptr(positions), _ptr(q_fp4), _ptr(q_sf),
                              _ptr(workspace), workspace.numel(), _stream(stream)), "iq_prepare_q")
    return q_fp4, q_sf


def _require_host_side(t: torch.Tensor, name: str, dtypes, shape):
    """A page-locked CPU tensor (or a CUDA tensor) of the given dtype and shape."""
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be in page-locked host memory (tensor.pin_memory()) or on the GPU")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def prepare_q_host_workspace_bytes(M: int, fp4_format: str = "mx") -> int:
    return int(lib().iq_prepare_q_host_workspace(M, FP4_FORMATS[fp4_format]))


def prepare_q_host(latent: torch.Tensor, wq: torch.Tensor, wq_sf: torch.Tensor, positions: torch.Tensor, *,
                   q_fp4: torch.Tensor | None = None, q_sf: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, fp4_format: str = "mx", stream=None):
    """Indexer-Q preparation on host-resident tokens (iq_prepare_q_host):
    latent [M, 1536] bf16 and positions [M] int32 in page-locked host memory;
    returns (q_fp4 uint8 [M, 4096], q_sf uint8 [M, 256] or [M, 512]) in
    page-locked host memory, complete once `stream` reaches the point after
    this call.  W and its scales are on the GPU."""
    M = latent.shape[0]
    if fp4_format not in FP4_FORMATS:
        raise ValueError(f"fp4_format must be one of {sorted(FP4_FORMATS)}")
    _require_host_side(latent, "latent", (torch.bfloat16,), (M, LATENT_DIM))
    _require_host_side(positions, "positions", (torch.int32,), (M,))
    _require(wq, "wq", _U8, (Q_DIM, LATENT_DIM))
    _require(wq_sf, "wq_sf", (torch.uint8,), (N_HEADS, LATENT_DIM // 128))
    sf_cols = Q_DIM // 16 if fp4_format == "nv" else Q_DIM // 32
    if q_fp4 is None:
        q_fp4 = torch.empty((M, Q_DIM // 2), dtype=torch.uint8).pin_memory()
    if q_sf is None:
        q_sf = torch.empty((M, sf_cols), dtype=torch.uint8).pin_memory()
    _require_host_side(q_fp4, "q_fp4", (torch.uint8,), (M, Q_DIM // 2))
    _require_host_side(q_sf, "q_sf", (torch.uint8,), (M, sf_cols))
    if workspace is None:
        workspace = torch.empty(max(prepare_q_host_workspace_bytes(M, fp4_format), 1), dtype=torch.uint8,
                                device=wq.device)
    _require(workspace, "workspace", (torch.uint8,))
    _check(lib().iq_prepare_q_host(_ptr(latent), M, _ptr(wq), _ptr(wq_sf), _ptr(positions),
                                   FP4_FORMATS[fp4_format], _ptr(q_fp4), _ptr(q_sf), _ptr(workspace),
                                   workspace.numel(), _stream(stream)), "iq_prepare_q_host")
    return q_fp4, q_sf


def set_host_chunk_rows(rows: int) -> int:
    """Rows per chunk of prepare_q_host (a multiple of 256); returns the
    previous value."""
    return int(lib().iq_set_host_chunk_rows(int(rows)))


def host_chunk_rows() -> int:
    return int(lib().iq_host_chunk_rows())


def gemm_rope_hadamard_fp4(xq: torch.Tensor, x_scales: torch.Tensor, wq: torch.Tensor, wq_sf: torch.Tensor,
                           positions: torch.Tensor, *, q_fp4: torch.Tensor | None = None,
                           q_sf: torch.Tensor | None = None, q_prequant: torch.Tensor | None = None, stream=None):
    """Second stage alone on an FP8 latent [M, 1536] and its packed scales
    [3, align4(M)]."""
    M = xq.shape[0]
    _require(xq, "xq", _U8, (M, LATENT_DIM))
    _require(x_scales, "x_scales", (torch.int32,), (3, (M + 3) // 4 * 4))
    _require(wq, "wq", _U8, (Q_DIM, LATENT_DIM))
    _require(wq_sf, "wq_sf", (torch.uint8,), (N_HEADS, LATENT_DIM // 128))
    _require(positions, "positions", (torch.int32,), (M,))
    q_fp4, q_sf = _prepare_out(M, xq.device, q_fp4, q_sf)
    if q_prequant is not None:
        _require(q_prequant, "q_prequant", (torch.float32,), (M, Q_DIM))
    _check(lib().iq_gemm_rope_hadamard_fp4(_ptr(xq), _ptr(x_scales), M, _ptr(wq), _ptr(wq_sf), _ptr(positions),
                                           _ptr(q_fp4), _ptr(q_sf), _ptr(q_prequant), _stream(stream)),
           "iq_gemm_rope_hadamard_fp4")
    return q_fp4, q_sf


def device_status(reset: bool = False) -> int:
    """Device status word (bits of waits that gave up); synchronizes."""
    v = ctypes.c_uint32(0)
    code = lib().iq_device_status(ctypes.byref(v), 1 if reset else 0)
    if code not in (0, -7):
        raise IQError(code, "iq_device_status")
    return int(v.value)


def set_gemm_tiling(tile_n: int = 0, order: int = 0) -> None:
    """Tuning override of the CTA-pair kernel's tiling (include/iq.h,
    iq_set_gemm_tiling): tile_n 128 or 256, order 1 feature-major, 2
    token-major or 3 interleaved; 0 restores the default."""
    lib().iq_set_gemm_tiling(int(tile_n), int(order))


def set_quant_fusion(on: bool) -> bool:
    """The quantizer fused into the CTA-pair kernel (include/iq.h,
    iq_set_quant_fusion); returns the previous setting."""
    return bool(lib().iq_set_quant_fusion(1 if on else 0))


def debug_delay_quant_ns(ns: int) -> None:
    """Diagnostics: delay of the fused quantizer's signals (iq_debug_delay_quant_ns)."""
    lib().iq_debug_delay_quant_ns(int(ns))


def set_wait_timeout_ns(ns: int) -> None:
    lib().iq_set_wait_timeout_ns(int(ns))


def set_small_m_threshold(max_tokens: int) -> int:
    """Largest M routed to the small-M (swapped-operand) kernel, clamped to
    [0, 64]; returns the previous value."""
    return int(lib().iq_set_small_m_threshold(int(max_tokens)))


def small_m_threshold() -> int:
    return int(lib().iq_small_m_threshold())


def indexer_logits(q_fp4: torch.Tensor, q_sf: torch.Tensor, k_fp4: torch.Tensor, k_sf: torch.Tensor,
                   weights: torch.Tensor, lengths: torch.Tensor, *, logits: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Indexer scores (include/iq.h, iq_indexer_logits): q_fp4 uint8 [M, 4096],
    q_sf uint8 [M, 256], k_fp4 uint8 [N, 64], k_sf uint8 [N, 4], weights
    float32 [M, 64], lengths int32 [M] -> logits float32 [M, N] (row stride may
    exceed N); entries at s >= lengths[t] are left as they were."""
    M, N = q_fp4.shape[0], k_fp4.shape[0]
    _require(q_fp4, "q_fp4", (torch.uint8,), (M, Q_DIM // 2))
    _require(q_sf, "q_sf", (torch.uint8,), (M, Q_DIM // 32))
    _require(k_fp4, "k_fp4", (torch.uint8,), (N, HEAD_DIM // 2))
    _require(k_sf, "k_sf", (torch.uint8,), (N, HEAD_DIM // 32))
    _require(weights, "weights", (torch.float32,), (M, N_HEADS))
    _require(lengths, "lengths", (torch.int32,), (M,))
    if logits is None:
        logits = torch.empty((M, N), dtype=torch.float32, device=q_fp4.device)
    if logits.dim() != 2 or logits.shape[0] != M or logits.shape[1] < N or logits.stride(1) != 1:
        raise ValueError("logits must be float32 [M, >= N] with unit column stride")
    _require(logits, "logits", (torch.float32,), contiguous=False)
    _check(lib().iq_indexer_logits(_ptr(q_fp4), _ptr(q_sf), M, _ptr(k_fp4), _ptr(k_sf), N, _ptr(weights),
                                   _ptr(lengths), _ptr(logits), logits.stride(0), _stream(stream)),
           "iq_indexer_logits")
    return logits


def indexer_topk(logits: torch.Tensor, lengths: torch.Tensor, k: int, *, N: int | None = None,
                 indices: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Top-k key selection per query row (include/iq.h, iq_indexer_topk):
    int32 [M, k] ascending indices, -1 padded.  N defaults to logits.shape[1]."""
    M = logits.shape[0]
    N = logits.shape[1] if N is None else N
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be a 2-D tensor with unit column stride")
    _require(logits, "logits", (torch.float32,), contiguous=False)
    _require(lengths, "lengths", (torch.int32,), (M,))
    if indices is None:
        indices = torch.empty((M, k), dtype=torch.int32, device=logits.device)
    _require(indices, "indices", (torch.int32,), (M, k))
    _check(lib().iq_indexer_topk(_ptr(logits), logits.stride(0), M, N, _ptr(lengths), int(k), _ptr(indices),
                                 _stream(stream)), "iq_indexer_topk")
    return indices


# ------------------------------------------------------------ 8-bit KV cache

class _KVCacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", _P), ("v_codes", _P), ("k_sf", _P), ("v_sf", _P), ("num_pages", _I), ("kv_heads", _I),
                ("page_size", _I), ("head_dim", _I)]


class _KVBatchStruct(ctypes.Structure):
    _fields_ = [("block_table", _P), ("table_ld", _LL), ("max_pages", _I), ("row_start", _P), ("kv_len", _P),
                ("num_seqs", _I), ("num_rows", _I)]


class KVCache:
    """A paged 8-bit KV cache (include/iq.h, iq_kv_cache) over the caller's
    tensors: k_codes and v_codes uint8 (or float8_e4m3fn)
    [num_pages, kv_heads, page_size, head_dim], k_sf and v_sf uint8
    [num_pages, kv_heads], all contiguous on one GPU.  KVCache.empty allocates
    them."""

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_sf: torch.Tensor, v_sf: torch.Tensor):
        shape = k_codes.shape
        device = k_codes.device
        if not (len(shape) == 4 and v_codes.shape == shape and k_sf.shape == shape[:2] == v_sf.shape and k_codes.is_cuda
                and k_codes.dtype in _U8 and v_codes.dtype in _U8 and k_sf.dtype is v_sf.dtype is torch.uint8
                and device == v_codes.device == k_sf.device == v_sf.device and k_codes.is_contiguous()
                and v_codes.is_contiguous() and k_sf.is_contiguous() and v_sf.is_contiguous()):
            self._explain(k_codes, v_codes, k_sf, v_sf)
        self.device = device
        self.k_codes, self.v_codes, self.k_sf, self.v_sf = k_codes, v_codes, k_sf, v_sf
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = shape
        self._struct = _KVCacheStruct(k_codes.data_ptr(), v_codes.data_ptr(), k_sf.data_ptr(), v_sf.data_ptr(), *shape)

    @staticmethod
    def _explain(k_codes, v_codes, k_sf, v_sf):
        """Raises for the first thing that is wrong with the tensors."""
        shape = k_codes.shape
        if len(shape) != 4:
            raise ValueError("k_codes must be [num_pages, kv_heads, page_size, head_dim]")
        _require(k_codes, "k_codes", _U8)
        _require(v_codes, "v_codes", _U8, shape)
        _require(k_sf, "k_sf", (torch.uint8,), shape[:2])
        _require(v_sf, "v_sf", (torch.uint8,), shape[:2])
        raise ValueError("the cache's tensors must be on one GPU")

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, page_size: int = 64, head_dim: int = 128, device="cuda") -> "KVCache":
        """A cache with unwritten pages (any bytes)."""
        codes = [torch.empty((num_pages, kv_heads, page_size, head_dim), dtype=torch.uint8, device=device)
                 for _ in range(2)]
        sf = [torch.empty((num_pages, kv_heads), dtype=torch.uint8, device=device) for _ in range(2)]
        return cls(*codes, *sf)


def _unit_columns(t: torch.Tensor) -> bool:
    """Whether a 2-D tensor's rows are contiguous (one column is, whatever its stride says)."""
    return t.stride(1) == 1 or t.shape[1] == 1


def _kv_batch(cache: KVCache, rows: int, block_table, row_start, kv_len) -> _KVBatchStruct:
    seqs = kv_len.shape[0]
    shape, device = block_table.shape, cache.device
    if not (len(shape) == 2 and shape[0] == seqs and _unit_columns(block_table) and row_start.shape == (seqs + 1,)
            and kv_len.dim() == 1 and block_table.dtype is row_start.dtype is kv_len.dtype is torch.int32
            and device == block_table.device == row_start.device == kv_len.device and row_start.is_contiguous()
            and kv_len.is_contiguous()):
        if len(shape) != 2 or shape[0] != seqs or not _unit_columns(block_table):
            raise ValueError("block_table must be [num_seqs, max_pages] with unit column stride")
        _require(block_table, "block_table", (torch.int32,), contiguous=False)
        _require(row_start, "row_start", (torch.int32,), (seqs + 1,))
        _require(kv_len, "kv_len", (torch.int32,), (seqs,))
        raise ValueError("block_table, row_start and kv_len must be on the cache's GPU")
    pages = shape[1]
    ld = block_table.stride(0) if seqs > 1 else pages
    return _KVBatchStruct(block_table.data_ptr(), ld, pages, row_start.data_ptr(), kv_len.data_ptr(), seqs, rows)


def _kv_rows(t: torch.Tensor, name: str, cache: KVCache, rows: int, heads: int) -> int:
    """Checks a BF16 [rows, heads, head_dim] tensor whose rows are contiguous
    and returns its row stride in elements."""
    D = cache.head_dim
    if t.dtype is not torch.bfloat16 or t.device != cache.device:
        raise ValueError(f"{name} must be a bfloat16 tensor on the cache's GPU")
    if t.shape != (rows, heads, D):
        raise ValueError(f"{name} must have shape {(rows, heads, D)}, got {tuple(t.shape)}")
    ld, inner, unit = t.stride()
    if unit != 1 or (heads > 1 and inner != D):
        raise ValueError(f"the heads of one row of {name} must be contiguous")
    return ld if rows > 1 else heads * D


def _kv_stream(cache: KVCache, stream) -> int:
    """The raw stream of a call: the given one, or PyTorch's current stream.  The
    kernels run on the current GPU, so the cache has to lie there."""
    if torch._C._cuda_getDevice() != cache.device.index:
        raise ValueError(f"the cache is on {cache.device}, which is not the current GPU")
    return torch._C._cuda_getCurrentRawStream(cache.device.index) if stream is None else _stream(stream)


def _kv_empty(shape, dtype, cache: KVCache, stream) -> torch.Tensor:
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=cache.device)
    with _on_stream(stream):
        return torch.empty(shape, dtype=dtype, device=cache.device)


def _on_stream(stream):
    """The context in which to allocate what a call on `stream` uses, so that
    the allocator orders its reuse after that stream's work."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def kv_cache_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor,
                   row_start: torch.Tensor, kv_len: torch.Tensor, *, stream=None) -> None:
    """Quantises the newest tokens' rows into their pages (include/iq.h,
    iq_kv_cache_write): k, v bfloat16 [T, kv_heads, head_dim] (the row stride
    may be larger); block_table int32 [B, max_pages], row_start int32 [B + 1],
    kv_len int32 [B] (lengths with these rows)."""
    rows = k.shape[0]
    batch = _kv_batch(cache, rows, block_table, row_start, kv_len)
    ldk = _kv_rows(k, "k", cache, rows, cache.kv_heads)
    ldv = _kv_rows(v, "v", cache, rows, cache.kv_heads)
    _check(lib().iq_kv_cache_write(ctypes.byref(cache._struct), ctypes.byref(batch), k.data_ptr(), ldk, v.data_ptr(),
                                   ldv, _kv_stream(cache, stream)), "iq_kv_cache_write")


def kv_cache_read(cache: KVCache, rows: int, block_table: torch.Tensor, row_start: torch.Tensor,
                  kv_len: torch.Tensor, *, k: torch.Tensor | None = None, v: torch.Tensor | None = None, stream=None):
    """The batch's `rows` = row_start[-1] newest tokens as bfloat16
    (k, v) [rows, kv_heads, head_dim] (include/iq.h, iq_kv_cache_read)."""
    batch = _kv_batch(cache, rows, block_table, row_start, kv_len)
    shape = (rows, cache.kv_heads, cache.head_dim)
    ldk = ldv = cache.kv_heads * cache.head_dim
    if k is None:
        k = _kv_empty(shape, torch.bfloat16, cache, stream)
    else:
        ldk = _kv_rows(k, "k", cache, rows, cache.kv_heads)
    if v is None:
        v = _kv_empty(shape, torch.bfloat16, cache, stream)
    else:
        ldv = _kv_rows(v, "v", cache, rows, cache.kv_heads)
    _check(lib().iq_kv_cache_read(ctypes.byref(cache._struct), ctypes.byref(batch), k.data_ptr(), ldk, v.data_ptr(),
                                  ldv, _kv_stream(cache, stream)), "iq_kv_cache_read")
    return k, v


@functools.lru_cache(maxsize=256)
def kv_attention_workspace_bytes(rows: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().iq_kv_attention_workspace(rows, q_heads, kv_heads, head_dim))


def _on_cache_gpu(t: torch.Tensor, name: str, cache: KVCache) -> None:
    if t.device != cache.device:
        raise ValueError(f"{name} must be on the cache's GPU")


def _kv_indices(indices: torch.Tensor, cache: KVCache, rows: int) -> tuple[int, int]:
    """Checks the lists of a call of `rows` rows; their length and row stride."""
    if indices.dim() != 2 or indices.shape[0] != rows or not _unit_columns(indices):
        raise ValueError("indices must be [rows, k] with unit column stride")
    _require(indices, "indices", (torch.int32,), contiguous=False)
    _on_cache_gpu(indices, "indices", cache)
    return indices.shape[1], indices.stride(0) if rows > 1 else indices.shape[1]


def _kv_attention(cache, q, indices, block_table, row_start, kv_len, scale, out, workspace, stream):
    if q.dim() != 3:
        raise ValueError("q must be [rows, q_heads, head_dim]")
    rows, heads, _ = q.shape
    batch = _kv_batch(cache, rows, block_table, row_start, kv_len)
    ldq = _kv_rows(q, "q", cache, rows, heads)
    L = lib()
    need = kv_attention_workspace_bytes(rows, heads, cache.kv_heads, cache.head_dim)
    if out is None:
        out, ldo = _kv_empty((rows, heads, cache.head_dim), torch.bfloat16, cache, stream), heads * cache.head_dim
    else:
        ldo = _kv_rows(out, "out", cache, rows, heads)
    if workspace is None:
        workspace = _kv_empty(max(need, 1), torch.uint8, cache, stream)
    else:
        _require(workspace, "workspace", (torch.uint8,))
        _on_cache_gpu(workspace, "workspace", cache)
    scale = cache.head_dim ** -0.5 if scale is None else scale
    args = (ctypes.byref(cache._struct), ctypes.byref(batch), q.data_ptr(), ldq, heads)
    tail = (scale, out.data_ptr(), ldo, workspace.data_ptr(), workspace.numel(), _kv_stream(cache, stream))
    if indices is None:
        _check(L.iq_kv_attention(*args, *tail), "iq_kv_attention")
        return out
    k, ld_idx = _kv_indices(indices, cache, rows)
    _check(L.iq_kv_attention_topk(*args, indices.data_ptr(), ld_idx, k, *tail), "iq_kv_attention_topk")
    return out


def kv_attention(cache: KVCache, q: torch.Tensor, block_table: torch.Tensor, row_start: torch.Tensor,
                 kv_len: torch.Tensor, *, scale: float | None = None, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of the newest tokens' queries over the cache
    (include/iq.h, iq_kv_attention): q bfloat16 [T, q_heads, head_dim] (the row
    stride may be larger) -> bfloat16 of the same shape.  scale defaults to
    1 / sqrt(head_dim)."""
    return _kv_attention(cache, q, None, block_table, row_start, kv_len, scale, out, workspace, stream)


def kv_attention_topk(cache: KVCache, q: torch.Tensor, indices: torch.Tensor, block_table: torch.Tensor,
                      row_start: torch.Tensor, kv_len: torch.Tensor, *, scale: float | None = None,
                      out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """Attention over selected keys (include/iq.h, iq_kv_attention_topk):
    indices int32 [T, k] positions per row, -1 where there is none, as
    indexer_topk returns them."""
    return _kv_attention(cache, q, indices, block_table, row_start, kv_len, scale, out, workspace, stream)
