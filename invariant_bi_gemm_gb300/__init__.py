"""Python binding of the batch-invariant operators (libbi_gemm.so, C ABI in include/bi_gemm.h,
bi_rmsnorm.h, bi_prenorm.h, bi_qkrope.h, bi_prompt.h, bi_attention.h, bi_fp4.h and bi_attention4.h).

Argument marshalling only: every step of y = x·W (and of the other operators) runs in the CUDA kernels of
``csrc/``.  PyTorch supplies device memory and streams.  There is no CPU or
PyTorch fallback: importing this module fails if the library has not been built
(``python -m invariant_bi_gemm_gb300.build``), and every call that the library
refuses raises ``BiGemmError``.

Low-level functions carry the C names (``bi_gemm_create``, ``bi_gemm_run``, ...,
``bi_rmsnorm_run``) and take raw device pointers; ``BiGemm``, ``BiRmsNorm``, ``BiPreNorm`` and,
around one paged KV cache, ``BiQkRope`` (norm, rotation, append), ``BiPromptAttention`` and
``BiAttention`` (single tokens; ``run_shared`` for tokens behind a common prefix) wrap them for
torch tensors, and so do, in 4 bits, ``BiQuant4`` and ``BiGemm4`` (matrices), ``BiQkRope.run4`` and
``BiAttention4`` (the cache).  Their calls run on `stream` (a torch stream or a cudaStream_t value; the current
stream for None); an output that a call makes itself is memory of that stream, and work of another one
on it is ordered by the caller.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

BI_BF16_OUT_BF16 = 0
BI_BF16_OUT_F32 = 1
BI_MXFP8E4M3_OUT_BF16 = 2
BI_SCALES_NONE = 0
BI_SCALES_E8M0_K32 = 1
BI_GEMM_FLAG_STATIC_W = 1
BI_MXFP4 = 0
BI_NVFP4 = 1

BI_GEMM_OK = 0
BI_GEMM_ERR_INVALID_ARG = -1
BI_GEMM_ERR_UNSUPPORTED = -2
BI_GEMM_ERR_ALIGNMENT = -3
BI_GEMM_ERR_CUDA = -4
BI_GEMM_ERR_OOM = -5
BI_GEMM_ERR_TIMEOUT = -6
BI_GEMM_ERR_SCRATCH_LIMIT = -7

# every symbol include/bi_gemm.h declares
EXPORTED_SYMBOLS = (
    "bi_gemm_create", "bi_gemm_create_ex", "bi_gemm_run", "bi_gemm_get_device_error",
    "bi_gemm_destroy", "bi_gemm_get_config", "bi_gemm_workspace_size", "bi_gemm_strerror",
    "bi_gemm_version", "bi_gemm_run_noalloc", "bi_gemm_run_gathered",
)
# every symbol include/bi_rmsnorm.h declares
RMSNORM_EXPORTED_SYMBOLS = ("bi_rmsnorm_create", "bi_rmsnorm_run", "bi_rmsnorm_get_config", "bi_rmsnorm_destroy")
# every symbol include/bi_prenorm.h declares
PRENORM_EXPORTED_SYMBOLS = ("bi_prenorm_create", "bi_prenorm_run", "bi_prenorm_get_config", "bi_prenorm_destroy")
# every symbol include/bi_prompt.h declares
PROMPT_EXPORTED_SYMBOLS = ("bi_prompt_create", "bi_prompt_run", "bi_prompt_workspace_size",
                           "bi_prompt_get_device_error", "bi_prompt_get_config", "bi_prompt_destroy")
# every symbol include/bi_qkrope.h declares
QKROPE_EXPORTED_SYMBOLS = ("bi_qkrope_create", "bi_qkrope_run", "bi_qkrope_get_device_error", "bi_qkrope_get_config",
                           "bi_qkrope_destroy", "bi_qkrope_run4")
# every symbol include/bi_attention.h declares
ATTENTION_EXPORTED_SYMBOLS = ("bi_attention_create", "bi_attention_run", "bi_attention_workspace_size",
                              "bi_attention_get_device_error", "bi_attention_get_config", "bi_attention_destroy",
                              "bi_attention_run_shared", "bi_attention_shared_workspace_size")
# every symbol include/bi_fp4.h declares
FP4_EXPORTED_SYMBOLS = ("bi_quant4_create", "bi_quant4_scale_bytes", "bi_quant4_run", "bi_quant4_expand",
                        "bi_quant4_get_config", "bi_quant4_destroy", "bi_gemm4_create", "bi_gemm4_run",
                        "bi_gemm4_get_device_error", "bi_gemm4_get_config", "bi_gemm4_destroy")

# every symbol include/bi_attention4.h declares
ATTENTION4_EXPORTED_SYMBOLS = ("bi_attention4_create", "bi_attention4_run", "bi_attention4_workspace_size",
                               "bi_attention4_expand", "bi_attention4_get_device_error", "bi_attention4_get_config",
                               "bi_attention4_destroy")


class BiGemmError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {bi_gemm_strerror(code)} ({code})")


class bi_gemm_scales(ctypes.Structure):
    _fields_ = [("sx", ctypes.c_void_p), ("sw", ctypes.c_void_p)]


class bi_gemm_block(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("sx", ctypes.c_void_p), ("rows", ctypes.c_int64)]


class bi_gemm_options(ctypes.Structure):
    _fields_ = [("split_k", ctypes.c_int32), ("max_ctas", ctypes.c_int32), ("timeout_ns", ctypes.c_uint64),
                ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class bi_gemm_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "block_m", "block_n", "block_k", "mma_m", "mma_n", "mma_k", "stages", "split_k",
        "num_sms", "max_ctas", "threads", "smem_bytes", "tmem_cols", "ctas_per_tile", "max_groups")]


class bi_rmsnorm_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("d", "threads", "vectors_per_thread", "max_ctas", "num_sms")]


class bi_attention_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_q_heads", "num_kv_heads", "head_dim", "page_size", "split_size",
                                              "threads", "stage_positions", "max_ctas", "num_sms", "tma_pages",
                                              "ring_stages")]


class bi_qkrope_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_q_heads", "num_kv_heads", "head_dim", "page_size", "rot_dim",
                                              "interleaved", "threads", "tokens_per_block", "ring_tokens", "ring_ctas",
                                              "ring_from")]


class bi_prompt_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_q_heads", "num_kv_heads", "head_dim", "page_size", "tile_positions",
                                              "block_positions", "stages", "threads", "max_ctas", "tma_pages")]


class bi_prenorm_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("K", "N", "chunk", "splits", "tile_rows")]


class bi_quant4_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("K", "format", "block", "threads")]


class bi_gemm4_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("K", "N", "format", "out_f32", "tile_rows", "tile_cols", "stages",
                                              "max_groups", "few_rows", "smem_bytes")]


class bi_attention4_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_q_heads", "num_kv_heads", "head_dim", "page_size", "split_size",
                                              "threads", "max_ctas", "tokens_per_launch")]


def _load() -> ctypes.CDLL:
    path = _build.lib_path("libbi_gemm.so")
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: the CUDA library has not been built "
            "(run `python -m invariant_bi_gemm_gb300.build`); there is no fallback path")
    L = ctypes.CDLL(path)
    P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.bi_gemm_create.argtypes = [ctypes.POINTER(P), I64, I64, I32, I32]
    L.bi_gemm_create_ex.argtypes = [ctypes.POINTER(P), I64, I64, I32, I32, ctypes.POINTER(bi_gemm_options)]
    L.bi_gemm_run.argtypes = [P, P, I64, P, ctypes.POINTER(bi_gemm_scales), P, P]
    L.bi_gemm_run_noalloc.argtypes = [P, P, I64, P, ctypes.POINTER(bi_gemm_scales), P, P]
    L.bi_gemm_run_gathered.argtypes = [P, ctypes.POINTER(bi_gemm_block), ctypes.c_int32, P, P, P, P, P, P]
    L.bi_gemm_get_device_error.argtypes = [P, P]
    L.bi_gemm_destroy.argtypes = [P]
    L.bi_gemm_get_config.argtypes = [P, ctypes.POINTER(bi_gemm_config)]
    L.bi_gemm_workspace_size.argtypes = [P, I64, ctypes.POINTER(ctypes.c_uint64)]
    L.bi_gemm_strerror.argtypes = [I32]
    L.bi_gemm_strerror.restype = ctypes.c_char_p
    L.bi_gemm_version.argtypes = []
    L.bi_rmsnorm_create.argtypes = [ctypes.POINTER(P), I64, ctypes.c_float]
    L.bi_rmsnorm_run.argtypes = [P, P, I64, P, P, P]
    L.bi_rmsnorm_get_config.argtypes = [P, ctypes.POINTER(bi_rmsnorm_config)]
    L.bi_rmsnorm_destroy.argtypes = [P]
    L.bi_attention_create.argtypes = [ctypes.POINTER(P), I64, I64, I64, I64, ctypes.c_float, I64]
    L.bi_attention_run.argtypes = [P, P, I64, P, P, P, P, I64, P, I64, I64, I64, P, P]
    L.bi_attention_workspace_size.argtypes = [P, I64, I64, ctypes.POINTER(ctypes.c_uint64)]
    L.bi_attention_run_shared.argtypes = [P, P, I64, P, P, P, P, I64, P, I64, I64, I64, P, P, I64, P, P]
    L.bi_attention_shared_workspace_size.argtypes = [P, I64, I64, I64, ctypes.POINTER(ctypes.c_uint64)]
    L.bi_attention_get_device_error.argtypes = [P, P]
    L.bi_attention_get_config.argtypes = [P, ctypes.POINTER(bi_attention_config)]
    L.bi_attention_destroy.argtypes = [P]
    L.bi_prenorm_create.argtypes = [ctypes.POINTER(P), I64, I64, ctypes.c_float, I64]
    L.bi_prenorm_run.argtypes = [P, P, I64, P, P, P]
    L.bi_prenorm_get_config.argtypes = [P, ctypes.POINTER(bi_prenorm_config)]
    L.bi_prenorm_destroy.argtypes = [P]
    L.bi_qkrope_create.argtypes = [ctypes.POINTER(P), I64, I64, I64, I64, I64, ctypes.c_int32, ctypes.c_float]
    L.bi_qkrope_run.argtypes = [P, P, I64, I64, P, P, P, I64, P, P, P, P, I64, P, I64, I64, P, P]
    L.bi_qkrope_get_device_error.argtypes = [P, P]
    L.bi_qkrope_get_config.argtypes = [P, ctypes.POINTER(bi_qkrope_config)]
    L.bi_qkrope_destroy.argtypes = [P]
    L.bi_prompt_create.argtypes = [ctypes.POINTER(P), I64, I64, I64, I64, ctypes.c_float]
    L.bi_prompt_run.argtypes = [P, P, I64, P, P, I64, P, P, I64, P, I64, I64, P, P]
    L.bi_prompt_workspace_size.argtypes = [P, I64, I64, ctypes.POINTER(ctypes.c_uint64)]
    L.bi_prompt_get_device_error.argtypes = [P, P]
    L.bi_prompt_get_config.argtypes = [P, ctypes.POINTER(bi_prompt_config)]
    L.bi_prompt_destroy.argtypes = [P]
    L.bi_quant4_create.argtypes = [ctypes.POINTER(P), I64, ctypes.c_int32, ctypes.c_float]
    L.bi_quant4_scale_bytes.argtypes = [P, I64, ctypes.POINTER(ctypes.c_uint64)]
    L.bi_quant4_run.argtypes = [P, P, I64, I64, P, P, P]
    L.bi_quant4_expand.argtypes = [P, P, P, I64, P, P]
    L.bi_quant4_get_config.argtypes = [P, ctypes.POINTER(bi_quant4_config)]
    L.bi_quant4_destroy.argtypes = [P]
    L.bi_gemm4_create.argtypes = [ctypes.POINTER(P), I64, I64, ctypes.c_int32, ctypes.c_int32]
    L.bi_gemm4_run.argtypes = [P, P, P, I64, P, P, ctypes.c_float, P, P]
    L.bi_gemm4_get_device_error.argtypes = [P, P]
    L.bi_gemm4_get_config.argtypes = [P, ctypes.POINTER(bi_gemm4_config)]
    L.bi_gemm4_destroy.argtypes = [P]
    F = ctypes.c_float
    L.bi_qkrope_run4.argtypes = [P, P, I64, I64, P, P, P, I64, P, P, P, P, P, P, F, F, I64, P, I64, I64, P, P]
    L.bi_attention4_create.argtypes = [ctypes.POINTER(P), I64, I64, I64, I64, F, F, F, I64]
    L.bi_attention4_run.argtypes = [P, P, I64, P, P, P, P, P, P, I64, P, I64, I64, I64, P, P]
    L.bi_attention4_workspace_size.argtypes = [P, I64, I64, ctypes.POINTER(ctypes.c_uint64)]
    L.bi_attention4_expand.argtypes = [P, P, P, P, P, I64, P, I64, P, P, P]
    L.bi_attention4_get_device_error.argtypes = [P, P]
    L.bi_attention4_get_config.argtypes = [P, ctypes.POINTER(bi_attention4_config)]
    L.bi_attention4_destroy.argtypes = [P]
    for n in ("bi_gemm_create", "bi_gemm_create_ex", "bi_gemm_run", "bi_gemm_run_noalloc", "bi_gemm_run_gathered",
              "bi_gemm_get_device_error",
              "bi_gemm_destroy", "bi_gemm_get_config", "bi_gemm_workspace_size", "bi_gemm_version") + \
            RMSNORM_EXPORTED_SYMBOLS + ATTENTION_EXPORTED_SYMBOLS + PRENORM_EXPORTED_SYMBOLS + QKROPE_EXPORTED_SYMBOLS + \
            PROMPT_EXPORTED_SYMBOLS + FP4_EXPORTED_SYMBOLS + ATTENTION4_EXPORTED_SYMBOLS:
        getattr(L, n).restype = I32
    return L


_lib = None
LIB_PATH = _build.lib_path("libbi_gemm.so")


def library() -> ctypes.CDLL:
    """The loaded libbi_gemm.so (loaded on first use; ImportError if it was never built)."""
    global _lib
    if _lib is None:
        _lib = _load()
    return _lib


def _check(rc: int, where: str) -> None:
    if rc != BI_GEMM_OK:
        raise BiGemmError(rc, where)


def _new_output(make, stream, device):
    """An output that a call on `stream` makes itself.  Its memory comes from that stream's pool: a
    block of the current stream's may still be in use by work queued there.  The current stream counts as a
    user of it, so that it is not given out again before what is queued there when it is dropped is over
    (ordering that work behind the call is the caller's, as with any other stream)."""
    if stream is None:
        return make()
    import torch
    current = torch.cuda.current_stream(device)
    if not hasattr(stream, "cuda_stream"):
        number = int(stream)                    # 0 and 1 are names of the default stream
        stream = torch.cuda.default_stream(device) if number in (0, 1) else torch.cuda.ExternalStream(number, device)
    if stream.cuda_stream == current.cuda_stream:
        return make()
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(current)
    return t


# --------------------------------------------------------------------- C names

def bi_gemm_strerror(code: int) -> str:
    return library().bi_gemm_strerror(int(code)).decode()


def bi_gemm_version() -> int:
    return library().bi_gemm_version()


def bi_gemm_create(K: int, N: int, dtype: int, scale_layout: int = BI_SCALES_NONE,
                   options: bi_gemm_options | None = None) -> int:
    """Returns the handle (an opaque integer); raises BiGemmError on refusal."""
    h = ctypes.c_void_p()
    if options is None:
        rc = library().bi_gemm_create(ctypes.byref(h), int(K), int(N), int(dtype), int(scale_layout))
    else:
        rc = library().bi_gemm_create_ex(ctypes.byref(h), int(K), int(N), int(dtype), int(scale_layout),
                                   ctypes.byref(options))
    _check(rc, "bi_gemm_create")
    return h.value


def bi_gemm_run(h: int, x: int, M: int, W: int, scales: bi_gemm_scales | None, y: int, stream: int) -> None:
    """Raw-pointer call: x, W, y device addresses, stream a cudaStream_t value."""
    rc = library().bi_gemm_run(ctypes.c_void_p(h), ctypes.c_void_p(x), int(M), ctypes.c_void_p(W),
                         ctypes.byref(scales) if scales is not None else None, ctypes.c_void_p(y),
                         ctypes.c_void_p(stream))
    _check(rc, "bi_gemm_run")


def bi_gemm_run_noalloc(h: int, x: int, M: int, W: int, scales: bi_gemm_scales | None, y: int,
                        stream: int) -> None:
    """bi_gemm_run for callers that may not allocate device memory: a split count > 1 keeps its
    scratch in the library's fixed 8 MiB per-device array; too large a run raises
    BiGemmError(BI_GEMM_ERR_SCRATCH_LIMIT).  Calls that overlap on the GPU race on that array."""
    rc = library().bi_gemm_run_noalloc(ctypes.c_void_p(h), ctypes.c_void_p(x), int(M), ctypes.c_void_p(W),
                                       ctypes.byref(scales) if scales is not None else None, ctypes.c_void_p(y),
                                       ctypes.c_void_p(stream))
    _check(rc, "bi_gemm_run_noalloc")


def bi_gemm_get_device_error(h: int, stream: int = 0) -> int:
    return library().bi_gemm_get_device_error(ctypes.c_void_p(h), ctypes.c_void_p(stream))


def bi_gemm_destroy(h: int) -> None:
    _check(library().bi_gemm_destroy(ctypes.c_void_p(h)), "bi_gemm_destroy")


def bi_gemm_get_config(h: int) -> dict:
    c = bi_gemm_config()
    _check(library().bi_gemm_get_config(ctypes.c_void_p(h), ctypes.byref(c)), "bi_gemm_get_config")
    return {n: getattr(c, n) for n, _ in bi_gemm_config._fields_}


def bi_gemm_workspace_size(h: int, M: int) -> int:
    b = ctypes.c_uint64()
    _check(library().bi_gemm_workspace_size(ctypes.c_void_p(h), int(M), ctypes.byref(b)), "bi_gemm_workspace_size")
    return b.value


def bi_rmsnorm_create(d: int, eps: float) -> int:
    """Returns the handle (an opaque integer); raises BiGemmError on refusal."""
    h = ctypes.c_void_p()
    _check(library().bi_rmsnorm_create(ctypes.byref(h), int(d), float(eps)), "bi_rmsnorm_create")
    return h.value


def bi_rmsnorm_run(h: int, x: int, M: int, g: int, y: int, stream: int) -> None:
    """Raw-pointer call: x, g, y device addresses, stream a cudaStream_t value."""
    rc = library().bi_rmsnorm_run(ctypes.c_void_p(h), ctypes.c_void_p(x), int(M), ctypes.c_void_p(g),
                                  ctypes.c_void_p(y), ctypes.c_void_p(stream))
    _check(rc, "bi_rmsnorm_run")


def bi_rmsnorm_get_config(h: int) -> dict:
    c = bi_rmsnorm_config()
    _check(library().bi_rmsnorm_get_config(ctypes.c_void_p(h), ctypes.byref(c)), "bi_rmsnorm_get_config")
    return {n: getattr(c, n) for n, _ in bi_rmsnorm_config._fields_}


def bi_rmsnorm_destroy(h: int) -> None:
    _check(library().bi_rmsnorm_destroy(ctypes.c_void_p(h)), "bi_rmsnorm_destroy")


def bi_attention_create(num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int, scale: float,
                        split_size: int = 0) -> int:
    """Returns the handle (an opaque integer); raises BiGemmError on refusal."""
    h = ctypes.c_void_p()
    _check(library().bi_attention_create(ctypes.byref(h), int(num_q_heads), int(num_kv_heads), int(head_dim),
                                         int(page_size), float(scale), int(split_size)), "bi_attention_create")
    return h.value


def bi_attention_run(h: int, q: int, T: int, q_seq: int, q_pos: int, k_cache: int, v_cache: int, num_pages: int,
                     page_table: int, num_seqs: int, max_pages: int, max_pos: int, o: int, stream: int) -> None:
    """Raw-pointer call (device addresses, stream a cudaStream_t value)."""
    V = ctypes.c_void_p
    rc = library().bi_attention_run(V(h), V(q), int(T), V(q_seq), V(q_pos), V(k_cache), V(v_cache), int(num_pages),
                                     V(page_table), int(num_seqs), int(max_pages), int(max_pos), V(o), V(stream))
    _check(rc, "bi_attention_run")


def bi_attention_run_shared(h: int, q: int, T: int, q_seq: int, q_pos: int, k_cache: int, v_cache: int,
                            num_pages: int, page_table: int, num_seqs: int, max_pages: int, max_pos: int,
                            group_start: int, group_len: int, num_groups: int, o: int, stream: int) -> None:
    """Raw-pointer call (device addresses, stream a cudaStream_t value)."""
    _check(library().bi_attention_run_shared(h, q, T, q_seq, q_pos, k_cache, v_cache, num_pages, page_table, num_seqs,
                                             max_pages, max_pos, group_start, group_len, num_groups, o, stream),
           "bi_attention_run_shared")


def bi_attention_shared_workspace_size(h: int, T: int, max_pos: int, num_groups: int) -> int:
    b = ctypes.c_uint64()
    _check(library().bi_attention_shared_workspace_size(ctypes.c_void_p(h), int(T), int(max_pos), int(num_groups),
                                                        ctypes.byref(b)), "bi_attention_shared_workspace_size")
    return b.value


def bi_attention_get_config(h: int) -> dict:
    c = bi_attention_config()
    _check(library().bi_attention_get_config(ctypes.c_void_p(h), ctypes.byref(c)), "bi_attention_get_config")
    return {n: getattr(c, n) for n, _ in bi_attention_config._fields_}


def bi_attention_workspace_size(h: int, T: int, max_pos: int) -> int:
    b = ctypes.c_uint64()
    _check(library().bi_attention_workspace_size(ctypes.c_void_p(h), int(T), int(max_pos), ctypes.byref(b)),
           "bi_attention_workspace_size")
    return b.value


def bi_attention_get_device_error(h: int, stream: int = 0) -> int:
    return library().bi_attention_get_device_error(ctypes.c_void_p(h), ctypes.c_void_p(stream))


def bi_attention_destroy(h: int) -> None:
    _check(library().bi_attention_destroy(ctypes.c_void_p(h)), "bi_attention_destroy")


def bi_qkrope_create(num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int, rot_dim: int,
                     interleaved: bool, eps: float) -> int:
    """Returns the handle (an opaque integer); raises BiGemmError on refusal."""
    h = ctypes.c_void_p()
    _check(library().bi_qkrope_create(ctypes.byref(h), int(num_q_heads), int(num_kv_heads), int(head_dim),
                                      int(page_size), int(rot_dim), int(bool(interleaved)), float(eps)),
           "bi_qkrope_create")
    return h.value


def bi_qkrope_run(h: int, qkv: int, T: int, qkv_stride: int, gq: int | None, gk: int | None, cos_sin: int,
                  num_positions: int, q_seq: int, q_pos: int, k_cache: int, v_cache: int, num_pages: int,
                  page_table: int, num_seqs: int, max_pages: int, q_out: int, stream: int) -> None:
    """Raw-pointer call (device addresses, stream a cudaStream_t value)."""
    V = ctypes.c_void_p
    rc = library().bi_qkrope_run(V(h), V(qkv), int(T), int(qkv_stride), V(gq), V(gk), V(cos_sin), int(num_positions),
                                 V(q_seq), V(q_pos), V(k_cache), V(v_cache), int(num_pages), V(page_table),
                                 int(num_seqs), int(max_pages), V(q_out), V(stream))
    _check(rc, "bi_qkrope_run")


def bi_qkrope_run4(h: int, qkv: int, T: int, qkv_stride: int, gq: int | None, gk: int | None, cos_sin: int,
                   num_positions: int, q_seq: int, q_pos: int, k_codes: int, k_scales: int, v_codes: int, v_scales: int,
                   k_scale: float, v_scale: float, num_pages: int, page_table: int, num_seqs: int, max_pages: int,
                   q_out: int, stream: int) -> None:
    """Raw-pointer call (device addresses, stream a cudaStream_t value)."""
    _check(library().bi_qkrope_run4(h, qkv, T, qkv_stride, gq, gk, cos_sin, num_positions, q_seq, q_pos, k_codes, k_scales,
                                    v_codes, v_scales, k_scale, v_scale, num_pages, page_table, num_seqs, max_pages,
                                    q_out, stream), "bi_qkrope_run4")


def bi_qkrope_get_device_error(h: int, stream: int = 0) -> int:
    return library().bi_qkrope_get_device_error(ctypes.c_void_p(h), ctypes.c_void_p(stream))


def bi_qkrope_get_config(h: int) -> dict:
    c = bi_qkrope_config()
    _check(library().bi_qkrope_get_config(ctypes.c_void_p(h), ctypes.byref(c)), "bi_qkrope_get_config")
    return {n: getattr(c, n) for n, _ in bi_qkrope_config._fields_}


def bi_qkrope_destroy(h: int) -> None:
    _check(library().bi_qkrope_destroy(ctypes.c_void_p(h)), "bi_qkrope_destroy")


def bi_prompt_create(num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int, scale: float) -> int:
    """Returns the handle (an opaque integer); raises BiGemmError on refusal."""
    h = ctypes.c_void_p()
    _check(library().bi_prompt_create(ctypes.byref(h), int(num_q_heads), int(num_kv_heads), int(head_dim),
                                      int(page_size), float(scale)), "bi_prompt_create")
    return h.value


def bi_prompt_run(h: int, q: int, T: int, q_start: int, q_pos0: int, num_seqs: int, k_cache: int, v_cache: int,
                  num_pages: int, page_table: int, max_pages: int, max_pos: int, o: int, stream: int) -> None:
    """Raw-pointer call (device addresses, stream a cudaStream_t value)."""
    _check(library().bi_prompt_run(h, q, T, q_start, q_pos0, num_seqs, k_cache, v_cache, num_pages, page_table,
                                   max_pages, max_pos, o, stream), "bi_prompt_run")


def bi_prompt_workspace_size(h: int, T: int, num_seqs: int) -> int:
    b = ctypes.c_uint64()
    _check(library().bi_prompt_workspace_size(ctypes.c_void_p(h), int(T), int(num_seqs), ctypes.byref(b)),
           "bi_prompt_workspace_size")
    return b.value


def bi_prompt_get_device_error(h: int, stream: int = 0) -> int:
    return library().bi_prompt_get_device_error(ctypes.c_void_p(h), ctypes.c_void_p(stream))


def bi_prompt_get_config(h: int) -> dict:
    c = bi_prompt_config()
    _check(library().bi_prompt_get_config(ctypes.c_void_p(h), ctypes.byref(c)), "bi_prompt_get_config")
    return {n: getattr(c, n) for n, _ in bi_prompt_config._fields_}


def bi_prompt_destroy(h: int) -> None:
    _check(library().bi_prompt_destroy(ctypes.c_void_p(h)), "bi_prompt_destroy")


def bi_prenorm_create(K: int, N: int, eps: float, chunk: int = 0) -> int:
    """Returns the handle (an opaque integer); raises BiGemmError on refusal."""
    h = ctypes.c_void_p()
    _check(library().bi_prenorm_create(ctypes.byref(h), int(K), int(N), float(eps), int(chunk)), "bi_prenorm_create")
    return h.value


def bi_prenorm_run(h: int, x: int, M: int, W: int, y: int, stream: int) -> None:
    """Raw-pointer call: x, W, y device addresses, stream a cudaStream_t value."""
    V = ctypes.c_void_p
    _check(library().bi_prenorm_run(V(h), V(x), int(M), V(W), V(y), V(stream)), "bi_prenorm_run")


def bi_prenorm_get_config(h: int) -> dict:
    c = bi_prenorm_config()
    _check(library().bi_prenorm_get_config(ctypes.c_void_p(h), ctypes.byref(c)), "bi_prenorm_get_config")
    return {n: getattr(c, n) for n, _ in bi_prenorm_config._fields_}


def bi_prenorm_destroy(h: int) -> None:
    _check(library().bi_prenorm_destroy(ctypes.c_void_p(h)), "bi_prenorm_destroy")


def bi_attention4_create(num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int, scale: float,
                         k_scale: float = 1.0, v_scale: float = 1.0, split_size: int = 0) -> int:
    """Returns the handle (an opaque integer); raises BiGemmError on refusal."""
    h = ctypes.c_void_p()
    _check(library().bi_attention4_create(ctypes.byref(h), int(num_q_heads), int(num_kv_heads), int(head_dim),
                                          int(page_size), float(scale), float(k_scale), float(v_scale),
                                          int(split_size)), "bi_attention4_create")
    return h.value


def bi_attention4_run(h: int, q: int, T: int, q_seq: int, q_pos: int, k_codes: int, k_scales: int, v_codes: int,
                      v_scales: int, num_pages: int, page_table: int, num_seqs: int, max_pages: int, max_pos: int,
                      o: int, stream: int) -> None:
    """Raw-pointer call (device addresses, stream a cudaStream_t value)."""
    _check(library().bi_attention4_run(h, q, T, q_seq, q_pos, k_codes, k_scales, v_codes, v_scales, num_pages, page_table,
                                       num_seqs, max_pages, max_pos, o, stream), "bi_attention4_run")


def bi_attention4_workspace_size(h: int, T: int, max_pos: int) -> int:
    b = ctypes.c_uint64()
    _check(library().bi_attention4_workspace_size(ctypes.c_void_p(h), int(T), int(max_pos), ctypes.byref(b)),
           "bi_attention4_workspace_size")
    return b.value


def bi_attention4_expand(h: int, k_codes: int, k_scales: int, v_codes: int, v_scales: int, num_pages: int, pages: int,
                         n: int, k_out: int, v_out: int, stream: int) -> None:
    """Raw-pointer call (device addresses, stream a cudaStream_t value)."""
    _check(library().bi_attention4_expand(h, k_codes, k_scales, v_codes, v_scales, num_pages, pages, n, k_out, v_out,
                                          stream), "bi_attention4_expand")


def bi_attention4_get_device_error(h: int, stream: int = 0) -> int:
    return library().bi_attention4_get_device_error(ctypes.c_void_p(h), ctypes.c_void_p(stream))


def bi_attention4_get_config(h: int) -> dict:
    c = bi_attention4_config()
    _check(library().bi_attention4_get_config(ctypes.c_void_p(h), ctypes.byref(c)), "bi_attention4_get_config")
    return {n: getattr(c, n) for n, _ in bi_attention4_config._fields_}


def bi_attention4_destroy(h: int) -> None:
    _check(library().bi_attention4_destroy(ctypes.c_void_p(h)), "bi_attention4_destroy")


def bi_quant4_create(K: int, format: int, tensor_scale: float = 1.0) -> int:
    """Returns the handle (an opaque integer); raises BiGemmError on refusal."""
    h = ctypes.c_void_p()
    _check(library().bi_quant4_create(ctypes.byref(h), int(K), int(format), float(tensor_scale)), "bi_quant4_create")
    return h.value


def bi_quant4_scale_bytes(h: int, M: int) -> int:
    b = ctypes.c_uint64()
    _check(library().bi_quant4_scale_bytes(ctypes.c_void_p(h), int(M), ctypes.byref(b)), "bi_quant4_scale_bytes")
    return b.value


def bi_quant4_run(h: int, x: int, M: int, x_stride: int, codes: int, scales: int, stream: int) -> None:
    """Raw-pointer call (device addresses, stream a cudaStream_t value)."""
    _check(library().bi_quant4_run(h, x, M, x_stride, codes, scales, stream), "bi_quant4_run")


def bi_quant4_expand(h: int, codes: int, scales: int, M: int, y: int, stream: int) -> None:
    """Raw-pointer call (device addresses, stream a cudaStream_t value)."""
    _check(library().bi_quant4_expand(h, codes, scales, M, y, stream), "bi_quant4_expand")


def bi_quant4_get_config(h: int) -> dict:
    c = bi_quant4_config()
    _check(library().bi_quant4_get_config(ctypes.c_void_p(h), ctypes.byref(c)), "bi_quant4_get_config")
    return {n: getattr(c, n) for n, _ in bi_quant4_config._fields_}


def bi_quant4_destroy(h: int) -> None:
    _check(library().bi_quant4_destroy(ctypes.c_void_p(h)), "bi_quant4_destroy")


def bi_gemm4_create(K: int, N: int, format: int, out_f32: bool = False) -> int:
    """Returns the handle (an opaque integer); raises BiGemmError on refusal."""
    h = ctypes.c_void_p()
    _check(library().bi_gemm4_create(ctypes.byref(h), int(K), int(N), int(format), int(bool(out_f32))),
           "bi_gemm4_create")
    return h.value


def bi_gemm4_run(h: int, x: int, sx: int, M: int, w: int, sw: int, alpha: float, y: int, stream: int) -> None:
    """Raw-pointer call (device addresses, stream a cudaStream_t value)."""
    _check(library().bi_gemm4_run(h, x, sx, M, w, sw, alpha, y, stream), "bi_gemm4_run")


def bi_gemm4_get_device_error(h: int, stream: int = 0) -> int:
    return library().bi_gemm4_get_device_error(ctypes.c_void_p(h), ctypes.c_void_p(stream))


def bi_gemm4_get_config(h: int) -> dict:
    c = bi_gemm4_config()
    _check(library().bi_gemm4_get_config(ctypes.c_void_p(h), ctypes.byref(c)), "bi_gemm4_get_config")
    return {n: getattr(c, n) for n, _ in bi_gemm4_config._fields_}


def bi_gemm4_destroy(h: int) -> None:
    _check(library().bi_gemm4_destroy(ctypes.c_void_p(h)), "bi_gemm4_destroy")


# --------------------------------------------------------------------- torch wrappers

_DTYPES = {"bf16": BI_BF16_OUT_BF16, "bf16_f32": BI_BF16_OUT_F32, "mxfp8": BI_MXFP8E4M3_OUT_BF16}


class BiGemm:
    """y = x·W for fixed (K, N) on torch tensors.

    kind: "bf16" (bf16 in/out), "bf16_f32" (bf16 in, fp32 out) or "mxfp8" (E4M3 codes as
    uint8 / float8_e4m3fn tensors, E8M0 scales as uint8, bf16 out).
    """

    def __init__(self, K: int, N: int, kind: str = "bf16", split_k: int = 0, max_ctas: int = 0,
                 timeout_ns: int = 0, static_w: bool = False):
        self.K, self.N, self.kind = int(K), int(N), kind
        self.dtype = _DTYPES[kind]
        layout = BI_SCALES_E8M0_K32 if kind == "mxfp8" else BI_SCALES_NONE
        opts = None
        flags = BI_GEMM_FLAG_STATIC_W if static_w else 0
        if split_k or max_ctas or timeout_ns or flags:
            opts = bi_gemm_options(int(split_k), int(max_ctas), int(timeout_ns), flags, 0)
        self.handle = bi_gemm_create(self.K, self.N, self.dtype, layout, opts)

    @property
    def config(self) -> dict:
        return bi_gemm_get_config(self.handle)

    def out_dtype(self):
        import torch
        return torch.float32 if self.kind == "bf16_f32" else torch.bfloat16

    def run(self, x, W, y=None, sx=None, sw=None, stream=None):
        import torch
        M = int(x.shape[0])
        if x.dim() != 2 or x.shape[1] != self.K or tuple(W.shape) != (self.K, self.N):
            raise ValueError("shape mismatch: x [M, K], W [K, N] expected")
        if not (x.is_cuda and W.is_cuda and x.is_contiguous() and W.is_contiguous()):
            raise ValueError("x and W must be contiguous CUDA tensors")
        want = torch.bfloat16 if self.kind != "mxfp8" else None
        if want is not None and (x.dtype != want or W.dtype != want):
            raise ValueError("bf16 inputs expected")
        if want is None and (x.element_size() != 1 or W.element_size() != 1):
            raise ValueError("E4M3 inputs (1 byte per element) expected")
        if y is None:
            y = _new_output(lambda: torch.empty((M, self.N), dtype=self.out_dtype(), device=x.device), stream, x.device)
        if tuple(y.shape) != (M, self.N) or y.dtype != self.out_dtype() or not y.is_contiguous():
            raise ValueError("y must be a contiguous [M, N] tensor of the output dtype")
        scales = None
        if self.kind == "mxfp8":
            if sx is None or sw is None:
                raise ValueError("MXFP8 needs sx [M, K/32] and sw [K/32, N] E8M0 tensors")
            if tuple(sx.shape) != (M, self.K // 32) or tuple(sw.shape) != (self.K // 32, self.N):
                raise ValueError("scale shapes: sx [M, K/32], sw [K/32, N]")
            if sx.element_size() != 1 or sw.element_size() != 1 or not (sx.is_contiguous() and sw.is_contiguous()):
                raise ValueError("scales must be contiguous uint8 tensors")
            scales = bi_gemm_scales(sx.data_ptr(), sw.data_ptr())
        if stream is None:
            stream = torch.cuda.current_stream(x.device)
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        bi_gemm_run(self.handle, x.data_ptr(), M, W.data_ptr(), scales, y.data_ptr(), s)
        return y

    __call__ = run

    def run_gathered(self, blocks, W, x_out=None, y=None, sx_blocks=None, sx_out=None, sw=None, stream=None):
        """y = concat(blocks) · W through bi_gemm_run_gathered: the row blocks (contiguous [rows, K]
        CUDA tensors, in order; for MXFP8 with their scales sx_blocks) are gathered into x_out
        (and sx_out), then multiplied with the same kernel configuration as every other row.
        Returns (y, x_out, sx_out)."""
        import torch
        nb = len(blocks)
        if nb < 1 or (sx_blocks is not None and len(sx_blocks) != nb):
            raise ValueError("one or more blocks (and one scale block per block for MXFP8)")
        fp8 = self.kind == "mxfp8"
        for b in blocks:
            if b.dim() != 2 or b.shape[1] != self.K or not (b.is_cuda and b.is_contiguous()):
                raise ValueError("blocks must be contiguous [rows, K] CUDA tensors")
        M = sum(int(b.shape[0]) for b in blocks)
        dev = blocks[0].device
        if x_out is None:
            x_out = _new_output(lambda: torch.empty((M, self.K), dtype=blocks[0].dtype, device=dev), stream, dev)
        if fp8:
            if sx_blocks is None or sw is None:
                raise ValueError("MXFP8 needs sx_blocks and sw")
            if sx_out is None:
                sx_out = _new_output(lambda: torch.empty((M, self.K // 32), dtype=torch.uint8, device=dev), stream, dev)
        if y is None:
            y = _new_output(lambda: torch.empty((M, self.N), dtype=self.out_dtype(), device=dev), stream, dev)
        if tuple(x_out.shape) != (M, self.K) or tuple(y.shape) != (M, self.N):
            raise ValueError("x_out [M, K] and y [M, N] expected")
        arr = (bi_gemm_block * nb)()
        for i, b in enumerate(blocks):
            arr[i].x = b.data_ptr()
            arr[i].sx = sx_blocks[i].data_ptr() if fp8 else None
            arr[i].rows = int(b.shape[0])
        if stream is None:
            stream = torch.cuda.current_stream(dev)
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        rc = library().bi_gemm_run_gathered(ctypes.c_void_p(self.handle), arr, nb, ctypes.c_void_p(x_out.data_ptr()),
                                            ctypes.c_void_p(sx_out.data_ptr() if fp8 else None),
                                            ctypes.c_void_p(W.data_ptr()),
                                            ctypes.c_void_p(sw.data_ptr() if fp8 else None),
                                            ctypes.c_void_p(y.data_ptr()), ctypes.c_void_p(s))
        _check(rc, "bi_gemm_run_gathered")
        return y, x_out, sx_out

    def device_error(self, stream=None) -> int:
        s = 0
        if stream is not None:
            s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        return bi_gemm_get_device_error(self.handle, s)

    def workspace_size(self, M: int) -> int:
        return bi_gemm_workspace_size(self.handle, M)

    def close(self) -> None:
        if getattr(self, "handle", None):
            bi_gemm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BiRmsNorm:
    """y = RMSNorm(x) * g over rows of length d on torch bf16 tensors (x [M, d], g [d])."""

    def __init__(self, d: int, eps: float = 1e-6):
        self.d, self.eps = int(d), float(eps)
        self.handle = bi_rmsnorm_create(self.d, self.eps)

    @property
    def config(self) -> dict:
        return bi_rmsnorm_get_config(self.handle)

    def run(self, x, g, y=None, stream=None):
        import torch
        if x.dim() != 2 or x.shape[1] != self.d or tuple(g.shape) != (self.d,):
            raise ValueError("shape mismatch: x [M, d], g [d] expected")
        if x.dtype != torch.bfloat16 or g.dtype != torch.bfloat16:
            raise ValueError("bf16 inputs expected")
        if not (x.is_cuda and g.is_cuda and x.is_contiguous() and g.is_contiguous()):
            raise ValueError("x and g must be contiguous CUDA tensors")
        M = int(x.shape[0])
        if y is None:
            y = _new_output(lambda: torch.empty((M, self.d), dtype=torch.bfloat16, device=x.device), stream, x.device)
        if tuple(y.shape) != (M, self.d) or y.dtype != torch.bfloat16 or not y.is_contiguous():
            raise ValueError("y must be a contiguous [M, d] bf16 tensor")
        if stream is None:
            stream = torch.cuda.current_stream(x.device)
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        bi_rmsnorm_run(self.handle, x.data_ptr(), M, g.data_ptr(), y.data_ptr(), s)
        return y

    __call__ = run

    def close(self) -> None:
        if getattr(self, "handle", None):
            bi_rmsnorm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BiAttention:
    """Batch-invariant decode attention over a paged KV cache on torch tensors.

    q [T, Hq, D] bf16; k_cache, v_cache [pages, page_size, Hkv, D] bf16; page_table int32
    [num_seqs, max_pages]; q_seq, q_pos int32 [T] (request and position of each query token).
    """

    def __init__(self, num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int,
                 scale: float | None = None, split_size: int = 0):
        self.Hq, self.Hkv, self.D, self.page_size = int(num_q_heads), int(num_kv_heads), int(head_dim), int(page_size)
        self.scale = float(scale) if scale is not None else float(head_dim) ** -0.5
        self.handle = bi_attention_create(self.Hq, self.Hkv, self.D, self.page_size, self.scale, split_size)
        self._device = _handle_device()

    @property
    def config(self) -> dict:
        return bi_attention_get_config(self.handle)

    def run(self, q, q_seq, q_pos, k_cache, v_cache, page_table, max_pos: int, o=None, stream=None):
        import torch
        T = int(q.shape[0])
        if q.dim() != 3 or q.shape[1] != self.Hq or q.shape[2] != self.D:
            raise ValueError("q must be [T, num_q_heads, head_dim]")
        if k_cache.dim() != 4 or tuple(k_cache.shape[1:]) != (self.page_size, self.Hkv, self.D) or \
                v_cache.shape != k_cache.shape:
            raise ValueError("k_cache, v_cache must be [pages, page_size, num_kv_heads, head_dim]")
        for name, tns in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache)):
            if tns.dtype != torch.bfloat16 or not tns.is_cuda or not tns.is_contiguous():
                raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
        for name, tns in (("q_seq", q_seq), ("q_pos", q_pos), ("page_table", page_table)):
            if tns.dtype != torch.int32 or not tns.is_cuda or not tns.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
        if tuple(q_seq.shape) != (T,) or tuple(q_pos.shape) != (T,) or page_table.dim() != 2:
            raise ValueError("q_seq, q_pos [T]; page_table [num_seqs, max_pages]")
        if o is None:
            o = _new_output(lambda: torch.empty_like(q), stream, q.device)
        if o.shape != q.shape or o.dtype != torch.bfloat16 or not o.is_contiguous():
            raise ValueError("o must be a contiguous bf16 tensor shaped like q")
        if stream is None:
            stream = torch.cuda.current_stream(q.device)
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        bi_attention_run(self.handle, q.data_ptr(), T, q_seq.data_ptr(), q_pos.data_ptr(), k_cache.data_ptr(),
                         v_cache.data_ptr(), int(k_cache.shape[0]), page_table.data_ptr(), int(page_table.shape[0]),
                         int(page_table.shape[1]), int(max_pos), o.data_ptr(), s)
        return o

    __call__ = run

    def device_error(self, stream=None) -> int:
        s = 0
        if stream is not None:
            s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        return bi_attention_get_device_error(self.handle, s)

    def run_shared(self, q, q_seq, q_pos, k_cache, v_cache, page_table, max_pos: int, group_start, group_len,
                   o=None, stream=None):
        """run() for tokens in groups that share a prefix: group g is the tokens group_start[g] ..
        group_start[g + 1] - 1 (int32 [groups + 1], ascending), whose requests name the same pages
        for positions 0 .. group_len[g] - 1 (int32 [groups]).  The prefix is read once per group;
        the result has the bits of run()."""
        T, index, o = _check_queries(q, o, self.Hq, self.D, self._device, stream)
        pages, seqs, per = _check_cache(k_cache, v_cache, page_table, (self.page_size, self.Hkv, self.D), index)
        groups, i32 = group_len.shape[0], _torch.i32
        _check_tensor("q_seq", q_seq, i32, (T,), index)
        _check_tensor("q_pos", q_pos, i32, (T,), index)
        _check_tensor("group_len", group_len, i32, (groups,), index)
        _check_tensor("group_start", group_start, i32, (groups + 1,), index)
        _check(library().bi_attention_run_shared(self.handle, q.data_ptr(), T, q_seq.data_ptr(), q_pos.data_ptr(),
                                                 k_cache.data_ptr(), v_cache.data_ptr(), pages, page_table.data_ptr(),
                                                 seqs, per, max_pos, group_start.data_ptr(), group_len.data_ptr(),
                                                 groups, o.data_ptr(), _stream_of(stream, index)),
               "bi_attention_run_shared")
        return o

    def workspace_size(self, T: int, max_pos: int) -> int:
        return bi_attention_workspace_size(self.handle, T, max_pos)

    def shared_workspace_size(self, T: int, max_pos: int, num_groups: int) -> int:
        return bi_attention_shared_workspace_size(self.handle, T, max_pos, num_groups)

    def close(self) -> None:
        if getattr(self, "handle", None):
            bi_attention_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _Torch:
    """What the calls around the paged cache need of torch, looked up once (the module itself does not
    import it): these calls are on the path of a single token's step."""

    def __init__(self):
        import torch
        self.bf16, self.f32, self.i32, self.u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
        self.empty, self.empty_like, self.device = torch.empty, torch.empty_like, torch.device
        self.current_stream = torch._C._cuda_getCurrentRawStream
        self.current_device = torch.cuda.current_device


_torch = None


def _handle_device() -> int:
    """The device a handle made now belongs to."""
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch.current_device()


def _handle_devices():
    """The same as (index, torch.device)."""
    index = _handle_device()
    return index, _torch.device("cuda", index)


def _stream_of(stream, index: int) -> int:
    """The cudaStream_t of a stream argument; the device's current stream for None."""
    if stream is None:
        return _torch.current_stream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check_tensor(name: str, t, dtype, shape, index: int) -> None:
    """t: a contiguous tensor of this dtype and shape on CUDA device `index`.  (Plain attributes, no
    objects built unless something is wrong.)"""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', strided'}")


def _take(name: str, t, dtype, shape, index: int, stream, device):
    """The output t, checked, or a new one (made for `stream`) where it is None."""
    if t is not None:
        _check_tensor(name, t, dtype, shape, index)
        return t
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    return _new_output(lambda: _torch.empty(shape, dtype=dtype, device=device), stream, device)


def _check_cache(k_cache, v_cache, page_table, page_shape, index: int):
    """The paged cache of one layer: k_cache, v_cache [pages, page_size, Hkv, D] bf16, page_table
    [num_seqs, max_pages] int32.  Returns (pages, num_seqs, max_pages)."""
    shape = k_cache.shape
    if len(shape) != 4 or shape[1:] != page_shape:
        raise ValueError(f"k_cache must be [pages, page_size, num_kv_heads, head_dim] = [pages, {page_shape}]")
    _check_tensor("k_cache", k_cache, _torch.bf16, shape, index)
    _check_tensor("v_cache", v_cache, _torch.bf16, shape, index)
    table = page_table.shape
    if len(table) != 2:
        raise ValueError("page_table must be [num_seqs, max_pages]")
    _check_tensor("page_table", page_table, _torch.i32, table, index)
    return shape[0], table[0], table[1]


def _check_codes(k_codes, k_scales, v_codes, v_scales, page_shape, index: int) -> int:
    """The paged cache of one layer in 4 bits: codes [pages, page_size, Hkv, D / 2] and scales [.., D / 16], uint8.
    Returns its pages."""
    page, heads, D = page_shape
    shape, u8 = k_codes.shape, _torch.u8
    if len(shape) != 4 or shape[1:] != (page, heads, D // 2):
        raise ValueError(f"k_codes must be [pages, page_size, num_kv_heads, head_dim / 2] = [pages, {page}, {heads}, {D // 2}]")
    scales = (shape[0], page, heads, D // 16)
    _check_tensor("k_codes", k_codes, u8, shape, index)
    _check_tensor("v_codes", v_codes, u8, shape, index)
    _check_tensor("k_scales", k_scales, u8, scales, index)
    _check_tensor("v_scales", v_scales, u8, scales, index)
    return shape[0]


def _check_cache4(k_codes, k_scales, v_codes, v_scales, page_table, page_shape, index: int):
    """_check_cache for a cache in 4 bits."""
    pages = _check_codes(k_codes, k_scales, v_codes, v_scales, page_shape, index)
    table = page_table.shape
    if len(table) != 2:
        raise ValueError("page_table must be [num_seqs, max_pages]")
    _check_tensor("page_table", page_table, _torch.i32, table, index)
    return pages, table[0], table[1]


def _check_queries(q, o, Hq: int, D: int, device: int, stream):
    """q [T, Hq, D] bf16 and o like it (made for `stream` where it is None) on the handle's device.
    Returns (T, device index, o)."""
    shape, index = q.shape, q.get_device()
    if len(shape) != 3 or shape[1] != Hq or shape[2] != D or index != device:
        raise ValueError(f"q must be a tensor [T, num_q_heads, head_dim] on cuda:{device}")
    _check_tensor("q", q, _torch.bf16, shape, index)
    if o is None:
        o = _torch.empty_like(q) if stream is None else _new_output(lambda: _torch.empty_like(q), stream, q.device)
    else:
        _check_tensor("o", o, _torch.bf16, shape, index)
    return shape[0], index, o


class BiQkRope:
    """Per-head RMSNorm of queries and keys, rotation by position and append to the paged cache
    in one pass, on torch tensors (include/bi_qkrope.h has the definition and the conventions).

    qkv [T, (Hq + 2 Hkv) D] bf16 (rows may be strided); gq, gk [D] bf16, or both None for no norm;
    cos_sin [positions, rot_dim] fp32, the cosines of a position's rot_dim / 2 angles, then their
    sines; q_seq, q_pos int32 [T] (request and position of each token); caches and page table as in
    BiAttention.  Returns q [T, Hq, D]; keys and values go to their slots of the caches.
    """

    def __init__(self, num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int, rot_dim: int | None = None,
                 eps: float = 1e-6, interleaved: bool = False):
        self.Hq, self.Hkv, self.D, self.page_size = int(num_q_heads), int(num_kv_heads), int(head_dim), int(page_size)
        self.rot_dim = int(rot_dim) if rot_dim is not None else self.D
        self._width, self._page_shape = (self.Hq + 2 * self.Hkv) * self.D, (self.page_size, self.Hkv, self.D)
        self.handle = bi_qkrope_create(self.Hq, self.Hkv, self.D, self.page_size, self.rot_dim, interleaved, eps)
        self._device, self._on = _handle_devices()
        self._run, self._run4 = library().bi_qkrope_run, library().bi_qkrope_run4

    @property
    def config(self) -> dict:
        return bi_qkrope_get_config(self.handle)

    def _rows(self, qkv, gq, gk, cos_sin, q_seq, q_pos, q_out, stream):
        """The arguments that say nothing of the cache, checked: (device index, tokens, row stride, gq, gk, positions,
        q_out)."""
        bf16, i32 = _torch.bf16, _torch.i32
        shape, index, width = qkv.shape, qkv.get_device(), self._width
        if len(shape) != 2 or shape[1] != width or qkv.dtype is not bf16 or index != self._device:
            raise ValueError(f"qkv must be a bf16 tensor [T, (num_q_heads + 2 num_kv_heads) head_dim] on "
                             f"cuda:{self._device}")
        T, stride = shape[0], width
        if not qkv.is_contiguous():
            stride, inner = qkv.stride()
            if inner != 1 or stride < width:
                raise ValueError("qkv rows must be contiguous and must not overlap")
        if gq is None or gk is None:
            if gq is not gk:
                raise ValueError("gq and gk: both norm weights or neither")
            wq = wk = None
        else:
            _check_tensor("gq", gq, bf16, (self.D,), index)
            _check_tensor("gk", gk, bf16, (self.D,), index)
            wq, wk = gq.data_ptr(), gk.data_ptr()
        angles = cos_sin.shape
        if len(angles) != 2 or angles[1] != self.rot_dim:
            raise ValueError("cos_sin must be [positions, rot_dim]")
        _check_tensor("cos_sin", cos_sin, _torch.f32, angles, index)
        _check_tensor("q_seq", q_seq, i32, (T,), index)
        _check_tensor("q_pos", q_pos, i32, (T,), index)
        q_out = _take("q_out", q_out, bf16, (T, self.Hq, self.D), index, stream, self._on)
        return index, T, stride, wq, wk, angles[0], q_out

    def run(self, qkv, gq, gk, cos_sin, q_seq, q_pos, k_cache, v_cache, page_table, q_out=None, stream=None):
        index, T, stride, wq, wk, positions, q_out = self._rows(qkv, gq, gk, cos_sin, q_seq, q_pos, q_out, stream)
        pages, seqs, per = _check_cache(k_cache, v_cache, page_table, self._page_shape, index)
        rc = self._run(self.handle, qkv.data_ptr(), T, stride, wq, wk, cos_sin.data_ptr(), positions, q_seq.data_ptr(),
                       q_pos.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), pages, page_table.data_ptr(), seqs, per,
                       q_out.data_ptr(), _stream_of(stream, index))
        if rc:
            _check(rc, "bi_qkrope_run")
        return q_out

    def run4(self, qkv, gq, gk, cos_sin, q_seq, q_pos, k_codes, k_scales, v_codes, v_scales, page_table,
             k_scale: float = 1.0, v_scale: float = 1.0, q_out=None, stream=None):
        """run() into a cache in 4 bits (BiAttention4's): keys and values quantised with the tensor scales k_scale
        and v_scale, the codes and scales that BiQuant4 "nvfp4" gives the rows that run() would store.  A token at -1 is
        an empty place: nothing is appended, its row of q_out is left as it was (undefined in a new one)."""
        index, T, stride, wq, wk, positions, q_out = self._rows(qkv, gq, gk, cos_sin, q_seq, q_pos, q_out, stream)
        pages, seqs, per = _check_cache4(k_codes, k_scales, v_codes, v_scales, page_table, self._page_shape, index)
        rc = self._run4(self.handle, qkv.data_ptr(), T, stride, wq, wk, cos_sin.data_ptr(), positions, q_seq.data_ptr(),
                        q_pos.data_ptr(), k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
                        k_scale, v_scale, pages, page_table.data_ptr(), seqs, per, q_out.data_ptr(), _stream_of(stream, index))
        if rc:
            _check(rc, "bi_qkrope_run4")
        return q_out

    __call__ = run

    def device_error(self, stream=None) -> int:
        s = 0
        if stream is not None:
            s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        return bi_qkrope_get_device_error(self.handle, s)

    def close(self) -> None:
        if getattr(self, "handle", None):
            bi_qkrope_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BiPromptAttention:
    """Batch-invariant causal attention of packed prompts, or of chunks of them behind a cached
    context, over the paged KV cache of BiAttention, on torch tensors (include/bi_prompt.h).

    q [T, Hq, D] bf16, the sequences one after the other; q_start int32 [num_seqs + 1], the first row
    of each and the end of the last; q_pos0 int32 [num_seqs], the position of each first row (0 for
    a whole prompt); caches and page table as in BiAttention, holding the calls' own keys and values.
    max_pos: an upper bound of every position.  Returns o [T, Hq, D]; rows outside the sequences are
    left as they were (undefined in a new o).
    """

    def __init__(self, num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int,
                 scale: float | None = None):
        self.Hq, self.Hkv, self.D, self.page_size = int(num_q_heads), int(num_kv_heads), int(head_dim), int(page_size)
        self.scale = float(scale) if scale is not None else float(head_dim) ** -0.5
        self._page_shape = (self.page_size, self.Hkv, self.D)
        self.handle = bi_prompt_create(self.Hq, self.Hkv, self.D, self.page_size, self.scale)
        self._device = _handle_device()

    @property
    def config(self) -> dict:
        return bi_prompt_get_config(self.handle)

    def run(self, q, q_start, q_pos0, k_cache, v_cache, page_table, max_pos: int, o=None, stream=None):
        T, index, o = _check_queries(q, o, self.Hq, self.D, self._device, stream)
        pages, seqs, per = _check_cache(k_cache, v_cache, page_table, self._page_shape, index)
        _check_tensor("q_start", q_start, _torch.i32, (seqs + 1,), index)
        _check_tensor("q_pos0", q_pos0, _torch.i32, (seqs,), index)
        _check(library().bi_prompt_run(self.handle, q.data_ptr(), T, q_start.data_ptr(), q_pos0.data_ptr(), seqs,
                                       k_cache.data_ptr(), v_cache.data_ptr(), pages, page_table.data_ptr(), per,
                                       max_pos, o.data_ptr(), _stream_of(stream, index)), "bi_prompt_run")
        return o

    __call__ = run

    def device_error(self, stream=None) -> int:
        s = 0
        if stream is not None:
            s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        return bi_prompt_get_device_error(self.handle, s)

    def workspace_size(self, T: int, num_seqs: int) -> int:
        return bi_prompt_workspace_size(self.handle, T, num_seqs)

    def close(self) -> None:
        if getattr(self, "handle", None):
            bi_prompt_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BiAttention4:
    """Batch-invariant decode attention over a paged KV cache in 4 bits, on torch tensors (include/bi_attention4.h).

    q [T, Hq, D] bf16; k_codes, v_codes [pages, page_size, Hkv, D / 2] and k_scales, v_scales [pages, page_size, Hkv,
    D / 16] uint8, filled by BiQkRope.run4; k_scale, v_scale: the tensor scales they were made with; page_table
    int32 [num_seqs, max_pages]; q_seq, q_pos int32 [T] (request and position of each query token; a token at
    -1 sees nothing and gets zeros).  max_pos: an upper bound of every position.
    """

    def __init__(self, num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int, scale: float | None = None,
                 k_scale: float = 1.0, v_scale: float = 1.0, split_size: int = 0):
        self.Hq, self.Hkv, self.D, self.page_size = int(num_q_heads), int(num_kv_heads), int(head_dim), int(page_size)
        self.scale = float(scale) if scale is not None else float(head_dim) ** -0.5
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self._page_shape = (self.page_size, self.Hkv, self.D)
        self.handle = bi_attention4_create(self.Hq, self.Hkv, self.D, self.page_size, self.scale, self.k_scale,
                                           self.v_scale, split_size)
        self._device, self._on = _handle_devices()
        self._run, self._expand = library().bi_attention4_run, library().bi_attention4_expand

    @property
    def config(self) -> dict:
        return bi_attention4_get_config(self.handle)

    def run(self, q, q_seq, q_pos, k_codes, k_scales, v_codes, v_scales, page_table, max_pos: int, o=None, stream=None):
        T, index, o = _check_queries(q, o, self.Hq, self.D, self._device, stream)
        pages, seqs, per = _check_cache4(k_codes, k_scales, v_codes, v_scales, page_table, self._page_shape, index)
        _check_tensor("q_seq", q_seq, _torch.i32, (T,), index)
        _check_tensor("q_pos", q_pos, _torch.i32, (T,), index)
        rc = self._run(self.handle, q.data_ptr(), T, q_seq.data_ptr(), q_pos.data_ptr(), k_codes.data_ptr(),
                       k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(), pages, page_table.data_ptr(), seqs, per,
                       max_pos, o.data_ptr(), _stream_of(stream, index))
        if rc:
            _check(rc, "bi_attention4_run")
        return o

    __call__ = run

    def expand(self, k_codes, k_scales, v_codes, v_scales, pages, k=None, v=None, stream=None):
        """The values k, v [n, page_size, Hkv, D] bf16 of the cache's pages `pages` (int32 [n]; page i of the result
        is left as it was, undefined in a new one, where the entry is -1)."""
        index, n = k_codes.get_device(), pages.shape[0]
        if index != self._device:
            raise ValueError(f"k_codes must be a tensor on cuda:{self._device}")
        count = _check_codes(k_codes, k_scales, v_codes, v_scales, self._page_shape, index)
        _check_tensor("pages", pages, _torch.i32, (n,), index)
        k = _take("k", k, _torch.bf16, (n, *self._page_shape), index, stream, self._on)
        v = _take("v", v, _torch.bf16, (n, *self._page_shape), index, stream, self._on)
        rc = self._expand(self.handle, k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(), count,
                          pages.data_ptr(), n, k.data_ptr(), v.data_ptr(), _stream_of(stream, index))
        if rc:
            _check(rc, "bi_attention4_expand")
        return k, v

    def device_error(self, stream=None) -> int:
        s = 0
        if stream is not None:
            s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        return bi_attention4_get_device_error(self.handle, s)

    def workspace_size(self, T: int, max_pos: int) -> int:
        return bi_attention4_workspace_size(self.handle, T, max_pos)

    def close(self) -> None:
        if getattr(self, "handle", None):
            bi_attention4_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_FP4 = {"mxfp4": (BI_MXFP4, 32), "nvfp4": (BI_NVFP4, 16)}


def _scale_tiles(rows: int, K: int, block: int):
    """Shape of the scales of `rows` rows: tiles of 128 rows x 4 scales, row r's scale c at
    [r // 128, c // 4, r % 32, r // 32 % 4, c % 4]."""
    return (-(-rows // 128), K // (4 * block), 32, 4, 4)


class BiQuant4:
    """Rows of bf16 in 4 bits, on torch tensors (include/bi_fp4.h has the definition).

    kind "mxfp4" (E2M1 codes, a power of two per 32 elements) or "nvfp4" (an E4M3 scale per 16, times the
    constant tensor_scale).  run(x [M, K] bf16, rows may be strided) returns codes uint8 [M, K / 2] and
    scales uint8 in tiles [ceil(M / 128), K / (4 block), 32, 4, 4] (the bytes of rows past M are left as they
    were, undefined in new scales): the operands of BiGemm4.  expand() gives the values back as bf16.
    """

    def __init__(self, K: int, kind: str = "nvfp4", tensor_scale: float = 1.0):
        if kind not in _FP4:
            raise ValueError("kind: 'mxfp4' or 'nvfp4'")
        self.K, self.kind, self.tensor_scale = int(K), kind, float(tensor_scale)
        fmt, self.block = _FP4[kind]
        self.handle = bi_quant4_create(self.K, fmt, self.tensor_scale)
        self._device, self._on = _handle_devices()
        self._run, self._expand = library().bi_quant4_run, library().bi_quant4_expand

    @property
    def config(self) -> dict:
        return bi_quant4_get_config(self.handle)

    def run(self, x, codes=None, scales=None, stream=None):
        shape, index, K = x.shape, x.get_device(), self.K
        if len(shape) != 2 or shape[1] != K or x.dtype is not _torch.bf16 or index != self._device:
            raise ValueError(f"x must be a bf16 tensor [M, {K}] on cuda:{self._device}")
        M, stride = shape[0], K
        if not x.is_contiguous():
            stride, inner = x.stride()
            if inner != 1 or stride < K:
                raise ValueError("x rows must be contiguous and must not overlap")
        codes = _take("codes", codes, _torch.u8, (M, K // 2), index, stream, self._on)
        scales = _take("scales", scales, _torch.u8, _scale_tiles(M, K, self.block), index, stream, self._on)
        rc = self._run(self.handle, x.data_ptr(), M, stride, codes.data_ptr(), scales.data_ptr(), _stream_of(stream, index))
        if rc:
            _check(rc, "bi_quant4_run")
        return codes, scales

    __call__ = run

    def expand(self, codes, scales, y=None, stream=None):
        """The values [M, K] bf16 that codes and scales stand for."""
        index = codes.get_device()
        if len(codes.shape) != 2 or index != self._device:
            raise ValueError(f"codes must be a tensor [M, K / 2] on cuda:{self._device}")
        M = codes.shape[0]
        _check_tensor("codes", codes, _torch.u8, (M, self.K // 2), index)
        _check_tensor("scales", scales, _torch.u8, _scale_tiles(M, self.K, self.block), index)
        y = _take("y", y, _torch.bf16, (M, self.K), index, stream, self._on)
        rc = self._expand(self.handle, codes.data_ptr(), scales.data_ptr(), M, y.data_ptr(), _stream_of(stream, index))
        if rc:
            _check(rc, "bi_quant4_expand")
        return y

    def close(self) -> None:
        if getattr(self, "handle", None):
            bi_quant4_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BiGemm4:
    """y = alpha x w^T of two matrices in 4 bits for fixed (K, N), on torch tensors (include/bi_fp4.h).

    x [M, K / 2], w [N, K / 2] codes and sx, sw their scales in tiles, all uint8 as BiQuant4.run makes them (both
    of this handle's kind); y [M, N] bf16 or, with out="f32", fp32.  alpha carries the tensor scales of "nvfp4".
    """

    def __init__(self, K: int, N: int, kind: str = "nvfp4", out: str = "bf16"):
        if kind not in _FP4 or out not in ("bf16", "f32"):
            raise ValueError("kind: 'mxfp4' or 'nvfp4'; out: 'bf16' or 'f32'")
        self.K, self.N, self.kind, self.out = int(K), int(N), kind, out
        fmt, self.block = _FP4[kind]
        self.handle = bi_gemm4_create(self.K, self.N, fmt, out == "f32")
        self._device, self._on = _handle_devices()
        self._run = library().bi_gemm4_run
        self._w, self._sw = (self.N, self.K // 2), _scale_tiles(self.N, self.K, self.block)
        self._dtype = _torch.f32 if out == "f32" else _torch.bf16

    @property
    def config(self) -> dict:
        return bi_gemm4_get_config(self.handle)

    def run(self, x, sx, w, sw, alpha: float = 1.0, y=None, stream=None):
        index, u8 = x.get_device(), _torch.u8
        if len(x.shape) != 2 or index != self._device:
            raise ValueError(f"x must be a tensor [M, K / 2] on cuda:{self._device}")
        M = x.shape[0]
        _check_tensor("x", x, u8, (M, self.K // 2), index)
        _check_tensor("sx", sx, u8, _scale_tiles(M, self.K, self.block), index)
        _check_tensor("w", w, u8, self._w, index)
        _check_tensor("sw", sw, u8, self._sw, index)
        y = _take("y", y, self._dtype, (M, self.N), index, stream, self._on)
        rc = self._run(self.handle, x.data_ptr(), sx.data_ptr(), M, w.data_ptr(), sw.data_ptr(), alpha, y.data_ptr(),
                       _stream_of(stream, index))
        if rc:
            _check(rc, "bi_gemm4_run")
        return y

    __call__ = run

    def device_error(self, stream=None) -> int:
        s = 0
        if stream is not None:
            s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        return bi_gemm4_get_device_error(self.handle, s)

    def close(self) -> None:
        if getattr(self, "handle", None):
            bi_gemm4_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BiPreNorm:
    """mHC pre-norm projection y = RMSNorm(x) . W (fp32 out) on torch tensors: x [M, K] bf16,
    W [K, N] bf16 (a norm weight folded into W's rows)."""

    def __init__(self, K: int, N: int, eps: float = 1e-6, chunk: int = 0):
        self.K, self.N, self.eps = int(K), int(N), float(eps)
        self.handle = bi_prenorm_create(self.K, self.N, self.eps, chunk)

    @property
    def config(self) -> dict:
        return bi_prenorm_get_config(self.handle)

    def run(self, x, W, y=None, stream=None):
        import torch
        if x.dim() != 2 or x.shape[1] != self.K or tuple(W.shape) != (self.K, self.N):
            raise ValueError("shape mismatch: x [M, K], W [K, N] expected")
        if x.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
            raise ValueError("bf16 inputs expected")
        if not (x.is_cuda and W.is_cuda and x.is_contiguous() and W.is_contiguous()):
            raise ValueError("x and W must be contiguous CUDA tensors")
        M = int(x.shape[0])
        if y is None:
            y = _new_output(lambda: torch.empty((M, self.N), dtype=torch.float32, device=x.device), stream, x.device)
        if tuple(y.shape) != (M, self.N) or y.dtype != torch.float32 or not y.is_contiguous():
            raise ValueError("y must be a contiguous [M, N] fp32 tensor")
        if stream is None:
            stream = torch.cuda.current_stream(x.device)
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        bi_prenorm_run(self.handle, x.data_ptr(), M, W.data_ptr(), y.data_ptr(), s)
        return y

    __call__ = run

    def close(self) -> None:
        if getattr(self, "handle", None):
            bi_prenorm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


__all__ = [
    "BiQuant4", "bi_quant4_create", "bi_quant4_scale_bytes", "bi_quant4_run", "bi_quant4_expand", "bi_quant4_get_config",
    "bi_quant4_destroy", "bi_quant4_config", "BiGemm4", "bi_gemm4_create", "bi_gemm4_run", "bi_gemm4_get_device_error",
    "bi_gemm4_get_config", "bi_gemm4_destroy", "bi_gemm4_config", "FP4_EXPORTED_SYMBOLS", "BI_MXFP4", "BI_NVFP4",
    "BiAttention4", "bi_attention4_create", "bi_attention4_run", "bi_attention4_workspace_size", "bi_attention4_expand",
    "bi_attention4_get_device_error", "bi_attention4_get_config", "bi_attention4_destroy", "bi_attention4_config",
    "ATTENTION4_EXPORTED_SYMBOLS", "bi_qkrope_run4",
    "BiPromptAttention", "bi_prompt_create", "bi_prompt_run", "bi_prompt_workspace_size", "bi_prompt_get_device_error",
    "bi_prompt_get_config", "bi_prompt_destroy", "bi_prompt_config", "PROMPT_EXPORTED_SYMBOLS",
    "BiQkRope", "bi_qkrope_create", "bi_qkrope_run", "bi_qkrope_get_device_error", "bi_qkrope_get_config",
    "bi_qkrope_destroy", "bi_qkrope_config", "QKROPE_EXPORTED_SYMBOLS",
    "BiPreNorm", "bi_prenorm_create", "bi_prenorm_run", "bi_prenorm_get_config", "bi_prenorm_destroy",
    "bi_prenorm_config", "PRENORM_EXPORTED_SYMBOLS",
    "BiAttention", "bi_attention_create", "bi_attention_run", "bi_attention_get_config", "bi_attention_workspace_size",
    "bi_attention_get_device_error", "bi_attention_destroy", "bi_attention_config", "bi_attention_run_shared",
    "bi_attention_shared_workspace_size", "ATTENTION_EXPORTED_SYMBOLS",
    "BiRmsNorm", "bi_rmsnorm_create", "bi_rmsnorm_run", "bi_rmsnorm_get_config", "bi_rmsnorm_destroy",
    "bi_rmsnorm_config", "RMSNORM_EXPORTED_SYMBOLS",
    "BiGemm", "BiGemmError", "bi_gemm_create", "bi_gemm_run", "bi_gemm_run_noalloc", "bi_gemm_get_device_error",
    "bi_gemm_destroy", "bi_gemm_get_config", "bi_gemm_workspace_size", "bi_gemm_strerror",
    "bi_gemm_version", "bi_gemm_scales", "bi_gemm_options", "bi_gemm_block", "EXPORTED_SYMBOLS", "LIB_PATH", "library",
]
