"""Python binding of libexq: mixed-bitrate (EXL2-style) quantized linears on MI355X.

Argument marshalling only.  Every step of the path -- packing, dequantization
and the matmul -- runs in libexq (host C++ and gfx950 HIP kernels); PyTorch
is used for device memory and streams.  The library is loaded from this
directory; importing the package fails loudly when it is missing and cannot
be built, and there is no fallback path.

The C entry points keep their names (``exq_pack``, ``exq_layer_create``,
``exq_gemm``, ...); see ``include/exq.h`` for argument meaning, layout,
ownership and errors.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libexq.so")
GROUP = 128
MAX_DECODE_M = 16

EXQ_OK, EXQ_ERR_INVALID_ARG, EXQ_ERR_UNSUPPORTED, EXQ_ERR_HIP, EXQ_ERR_OOM = range(5)


class ExqError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str):
        super().__init__("%s failed: %s (%s)" % (what, _status_name(status), detail))
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        from . import build as _b
        try:
            _b.build()
        except RuntimeError:
            if not os.path.exists(LIB_PATH):
                raise
            # only the extension module failed: KVCache, which needs it, tries again and says why
    # PyTorch ships its own HIP runtime.  Importing it first makes libexq bind
    # to that already-loaded runtime instead of loading a second copy from
    # the ROCm install, so device pointers and streams from torch and from
    # libexq belong to one runtime.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.exq_status_string.argtypes = [i32]
    lib.exq_status_string.restype = ctypes.c_char_p
    lib.exq_last_error.argtypes = []
    lib.exq_last_error.restype = ctypes.c_char_p
    lib.exq_packed_bytes.argtypes = [i32, i32, i32, vp]
    lib.exq_packed_bytes.restype = u64
    lib.exq_pack.argtypes = [vp, i32, i32, i32, vp, vp, vp]
    lib.exq_layer_create.argtypes = [i32, i32, i32, vp, vp, vp, ctypes.POINTER(vp)]
    lib.exq_layer_destroy.argtypes = [vp]
    lib.exq_layer_destroy.restype = None
    lib.exq_gemm.argtypes = [vp, i32, vp, vp, vp]
    lib.exq_gemm_noalloc.argtypes = [vp, i32, vp, vp, vp]
    lib.exq_dequant.argtypes = [vp, vp, vp]
    lib.exq_plan_create.argtypes = [i32, vp, vp, vp, i32, ctypes.POINTER(vp)]
    lib.exq_plan_run.argtypes = [vp, vp]
    lib.exq_plan_destroy.argtypes = [vp]
    lib.exq_plan_destroy.restype = None
    lib.exq_stream_read.argtypes = [vp, u64, vp, i32, vp]
    lib.exq_gemm_gated.argtypes = [vp, i32, vp, vp, vp, vp]
    lib.exq_group_errors.argtypes = [vp, i32, i32, i32, vp]
    lib.exq_pack_qs.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp]
    lib.exq_layer_create_qs.argtypes = [i32, i32, i32, vp, vp, vp, vp, ctypes.POINTER(vp)]
    lib.exq_trimmed_mean.argtypes = [vp, i32]
    lib.exq_trimmed_mean.restype = ctypes.c_double
    lib.exq_autotune.argtypes = [vp, i32, vp, vp, vp, i32, i32, vp, vp]
    lib.exq_set_variant.argtypes = [vp, i32, i32]
    lib.exq_allocate_widths.argtypes = [vp, vp, i32, ctypes.c_int64, vp, ctypes.c_uint64, ctypes.c_int64, vp, vp]
    i64 = ctypes.c_int64
    lib.exq_cache_page_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.exq_cache_page_bytes.restype = u64
    lib.exq_cache_create.argtypes = [vp, i64, i32, i32, i32, i32, i32, ctypes.POINTER(vp)]
    lib.exq_cache_destroy.argtypes = [vp]
    lib.exq_cache_destroy.restype = None
    rows_call = [vp, vp, i64, i64, vp, i64, i64, i32, vp, i32, i32, i64, vp, vp, vp]
    lib.exq_cache_append.argtypes = rows_call
    lib.exq_cache_read.argtypes = rows_call
    lib.exq_attend_workspace_bytes.argtypes = [vp, i32, i32, i32]
    lib.exq_attend_workspace_bytes.restype = u64
    lib.exq_attend.argtypes = [vp, vp, i64, i64, i32, i32, vp, i32, i64, vp, ctypes.c_float, i32, vp, i64, i64, vp, vp,
                               u64, vp]
    f32 = ctypes.c_float
    pages = [vp, i32, i32, i64, i32, vp, vp, vp, vp, i32]
    lib.exq_pages_workspace_bytes.argtypes = [i32]
    lib.exq_pages_workspace_bytes.restype = u64
    lib.exq_pages_extend.argtypes = pages + [vp, vp, i32, vp, vp, vp, u64, vp]
    lib.exq_pages_trim.argtypes = pages + [vp, u64, vp]
    lib.exq_rotate.argtypes = [vp, i64, i64, vp, i64, i64, i32] * 2 + [i32, i32, i32, i32, vp, f32, vp, vp]
    lib.exq_adapters_create.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, ctypes.POINTER(vp)]
    lib.exq_adapters_destroy.argtypes = [vp]
    lib.exq_adapters_destroy.restype = None
    lib.exq_lora_workspace_bytes.argtypes = [vp, i32]
    lib.exq_lora_workspace_bytes.restype = u64
    lib.exq_lora_add.argtypes = [vp, vp, i64, i32, vp, vp, i64, vp, i64, vp, u64, vp]
    lib.exq_sample_workspace_bytes.argtypes = [i32, i32]
    lib.exq_sample_workspace_bytes.restype = u64
    lib.exq_sample.argtypes = [vp, i32, i32, i32, i64, vp, vp, f32, vp, i32, vp, f32, vp, f32, vp, vp, vp, u64, vp]
    for f in (lib.exq_pages_extend, lib.exq_pages_trim, lib.exq_rotate, lib.exq_adapters_create, lib.exq_lora_add, lib.exq_sample,
              lib.exq_pack, lib.exq_layer_create, lib.exq_gemm, lib.exq_gemm_noalloc, lib.exq_dequant, lib.exq_plan_create,
              lib.exq_plan_run, lib.exq_stream_read, lib.exq_gemm_gated, lib.exq_group_errors,
              lib.exq_allocate_widths, lib.exq_autotune, lib.exq_set_variant, lib.exq_pack_qs,
              lib.exq_layer_create_qs, lib.exq_cache_create, lib.exq_cache_append, lib.exq_cache_read, lib.exq_attend):
        f.restype = i32
    return lib


lib = _load()

# Symbols include/exq.h declares (checked by the tests).
EXPORTED = (
    "exq_status_string", "exq_last_error", "exq_packed_bytes", "exq_pack", "exq_layer_create",
    "exq_layer_destroy", "exq_gemm", "exq_dequant", "exq_plan_create", "exq_plan_run", "exq_plan_destroy",
    "exq_stream_read", "exq_gemm_gated", "exq_group_errors", "exq_allocate_widths", "exq_trimmed_mean",
    "exq_autotune", "exq_set_variant", "exq_pack_qs", "exq_layer_create_qs", "exq_gemm_noalloc",
    "exq_cache_page_bytes", "exq_cache_create", "exq_cache_destroy", "exq_cache_append", "exq_cache_read",
    "exq_attend_workspace_bytes", "exq_attend", "exq_pages_workspace_bytes", "exq_pages_extend", "exq_pages_trim", "exq_rotate",
    "exq_adapters_create", "exq_adapters_destroy", "exq_lora_workspace_bytes", "exq_lora_add", "exq_sample_workspace_bytes",
    "exq_sample",
)

VARIANT_DEFAULT, VARIANT_DECODE16, VARIANT_DECODE64, VARIANT_PREFILL = 0, 1, 2, 3


def _status_name(s: int) -> str:
    return lib.exq_status_string(s).decode()


def _check(status: int, what: str):
    if status != EXQ_OK:
        raise ExqError(status, what, lib.exq_last_error().decode())


def _np_ptr(a: np.ndarray) -> int:
    assert a.flags["C_CONTIGUOUS"]
    return a.ctypes.data


def _stream_ptr(stream) -> int | None:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


# ------------------------------------------------------------- entry points

def exq_status_string(status: int) -> str:
    return _status_name(status)


def exq_packed_bytes(K: int, N: int, widths, group_size: int = GROUP) -> int:
    w = np.ascontiguousarray(widths, dtype=np.uint8)
    return int(lib.exq_packed_bytes(K, N, group_size, _np_ptr(w)))


def exq_pack(W: np.ndarray, widths, group_size: int = GROUP):
    """Host quantize + pack.  W fp32 [N][K] -> (qweight uint8 bytes, scales fp16 bits uint16 [G][N])."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    w = np.ascontiguousarray(widths, dtype=np.uint8)
    nbytes = exq_packed_bytes(K, N, w, group_size)
    if nbytes == 0:
        _check(lib.exq_pack(_np_ptr(W), K, N, group_size, _np_ptr(w), None, None), "exq_pack")
    q = np.empty(nbytes, dtype=np.uint8)
    s = np.empty((K // group_size, N), dtype=np.uint16)
    _check(lib.exq_pack(_np_ptr(W), K, N, group_size, _np_ptr(w), _np_ptr(q), _np_ptr(s)), "exq_pack")
    return q, s


def exq_pack_qs(W: np.ndarray, widths, group_size: int = GROUP):
    """Host quantize + pack with quantized group scales.  W fp32 [N][K] ->
    (qweight uint8 bytes, 4-bit scale codes uint8 [G][N/2], column references fp16 bits uint16 [N])."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    w = np.ascontiguousarray(widths, dtype=np.uint8)
    nbytes = exq_packed_bytes(K, N, w, group_size)
    if nbytes == 0:
        _check(lib.exq_pack_qs(_np_ptr(W), K, N, group_size, _np_ptr(w), None, None, None), "exq_pack_qs")
    q = np.empty(nbytes, dtype=np.uint8)
    qs = np.empty((K // group_size, N // 2), dtype=np.uint8)
    ref = np.empty(N, dtype=np.uint16)
    _check(lib.exq_pack_qs(_np_ptr(W), K, N, group_size, _np_ptr(w), _np_ptr(q), _np_ptr(qs), _np_ptr(ref)),
           "exq_pack_qs")
    return q, qs, ref


def exq_layer_create_qs(K: int, N: int, widths, d_qweight: int, d_qscale: int, d_ref: int,
                        group_size: int = GROUP) -> int:
    w = np.ascontiguousarray(widths, dtype=np.uint8)
    h = ctypes.c_void_p()
    _check(lib.exq_layer_create_qs(K, N, group_size, _np_ptr(w), d_qweight, d_qscale, d_ref, ctypes.byref(h)),
           "exq_layer_create_qs")
    return h.value


def exq_layer_create(K: int, N: int, widths, d_qweight: int, d_scales: int, group_size: int = GROUP) -> int:
    w = np.ascontiguousarray(widths, dtype=np.uint8)
    h = ctypes.c_void_p()
    _check(lib.exq_layer_create(K, N, group_size, _np_ptr(w), d_qweight, d_scales, ctypes.byref(h)),
           "exq_layer_create")
    return h.value


def exq_layer_destroy(handle: int) -> None:
    lib.exq_layer_destroy(handle)


def exq_gemm(x_ptr: int, M: int, handle: int, y_ptr: int, stream=None) -> None:
    _check(lib.exq_gemm(x_ptr, M, handle, y_ptr, _stream_ptr(stream)), "exq_gemm")


def exq_gemm_noalloc(x_ptr: int, M: int, handle: int, y_ptr: int, stream=None) -> None:
    _check(lib.exq_gemm_noalloc(x_ptr, M, handle, y_ptr, _stream_ptr(stream)), "exq_gemm_noalloc")


def exq_gemm_gated(x_ptr: int, M: int, gate: int, up: int, h_ptr: int, stream=None) -> None:
    _check(lib.exq_gemm_gated(x_ptr, M, gate, up, h_ptr, _stream_ptr(stream)), "exq_gemm_gated")


def exq_group_errors(W: np.ndarray) -> np.ndarray:
    """Squared weight error of every group at every width: float64 [K/128][6] from W fp32 [N][K]."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    err = np.empty((K // 128, 6), dtype=np.float64)
    _check(lib.exq_group_errors(_np_ptr(W), K, N, 128, _np_ptr(err)), "exq_group_errors")
    return err


def exq_allocate_widths(err: np.ndarray, size, budget: int, min_width=None, seed: int = 0, iterations: int = 0):
    """(widths uint8 [G], total error) minimizing sum err[g][b_g] with sum b_g * size[g] <= budget."""
    err = np.ascontiguousarray(err, dtype=np.float64)
    G = err.shape[0]
    size = np.ascontiguousarray(np.broadcast_to(np.asarray(size, dtype=np.int32), (G,)))
    mw = None if min_width is None else np.ascontiguousarray(min_width, dtype=np.uint8)
    out = np.empty(G, dtype=np.uint8)
    total = ctypes.c_double()
    _check(lib.exq_allocate_widths(_np_ptr(err), _np_ptr(size), G, int(budget), None if mw is None else _np_ptr(mw),
                                   int(seed) & ((1 << 64) - 1), int(iterations), _np_ptr(out), ctypes.byref(total)),
           "exq_allocate_widths")
    return out, total.value


def exq_trimmed_mean(samples) -> float:
    s = np.ascontiguousarray(samples, dtype=np.float32)
    return lib.exq_trimmed_mean(_np_ptr(s), s.size)


def exq_autotune(x_ptr: int, M: int, handle: int, y_ptr: int, stream=None, warmup: int = 20, reps: int = 200):
    """(chosen variant, trimmed-mean microseconds per candidate from DECODE16 on)."""
    choice = ctypes.c_int()
    times = np.zeros(3, dtype=np.float32)
    _check(lib.exq_autotune(x_ptr, M, handle, y_ptr, _stream_ptr(stream), warmup, reps, ctypes.byref(choice),
                            _np_ptr(times)), "exq_autotune")
    return choice.value, times[: 3 if M > 16 else 2].tolist()


def exq_set_variant(handle: int, M: int, variant: int) -> None:
    _check(lib.exq_set_variant(handle, M, variant), "exq_set_variant")


def exq_dequant(handle: int, w_ptr: int, stream=None) -> None:
    _check(lib.exq_dequant(handle, w_ptr, _stream_ptr(stream)), "exq_dequant")


def exq_plan_create(handles, x_ptrs, y_ptrs, M: int) -> int:
    n = len(handles)
    H = (ctypes.c_void_p * n)(*handles)
    X = (ctypes.c_void_p * n)(*x_ptrs)
    Y = (ctypes.c_void_p * n)(*y_ptrs)
    p = ctypes.c_void_p()
    _check(lib.exq_plan_create(n, H, X, Y, M, ctypes.byref(p)), "exq_plan_create")
    return p.value


def exq_plan_run(plan: int, stream=None) -> None:
    _check(lib.exq_plan_run(plan, _stream_ptr(stream)), "exq_plan_run")


def exq_stream_read(buf_ptr: int, nbytes: int, sink_ptr: int, sink_words: int, stream=None) -> None:
    _check(lib.exq_stream_read(buf_ptr, nbytes, sink_ptr, sink_words, _stream_ptr(stream)), "exq_stream_read")


def exq_plan_destroy(plan: int) -> None:
    lib.exq_plan_destroy(plan)


def exq_cache_page_bytes(page_size: int, kv_heads: int, head_dim: int, k_bits: int, v_bits: int) -> int:
    return int(lib.exq_cache_page_bytes(page_size, kv_heads, head_dim, k_bits, v_bits))


def exq_cache_create(pages_ptr: int, n_pages: int, page_size: int, kv_heads: int, head_dim: int, k_bits: int,
                     v_bits: int) -> int:
    h = ctypes.c_void_p()
    _check(lib.exq_cache_create(pages_ptr, n_pages, page_size, kv_heads, head_dim, k_bits, v_bits, ctypes.byref(h)),
           "exq_cache_create")
    return h.value


def exq_cache_destroy(cache: int) -> None:
    lib.exq_cache_destroy(cache)


def exq_cache_append(cache: int, k_ptr: int, k_strides, v_ptr: int, v_strides, rows: int, table_ptr: int,
                     table_rows: int, table_width: int, table_stride: int, seqs_ptr: int, positions_ptr: int,
                     stream=None) -> None:
    """k_strides, v_strides: (row, head) in elements."""
    _check(lib.exq_cache_append(cache, k_ptr, k_strides[0], k_strides[1], v_ptr, v_strides[0], v_strides[1], rows,
                                table_ptr, table_rows, table_width, table_stride, seqs_ptr, positions_ptr,
                                _stream_ptr(stream)), "exq_cache_append")


def exq_cache_read(cache: int, k_ptr: int, k_strides, v_ptr: int, v_strides, rows: int, table_ptr: int,
                   table_rows: int, table_width: int, table_stride: int, seqs_ptr: int, positions_ptr: int,
                   stream=None) -> None:
    _check(lib.exq_cache_read(cache, k_ptr, k_strides[0], k_strides[1], v_ptr, v_strides[0], v_strides[1], rows,
                              table_ptr, table_rows, table_width, table_stride, seqs_ptr, positions_ptr,
                              _stream_ptr(stream)), "exq_cache_read")


def exq_attend_workspace_bytes(cache: int, rows: int, q_heads: int, table_width: int) -> int:
    return int(lib.exq_attend_workspace_bytes(cache, rows, q_heads, table_width))


def exq_attend(cache: int, q_ptr: int, q_strides, rows: int, q_heads: int, table_ptr: int, table_width: int,
               table_stride: int, lengths_ptr: int, scale: float, window: int, out_ptr: int, out_strides, lse_ptr=None,
               workspace_ptr=None, workspace_bytes: int = 0, stream=None) -> None:
    _check(lib.exq_attend(cache, q_ptr, q_strides[0], q_strides[1], rows, q_heads, table_ptr, table_width, table_stride,
                          lengths_ptr, scale, window, out_ptr, out_strides[0], out_strides[1], lse_ptr, workspace_ptr,
                          workspace_bytes, _stream_ptr(stream)), "exq_attend")


def exq_pages_workspace_bytes(sequences: int) -> int:
    return int(lib.exq_pages_workspace_bytes(sequences))


def exq_pages_extend(table_ptr: int, sequences: int, table_width: int, table_stride: int, page_size: int, lengths_ptr: int,
                     counts_ptr: int, free_ptr: int, free_count_ptr: int, n_pages: int, seqs_ptr: int, positions_ptr: int,
                     rows: int, offsets_ptr: int, served_ptr: int, workspace_ptr: int, workspace_bytes: int, stream=None) -> None:
    _check(lib.exq_pages_extend(table_ptr, sequences, table_width, table_stride, page_size, lengths_ptr, counts_ptr, free_ptr,
                                free_count_ptr, n_pages, seqs_ptr, positions_ptr, rows, offsets_ptr, served_ptr, workspace_ptr,
                                workspace_bytes, _stream_ptr(stream)), "exq_pages_extend")


def exq_pages_trim(table_ptr: int, sequences: int, table_width: int, table_stride: int, page_size: int, lengths_ptr: int,
                   keep_ptr: int, free_ptr: int, free_count_ptr: int, n_pages: int, workspace_ptr: int, workspace_bytes: int,
                   stream=None) -> None:
    _check(lib.exq_pages_trim(table_ptr, sequences, table_width, table_stride, page_size, lengths_ptr, keep_ptr, free_ptr,
                              free_count_ptr, n_pages, workspace_ptr, workspace_bytes, _stream_ptr(stream)), "exq_pages_trim")


def exq_rotate(q_ptr, q_strides, q_out_ptr, q_out_strides, q_heads: int, k_ptr, k_strides, k_out_ptr, k_out_strides,
               k_heads: int, rows: int, head_dim: int, rotary_dim: int, interleaved: bool, rates_ptr: int, factor: float,
               positions_ptr: int, stream=None) -> None:
    """Strides: (row, head) in elements."""
    _check(lib.exq_rotate(q_ptr, q_strides[0], q_strides[1], q_out_ptr, q_out_strides[0], q_out_strides[1], q_heads, k_ptr,
                          k_strides[0], k_strides[1], k_out_ptr, k_out_strides[0], k_out_strides[1], k_heads, rows, head_dim,
                          rotary_dim, int(interleaved), rates_ptr, factor, positions_ptr, _stream_ptr(stream)), "exq_rotate")


def exq_adapters_create(count: int, K: int, N: int, rank: int, a_ptr: int, b_ptr: int, scales_ptr=None, ranks_ptr=None) -> int:
    h = ctypes.c_void_p()
    _check(lib.exq_adapters_create(count, K, N, rank, a_ptr, b_ptr, scales_ptr, ranks_ptr, ctypes.byref(h)),
           "exq_adapters_create")
    return h.value


def exq_adapters_destroy(adapters: int) -> None:
    lib.exq_adapters_destroy(adapters)


def exq_lora_workspace_bytes(adapters: int, rows: int) -> int:
    return int(lib.exq_lora_workspace_bytes(adapters, rows))


def exq_lora_add(adapters: int, x_ptr: int, x_stride: int, rows: int, ids_ptr: int, y_ptr: int, y_stride: int, out_ptr: int,
                 out_stride: int, workspace_ptr: int, workspace_bytes: int, stream=None) -> None:
    _check(lib.exq_lora_add(adapters, x_ptr, x_stride, rows, ids_ptr, y_ptr, y_stride, out_ptr, out_stride, workspace_ptr,
                            workspace_bytes, _stream_ptr(stream)), "exq_lora_add")


def exq_sample_workspace_bytes(rows: int, vocab: int) -> int:
    return int(lib.exq_sample_workspace_bytes(rows, vocab))


def exq_sample(logits_ptr: int, bits: int, rows: int, vocab: int, row_stride: int, u_ptr: int, temperatures_ptr,
               temperature: float, top_ks_ptr, top_k: int, top_ps_ptr, top_p: float, min_ps_ptr, min_p: float, tokens_ptr: int,
               logprobs_ptr=None, workspace_ptr=None, workspace_bytes: int = 0, stream=None) -> None:
    _check(lib.exq_sample(logits_ptr, bits, rows, vocab, row_stride, u_ptr, temperatures_ptr, temperature, top_ks_ptr, top_k,
                          top_ps_ptr, top_p, min_ps_ptr, min_p, tokens_ptr, logprobs_ptr, workspace_ptr, workspace_bytes,
                          _stream_ptr(stream)), "exq_sample")


# ------------------------------------------------------------ conveniences

def _tensor_calls():
    """The module of the calls on tensors, which checks them and passes them to the library."""
    if not os.path.exists(os.path.join(_PKG, "_exq_torch.so")):
        from . import build as _b
        _b.build()
    from . import _exq_torch
    _exq_torch.set_error(ExqError)
    return _exq_torch


def _on(stream, device):
    """What a call runs under when it names a stream or its tensors' device is not the current one: that device and, for
    what the call allocates, that stream."""
    import torch
    if hasattr(stream, "cuda_stream") and getattr(stream, "device", device) != device:
        raise ExqError(EXQ_ERR_INVALID_ARG, "argument check", "a stream of %s for tensors on %s" % (stream.device, device))
    scope = contextlib.ExitStack()
    scope.enter_context(torch.cuda.device(device))
    if stream is not None:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        scope.enter_context(torch.cuda.stream(stream))
    return scope


def _call_on(stream, device, call, *args, own=()):
    """call(*args) under `stream` and `device`.  The tensors among args, and those that the called object keeps (`own`), may
    belong to another stream: they stay allocated until the named one is through with the call, also if the caller drops them
    before.  (Not for the handle of a stream that is not PyTorch's: its owner may destroy it before the tensors are dropped, and
    PyTorch would still wait for it then.)"""
    import torch
    with _on(stream, device):
        result = call(*args)
        if isinstance(stream, torch.cuda.Stream) and not isinstance(stream, torch.cuda.ExternalStream):
            for x in (*args, *own):
                if isinstance(x, torch.Tensor) and x.device == device:
                    x.record_stream(stream)
    return result


class Layer:
    """A packed layer resident on the GPU: owns its torch buffers and the handle."""

    def __init__(self, K: int, N: int, widths, qweight: np.ndarray, scales: np.ndarray, device="cuda", ref=None):
        """fp16 scales [G][N]; or, with `ref` (fp16 bits [N]), 4-bit scale codes [G][N/2] in `scales`."""
        import torch
        self.K, self.N = K, N
        self.widths = np.ascontiguousarray(widths, dtype=np.uint8)
        self.qweight = torch.from_numpy(np.ascontiguousarray(qweight)).to(device)
        if ref is None:
            self.scales = torch.from_numpy(np.ascontiguousarray(scales).view(np.int16)).to(device)
            self.ref = None
            self.handle = exq_layer_create(K, N, self.widths, self.qweight.data_ptr(), self.scales.data_ptr())
        else:
            self.scales = torch.from_numpy(np.ascontiguousarray(scales, dtype=np.uint8)).to(device)
            self.ref = torch.from_numpy(np.ascontiguousarray(ref).view(np.int16)).to(device)
            self.handle = exq_layer_create_qs(K, N, self.widths, self.qweight.data_ptr(), self.scales.data_ptr(),
                                              self.ref.data_ptr())

    @classmethod
    def from_weight(cls, W: np.ndarray, widths, device="cuda", quantized_scales: bool = False):
        N, K = W.shape
        if quantized_scales:
            q, qs, ref = exq_pack_qs(W, widths)
            return cls(K, N, widths, q, qs, device, ref=ref)
        q, s = exq_pack(W, widths)
        return cls(K, N, widths, q, s, device)

    @property
    def packed_bytes(self) -> int:
        return int(self.qweight.numel())

    def gemm(self, x, out=None, stream=None):
        """x: torch fp16 [M][K] on the GPU -> y fp16 [M][N]."""
        import torch
        assert x.dtype == torch.float16 and x.is_contiguous() and x.shape[-1] == self.K
        M = x.shape[0]
        if out is None:
            out = torch.empty((M, self.N), dtype=torch.float16, device=x.device)
        exq_gemm(x.data_ptr(), M, self.handle, out.data_ptr(), stream)
        return out

    def dequant(self, stream=None):
        import torch
        w = torch.empty((self.K, self.N), dtype=torch.float16, device=self.qweight.device)
        exq_dequant(self.handle, w.data_ptr(), stream)
        return w

    def close(self):
        if self.handle:
            exq_layer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gemm_gated(x, gate: "Layer", up: "Layer", out=None, stream=None):
    """x: torch fp16 [M][K] on the GPU -> h = SiLU(x gate^T) * (x up^T), fp16 [M][N]."""
    import torch
    assert x.dtype == torch.float16 and x.is_contiguous() and x.shape[-1] == gate.K
    M = x.shape[0]
    if out is None:
        out = torch.empty((M, gate.N), dtype=torch.float16, device=x.device)
    exq_gemm_gated(x.data_ptr(), M, gate.handle, up.handle, out.data_ptr(), stream)
    return out


class Plan:
    """Independent linears bound to fixed x/y buffers, run as one launch."""

    def __init__(self, layers, xs, ys, M: int):
        self.layers, self.xs, self.ys = list(layers), list(xs), list(ys)  # keep buffers alive
        self.handle = exq_plan_create([l.handle for l in self.layers], [x.data_ptr() for x in self.xs],
                                      [y.data_ptr() for y in self.ys], M)

    def run(self, stream=None):
        exq_plan_run(self.handle, stream)

    def close(self):
        if self.handle:
            exq_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


ATTEND_COUNTER_BYTES = 16384   # EXQ_ATTEND_COUNTER_BYTES


class KVCache:
    """A paged key-value cache on the GPU: owns (or borrows) its pages and the handle.

    K and V are held in `k_bits` and `v_bits` bits (each 4 or 8, or both 16).  `table` is int32 [sequences][width] and
    names each sequence's pages; position p of sequence s lies in page table[s][p // page_size].  Every call runs on
    `stream` (default: the current stream of the cache's device) and may be captured; all tensors are on that device.  Calls
    on different streams run side by side: order a read or attend after the append that it needs, and drop the cache after
    the last of them.  A call that names a torch.cuda.Stream keeps its tensors' memory until that stream is through
    with them (with another stream's handle the caller keeps them), and what it allocates belongs to that stream.
    """

    def __init__(self, n_pages: int, page_size: int, kv_heads: int, head_dim: int, k_bits: int = 4, v_bits: int = 4,
                 device="cuda", pages=None):
        """`pages`: uint8 [n_pages][page_bytes], contiguous, any content (default: allocated and zeroed, which is waited for)."""
        import torch
        self.handle = None
        page_bytes = exq_cache_page_bytes(page_size, kv_heads, head_dim, k_bits, v_bits)
        if page_bytes == 0:   # let the library say what is wrong
            exq_cache_create(None, n_pages, page_size, kv_heads, head_dim, k_bits, v_bits)
        if pages is None:
            pages = torch.zeros((n_pages, page_bytes), dtype=torch.uint8, device=device)
            if pages.is_cuda:   # the first append may come on any stream
                torch.cuda.current_stream(pages.device).synchronize()
        if not (pages.dtype is torch.uint8 and pages.is_contiguous() and pages.is_cuda
                and pages.numel() == n_pages * page_bytes):
            raise ExqError(EXQ_ERR_INVALID_ARG, "argument check",
                           "pages must be contiguous uint8 of %d x %d bytes on the GPU" % (n_pages, page_bytes))
        self.pages, self.n_pages, self.page_size, self.page_bytes = pages, n_pages, page_size, page_bytes
        self.kv_heads, self.head_dim, self.k_bits, self.v_bits = kv_heads, head_dim, k_bits, v_bits
        self.device, self._index = pages.device, pages.device.index
        self._torch, self._C, self._calls = torch, torch._C, _tensor_calls()
        self._scale = head_dim ** -0.5
        self._workspaces = {}   # by stream: calls on one stream run one after another
        self.handle = exq_cache_create(pages.data_ptr(), n_pages, page_size, kv_heads, head_dim, k_bits, v_bits)

    def append(self, k, v, table, seqs, positions, stream=None):
        """Store rows k, v (fp16 [rows][kv_heads][head_dim]) at positions[r] of sequence seqs[r] (int32 [rows]; < 0: skipped)."""
        index, C = self._index, self._C
        if stream is not None or C._cuda_getDevice() != index:
            return _call_on(stream, self.device, self.append, k, v, table, seqs, positions)
        self._calls.append(self.handle, self.kv_heads, self.head_dim, index, C._cuda_getCurrentRawStream(index), k, v, table,
                           seqs, positions)

    def read(self, table, seqs, positions, k_out=None, v_out=None, stream=None):
        """The values held for positions[r] of sequence seqs[r]: fp16 k, v [rows][kv_heads][head_dim].

        Rows with seqs[r] < 0 are left as they were in k_out and v_out (in tensors allocated here: unspecified)."""
        index, C = self._index, self._C
        if stream is not None or C._cuda_getDevice() != index:
            return _call_on(stream, self.device, self.read, table, seqs, positions, k_out, v_out)
        return self._calls.read(self.handle, self.kv_heads, self.head_dim, index, C._cuda_getCurrentRawStream(index), table,
                                seqs, positions, k_out, v_out)

    def workspace(self, nbytes: int):
        """A workspace for attend calls that need up to `nbytes` (exq_attend_workspace_bytes), to pass where calls must not
        share the cache's own: its counters are zeroed on the current stream."""
        torch = self._torch
        ws = torch.empty(max(nbytes, ATTEND_COUNTER_BYTES), dtype=torch.uint8, device=self.device)
        ws[:ATTEND_COUNTER_BYTES].view(torch.int32).zero_()
        return ws

    def attend(self, q, table, lengths, scale=None, window: int = 0, out=None, return_lse: bool = False, lse=None,
               workspace=None, stream=None):
        """Attention of one query token per row: q fp16 [rows][q_heads][head_dim] over the first lengths[r] tokens of
        table row r (the last `window` of them if window > 0) -> out, or (out, lse fp32 [rows][q_heads]).

        scale: default head_dim ** -0.5.  lengths[r] == 0 gives zeros (lse -inf); < 0 leaves the row as it was.
        workspace: from workspace(); by default the cache keeps one for each stream, and a call under graph capture makes
        one that belongs to the graph."""
        index, C = self._index, self._C
        if stream is not None or C._cuda_getDevice() != index:
            return _call_on(stream, self.device, self.attend, q, table, lengths, scale, window, out, return_lse, lse, workspace)
        raw = C._cuda_getCurrentRawStream(index)
        capturing = C._cuda_isCurrentStreamCapturing()
        if scale is None:
            scale = self._scale
        result = self._calls.attend(self.handle, self.kv_heads, self.head_dim, index, raw, q, table, lengths, scale, window, out,
                                    return_lse, lse, workspace, None if capturing else self._workspaces.get(raw))
        if type(result) is int:   # a call that splits its rows, and no workspace of that many bytes yet
            workspace = self.workspace(result)
            if not capturing:
                self._workspaces[raw] = workspace
            result = self._calls.attend(self.handle, self.kv_heads, self.head_dim, index, raw, q, table, lengths, scale, window,
                                        out, return_lse, lse, workspace, None)
        return result

    def close(self):
        if self.handle:
            exq_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagePool:
    """The pages of a KVCache, handed out to sequences and taken back on the GPU.

    Owns `table` (int32 [sequences][width], -1 where there is no page), `lengths` (int32 [sequences]), and the list of free
    pages (`free`, `free_count`).  extend() makes room for new tokens and says where they go; trim() cuts sequences; nothing is
    read back.  table and lengths are what KVCache's calls take.  Every call runs on `stream` (default: the current stream of
    the pool's device) and may be captured; calls on one pool, and what reads its tensors, are ordered by the caller.  A call
    that names a torch.cuda.Stream keeps its tensors' memory and the pool's until that stream is through with them; otherwise
    drop the pool, like any tensor, after the last call on another stream than its own, and after the graphs that hold calls.
    """

    def __init__(self, n_pages: int, page_size: int, sequences: int, width: int, device="cuda"):
        import torch
        if not (0 < n_pages < 1 << 31 and 0 < page_size <= 65536 and 0 < sequences and 0 < width
                and sequences * width < 1 << 31):
            raise ExqError(EXQ_ERR_INVALID_ARG, "argument check", "%d pages of %d tokens for %d sequences of %d pages"
                           % (n_pages, page_size, sequences, width))
        self.n_pages, self.page_size, self.sequences, self.width = n_pages, page_size, sequences, width
        self.table = torch.full((sequences, width), -1, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(sequences, dtype=torch.int32, device=device)
        self.free = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=device)
        self.free_count = torch.full((1,), n_pages, dtype=torch.int32, device=device)
        self.served = torch.full((1,), sequences, dtype=torch.int32, device=device)
        self._workspace = torch.empty(exq_pages_workspace_bytes(sequences) // 4, dtype=torch.int32, device=device)
        self.device, self._index = self.table.device, self.table.device.index
        self._C, self._calls = torch._C, _tensor_calls()
        if self.table.is_cuda:   # the first call may come on any stream
            torch.cuda.current_stream(self.device).synchronize()

    def _own(self):
        return self.table, self.lengths, self.free, self.free_count, self.served, self._workspace

    def extend(self, counts, rows: int, seqs=None, positions=None, offsets=None, stream=None):
        """Make room for counts[s] (int32 [sequences]) more tokens of every sequence -> (seqs, positions, offsets): for row r of
        `rows` its sequence (-1 behind the last) and position, and for sequence s its first row offsets[s].

        Where pages, rows or the table's width do not suffice, the first sequence concerned and all after it get nothing;
        `served` (int32 [1]) tells how many were served.  New outputs are chunks of one allocation."""
        index, C = self._index, self._C
        if stream is not None or C._cuda_getDevice() != index:
            return _call_on(stream, self.device, self.extend, counts, rows, seqs, positions, offsets, own=self._own())
        return self._calls.extend(index, C._cuda_getCurrentRawStream(index), self.page_size, self.table, self.lengths, self.free,
                                  self.free_count, self.served, self._workspace, counts, rows, seqs, positions, offsets)

    def trim(self, keep, stream=None):
        """Cut every sequence s to its first keep[s] tokens (int32 [sequences]; 0 releases it, negative leaves it as it is)."""
        index, C = self._index, self._C
        if stream is not None or C._cuda_getDevice() != index:
            return _call_on(stream, self.device, self.trim, keep, own=self._own())
        self._calls.trim(index, C._cuda_getCurrentRawStream(index), self.page_size, self.table, self.lengths, self.free,
                         self.free_count, self._workspace, keep)


def rotary_rates(rotary_dim: int, base: float = 10000.0, scaling=None):
    """(angles per token of each pair as a list of rotary_dim / 2, factor of the turned channels).

    Pair i turns by base ** (-2 i / rotary_dim) a token.  `scaling` stretches that for contexts longer than the trained one:
      {"kind": "linear", "factor": s}   positions divided by s;
      {"kind": "base", "factor": s}     the base times s ** (d / (d - 2)), d = rotary_dim: the slowest pair is stretched by s;
      {"kind": "parts", "factor": s, "context": c, "low": 1, "high": 32, "attention": None}
          pairs by the number of turns they make in the trained context of c tokens: below `low` divided by s, above
          `high` as they are, a mixture between; and the channels times `attention` (None: 0.1 ln s + 1).
          The mixture is linear in the number of turns.  Where a model was stretched with one that is linear in the pair's
          index, between bounds rounded to whole pairs, give Rotary those `rates`.
    """
    if rotary_dim < 2 or rotary_dim % 2 or not base > 0:
        raise ExqError(EXQ_ERR_INVALID_ARG, "argument check", "rotary_dim=%d base=%r" % (rotary_dim, base))
    given = dict(scaling or {"kind": "none"})
    kind = given.pop("kind", None)
    allowed = {"none": (), "linear": ("factor",), "base": ("factor",), "parts": ("factor", "context", "low", "high", "attention")}
    if kind not in allowed or not set(given) <= set(allowed[kind]):
        raise ExqError(EXQ_ERR_INVALID_ARG, "argument check", "scaling %r" % (scaling,))
    s, factor = float(given.get("factor", 1.0)), 1.0
    if not 0 < s < math.inf:
        raise ExqError(EXQ_ERR_INVALID_ARG, "argument check", "scaling factor %r" % s)
    if kind == "base" and rotary_dim > 2:
        base = base * s ** (rotary_dim / (rotary_dim - 2))
    rates = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if kind == "linear" or (kind == "base" and rotary_dim == 2):
        rates = [f / s for f in rates]
    elif kind == "parts":
        if "context" not in given:
            raise ExqError(EXQ_ERR_INVALID_ARG, "argument check", "scaling by parts needs the trained context")
        low, high = float(given.get("low", 1.0)), float(given.get("high", 32.0))
        if not low < high:
            raise ExqError(EXQ_ERR_INVALID_ARG, "argument check", "low=%r high=%r" % (low, high))
        keep = [min(1.0, max(0.0, (given["context"] * f / (2 * math.pi) - low) / (high - low))) for f in rates]
        rates = [(1 - g) * f / s + g * f for f, g in zip(rates, keep)]
        attention = given.get("attention")
        factor = 0.1 * math.log(s) + 1.0 if attention is None else float(attention)
    return rates, factor


class Rotary:
    """Rotary positions of a model's heads: the angles of its pairs of channels on the GPU.

    rotary_dim: the channels that turn (default: all); interleaved: pairs are neighbours, else halves apart; base and
    scaling: rotary_rates.  Or `rates` (angles per token, one a pair) and `factor` directly.  A call that names a
    torch.cuda.Stream keeps its tensors' memory and the rates' until that stream is through with them; otherwise drop the
    object, like any tensor, after the last call on another stream than its own, and after the graphs that hold calls."""

    def __init__(self, head_dim: int, rotary_dim=None, base: float = 10000.0, interleaved: bool = False, scaling=None, rates=None,
                 factor=None, device="cuda"):
        import torch
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        if rates is None:
            rates, scaled = rotary_rates(rotary_dim, base, scaling)
            factor = scaled if factor is None else factor
        elif scaling is not None:
            raise ExqError(EXQ_ERR_INVALID_ARG, "argument check", "rates and scaling")
        rates = torch.as_tensor(rates, dtype=torch.float64).to(device).contiguous().clone()
        if rates.dim() != 1 or 2 * rates.numel() != rotary_dim:
            raise ExqError(EXQ_ERR_INVALID_ARG, "argument check", "%d rates for %d channels" % (rates.numel(), rotary_dim))
        self.head_dim, self.rotary_dim, self.interleaved = head_dim, rotary_dim, bool(interleaved)
        self.rates, self.factor = rates, float(1.0 if factor is None else factor)
        self.device, self._index = rates.device, rates.device.index
        self._C, self._calls = torch._C, _tensor_calls()
        if rates.is_cuda:   # the first call may come on any stream
            torch.cuda.current_stream(self.device).synchronize()

    def rotate(self, q, positions, k=None, q_out=None, k_out=None, stream=None):
        """q (fp16 [rows][heads][head_dim]), and k if given, turned by positions (int32 [rows]; < 0: left as it was in the
        output) -> q_out, or (q_out, k_out), new ones as chunks of one allocation.  An output may be its input."""
        index, C = self._index, self._C
        if stream is not None or C._cuda_getDevice() != index:
            return _call_on(stream, self.device, self.rotate, q, positions, k, q_out, k_out, own=(self.rates,))
        return self._calls.rotate(index, C._cuda_getCurrentRawStream(index), self.head_dim, self.rotary_dim, self.interleaved,
                                  self.rates, self.factor, q, positions, k, q_out, k_out)


class Adapters:
    """Low-rank adapters of one linear: a fp16 [count][rank][K], b fp16 [count][N][rank], contiguous on the GPU (kept, not
    copied).  scales: fp32 [count]; ranks: int32 [count], where adapters have fewer than the stack's.  A call that names a
    torch.cuda.Stream keeps its tensors' memory and the adapters' until that stream is through with them; otherwise drop the
    adapters, like any tensor, after the last call on another stream than their own, and after the graphs that hold calls."""

    def __init__(self, a, b, scales=None, ranks=None):
        import torch
        self.handle = None
        count = a.shape[0] if a.dim() == 3 else 0
        fits = (a.dim() == 3 and b.dim() == 3 and b.shape[0] == count and b.shape[2] == a.shape[1]
                and all(x.is_cuda and x.is_contiguous() and x.device == a.device for x in (a, b, scales, ranks) if x is not None)
                and a.dtype is torch.float16 and b.dtype is torch.float16
                and (scales is None or (scales.dtype is torch.float32 and tuple(scales.shape) == (count,)))
                and (ranks is None or (ranks.dtype is torch.int32 and tuple(ranks.shape) == (count,))))
        if not fits:
            raise ExqError(EXQ_ERR_INVALID_ARG, "argument check", "a must be fp16 [count][rank][K], b fp16 [count][N][rank], scales "
                           "fp32 [count] and ranks int32 [count], contiguous on one GPU")
        self.a, self.b, self.scales, self.ranks = a, b, scales, ranks
        self.count, self.rank, self.K = a.shape
        self.N = b.shape[1]
        self.device, self._index = a.device, a.device.index
        self._C, self._calls = torch._C, _tensor_calls()
        self.handle = exq_adapters_create(self.count, self.K, self.N, self.rank, a.data_ptr(), b.data_ptr(),
                                          None if scales is None else scales.data_ptr(), None if ranks is None else ranks.data_ptr())

    def add(self, x, ids, y, out=None, workspace=None, stream=None):
        """out = y + scales[i] (x a[i]^T) b[i]^T with i = ids[row] (int32 [rows]; < 0: none): x fp16 [rows][K], y fp16
        [rows][N].  `out` may be y.  workspace: uint8, exq_lora_workspace_bytes() of them (default: allocated)."""
        index, C = self._index, self._C
        if stream is not None or C._cuda_getDevice() != index:
            return _call_on(stream, self.device, self.add, x, ids, y, out, workspace,
                            own=(self.a, self.b, self.scales, self.ranks))
        return self._calls.lora_add(index, C._cuda_getCurrentRawStream(index), self.handle, self.K, self.N, x, ids, y, out,
                                    workspace)

    def close(self):
        if self.handle:
            exq_adapters_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_sample = None


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None, return_logprobs: bool = False, logprobs=None,
           stream=None):
    """One token of every row of logits (fp16 or fp32 [rows][vocab]) from random numbers u (fp32 [rows], in [0, 1)).

    temperature, top_p, min_p: a number, or fp32 [rows]; top_k: a number, or int32 [rows] (0: off).  Filters apply in the
    order top-k, top-p, min-p (include/exq.h) -> tokens int32 [rows], or (tokens, logprobs fp32 [rows]) with the logarithm of
    the probability each was drawn with; new ones are chunks of one allocation.  A row with u < 0 is left as it was; one
    without a token to draw gets -1.  Runs on
    `stream` (default: the current stream of the logits' device) and may be captured."""
    global _sample
    if _sample is None:
        import torch
        _sample = (torch, torch._C, _tensor_calls())
    torch, C, calls = _sample
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda:
        raise ExqError(EXQ_ERR_INVALID_ARG, "argument check", "logits must be a tensor on the GPU")
    index = logits.get_device()
    if stream is not None or C._cuda_getDevice() != index:
        return _call_on(stream, logits.device, sample, logits, u, temperature, top_k, top_p, min_p, out, return_logprobs, logprobs)
    return calls.sample(index, C._cuda_getCurrentRawStream(index), logits, u, temperature, top_k, top_p, min_p, out,
                        return_logprobs, logprobs)
