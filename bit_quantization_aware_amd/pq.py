"""Thin Python binding of libpq (the C ABI in include/pq.h).

Argument marshalling only: every function here turns torch tensors into
device pointers and calls the C entry point of the same name; all of the
computation runs in libpq's HIP kernels.  Importing this module loads
``libpq.so`` and raises if it has not been built -- there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpq.so")

PQ_W1_BINARY, PQ_W158_SEQ_TERNARY, PQ_W2_SEQ, PQ_W3_LSQ, PQ_W4_LSQ = 0, 1, 2, 3, 4
PQ_W2_LSQ, PQ_W158_LSQ = 5, 6  # the LSQ ablation grids at 2 and 1.58 bits
MODES = (PQ_W1_BINARY, PQ_W158_SEQ_TERNARY, PQ_W2_SEQ, PQ_W3_LSQ, PQ_W4_LSQ, PQ_W2_LSQ, PQ_W158_LSQ)
MODE_NAMES = {PQ_W1_BINARY: "w1_binary", PQ_W158_SEQ_TERNARY: "w1.58_ternary",
              PQ_W2_SEQ: "w2_seq", PQ_W3_LSQ: "w3_lsq", PQ_W4_LSQ: "w4_lsq", PQ_W2_LSQ: "w2_lsq",
              PQ_W158_LSQ: "w1.58_lsq"}
CODE_BITS = {PQ_W1_BINARY: 1, PQ_W158_SEQ_TERNARY: 2, PQ_W2_SEQ: 2, PQ_W3_LSQ: 4, PQ_W4_LSQ: 4,
             PQ_W2_LSQ: 2, PQ_W158_LSQ: 2}
PQ_INIT_ALPHA = 1
PQ_G_F32, PQ_G_BF16 = 0, 1
STATUS = {0: "PQ_OK", 1: "PQ_ERR_NULL", 2: "PQ_ERR_SHAPE", 3: "PQ_ERR_MODE", 4: "PQ_ERR_ALIGN",
          5: "PQ_ERR_UNSUPPORTED", 6: "PQ_ERR_HIP", 7: "PQ_ERR_ARG"}

# Every symbol include/pq.h declares.
EXPORTS = ("pq_code_row_bytes", "pq_packed_bytes", "pq_default_grad_scale", "pq_status_str", "pq_version",
           "pq_gemm_workspace_bytes",
           "pq_quantize_fwd", "pq_quantize_bwd", "pq_pack_w2", "pq_pack_w4", "pq_w2a16_gemm",
           "pq_w4a16_gemm", "pq_quantize_fwd_grouped", "pq_quantize_bwd_grouped", "pq_qat_step",
           "pq_qat_step_grouped", "pq_pack", "pq_gemm", "pq_gemm_f32a", "pq_num_levels", "pq_level_stats",
           "pq_quantize_fwd_stats", "pq_weight_movement", "pq_pack_grouped", "pq_gemm_noalloc",
           "pq_rope_table", "pq_rope", "pq_kv_row_bytes", "pq_kv_append", "pq_kv_load",
           "pq_attn_decode_workspace_bytes", "pq_attn_decode")


class PQError(RuntimeError):
    def __init__(self, status: int, fn: str):
        super().__init__(f"{fn}: {STATUS.get(status, status)}")
        self.status = status


class pq_mat(ctypes.Structure):
    """Mirror of `struct pq_mat` in include/pq.h."""
    _fields_ = [("W", ctypes.c_void_p), ("alpha", ctypes.c_void_p), ("wq_bf16", ctypes.c_void_p),
                ("wq_f32", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("G", ctypes.c_void_p),
                ("dW", ctypes.c_void_p), ("dalpha", ctypes.c_void_p), ("mask_bits", ctypes.c_void_p),
                ("grad_scale", ctypes.c_double), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("alpha_bf16", ctypes.c_void_p)]


class pq_adamw(ctypes.Structure):
    """Mirror of `struct pq_adamw` in include/pq.h."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64)]


class pq_step_mat(ctypes.Structure):
    """Mirror of `struct pq_step_mat` in include/pq.h."""
    _fields_ = [("W", ctypes.c_void_p), ("alpha", ctypes.c_void_p), ("G", ctypes.c_void_p),
                ("mW", ctypes.c_void_p), ("vW", ctypes.c_void_p), ("m_alpha", ctypes.c_void_p),
                ("v_alpha", ctypes.c_void_p), ("wq_bf16", ctypes.c_void_p), ("codes", ctypes.c_void_p),
                ("dalpha", ctypes.c_void_p), ("grad_scale", ctypes.c_double), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


class pq_rope_scaling(ctypes.Structure):
    """Mirror of `struct pq_rope_scaling` in include/pq.h."""
    _fields_ = [("kind", ctypes.c_int32), ("reserved", ctypes.c_int32), ("factor", ctypes.c_double),
                ("trained", ctypes.c_double), ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double)]


class pq_kv_cache(ctypes.Structure):
    """Mirror of `struct pq_kv_cache` in include/pq.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_param", ctypes.c_void_p),
                ("v_param", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("format", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
    L = ctypes.CDLL(LIB_PATH)
    i64, vp, u32, dbl = ctypes.c_int64, ctypes.c_void_p, ctypes.c_uint, ctypes.c_double
    i32 = ctypes.c_int
    L.pq_code_row_bytes.argtypes = [i32, i64]
    L.pq_code_row_bytes.restype = i64
    L.pq_packed_bytes.argtypes = [i32, i64, i64]
    L.pq_packed_bytes.restype = i64
    L.pq_default_grad_scale.argtypes = [i32, i64, i64]
    L.pq_default_grad_scale.restype = dbl
    L.pq_status_str.argtypes = [i32]
    L.pq_status_str.restype = ctypes.c_char_p
    L.pq_version.restype = ctypes.c_char_p
    L.pq_quantize_fwd.argtypes = [i32, i64, i64, vp, vp, u32, vp, vp, vp, vp]
    L.pq_quantize_bwd.argtypes = [i32, i64, i64, vp, vp, vp, i32, dbl, vp, vp, vp, vp]
    L.pq_pack_w2.argtypes = [i64, i64, vp, vp, vp, vp, vp]
    L.pq_pack_w4.argtypes = [i64, i64, vp, vp, vp, vp, vp]
    L.pq_gemm_workspace_bytes.argtypes = [i32, i64, i64, i64]
    L.pq_gemm_workspace_bytes.restype = i64
    L.pq_w2a16_gemm.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp, i64, vp]
    L.pq_w4a16_gemm.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp, i64, vp]
    L.pq_pack.argtypes = [i32, i64, i64, vp, vp, vp, vp, vp]
    L.pq_gemm.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp, vp, i64, vp]
    L.pq_gemm_f32a.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp, vp, i64, vp]
    L.pq_gemm_noalloc.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp, vp]
    L.pq_num_levels.argtypes = [i32]
    L.pq_num_levels.restype = i32
    L.pq_level_stats.argtypes = [i32, i64, i64, vp, vp, vp, vp]
    L.pq_quantize_fwd_stats.argtypes = [i32, i64, i64, vp, vp, vp, vp, vp, vp, vp]
    L.pq_weight_movement.argtypes = [i64, i64, vp, vp, vp, vp, vp]
    L.pq_quantize_fwd_grouped.argtypes = [i32, i32, vp, vp, u32, vp]
    L.pq_quantize_bwd_grouped.argtypes = [i32, i32, vp, vp, i32, vp]
    L.pq_pack_grouped.argtypes = [i32, i32, vp, vp, vp]
    L.pq_qat_step.argtypes = [i32, i64, i64, vp, vp, vp, i32, dbl, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.pq_qat_step_grouped.argtypes = [i32, i32, vp, vp, i32, vp, vp]
    L.pq_rope_table.argtypes = [i64, i64, dbl, vp, vp, vp]
    L.pq_rope.argtypes = [i32, i64, i64, i64, i64, i32, i32, vp, i64, i64, vp, vp, i64, vp, i64, i64, vp]
    L.pq_kv_row_bytes.argtypes = [i32, i64]
    L.pq_kv_row_bytes.restype = i64
    L.pq_kv_append.argtypes = [vp, i32, i64, vp, i64, i64, vp, i64, i64, vp, vp, vp, i64, i64, i32,
                               vp, i64, i64, i64, vp, i64, i64, vp]
    L.pq_kv_load.argtypes = [vp, i32, i64, i64, vp, i64, i64, vp, vp, vp, i64, i64, vp, i64, i64, vp]
    L.pq_attn_decode_workspace_bytes.argtypes = [vp, i64, i64]
    L.pq_attn_decode_workspace_bytes.restype = i64
    L.pq_attn_decode.argtypes = [vp, i32, i64, i64, vp, i64, i64, vp, i64, i64, vp, dbl, i64, i64, vp, i64, i64,
                                 vp, vp, i64, vp]
    for name in EXPORTS:
        if name not in ("pq_kv_row_bytes", "pq_attn_decode_workspace_bytes", "pq_code_row_bytes", "pq_packed_bytes", "pq_default_grad_scale", "pq_status_str",
                        "pq_version", "pq_num_levels", "pq_gemm_workspace_bytes"):
            getattr(L, name).restype = i32
    return L


lib = _load()


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# torch's own accessors of the current stream's handle: current_stream() makes
# a Stream object first, 2.8 us against 0.3, as much as the launch itself.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _current_raw_stream is not None and torch.cuda.is_initialized():
            return _current_raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _memory_of(stream):
    """Where a buffer that a call on `stream` makes for itself comes from: the
    launch stream's own memory.  A block of the caller's current stream may
    have been freed there with work still queued on it, and nothing makes the
    launch stream wait for that work; one of the launch stream is handed out
    again only behind the call, in the stream's order."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _check(rc: int, fn: str) -> None:
    if rc != 0:
        raise PQError(rc, fn)


def pq_code_row_bytes(mode: int, cols: int) -> int:
    return int(lib.pq_code_row_bytes(mode, cols))


def pq_packed_bytes(mode: int, rows: int, cols: int) -> int:
    return int(lib.pq_packed_bytes(mode, rows, cols))


def pq_default_grad_scale(mode: int, rows: int, cols: int) -> float:
    return float(lib.pq_default_grad_scale(mode, rows, cols))


def pq_status_str(status: int) -> str:
    return lib.pq_status_str(status).decode()


def pq_version() -> str:
    return lib.pq_version().decode()


def pq_quantize_fwd(mode, rows, cols, W, alpha, flags=0, Wq_bf16=None, Wq_f32=None, codes=None,
                    stream=None) -> None:
    _check(lib.pq_quantize_fwd(mode, rows, cols, _ptr(W), _ptr(alpha), flags, _ptr(Wq_bf16),
                               _ptr(Wq_f32), _ptr(codes), _stream(stream)), "pq_quantize_fwd")


def pq_quantize_bwd(mode, rows, cols, W, alpha, G, g_dtype, grad_scale, dW, dalpha,
                    mask_bits=None, stream=None) -> None:
    _check(lib.pq_quantize_bwd(mode, rows, cols, _ptr(W), _ptr(alpha), _ptr(G), g_dtype,
                               float(grad_scale), _ptr(dW), _ptr(dalpha), _ptr(mask_bits),
                               _stream(stream)), "pq_quantize_bwd")


def pq_pack_w2(rows, cols, W, alpha, packed, alpha_bf16, stream=None) -> None:
    _check(lib.pq_pack_w2(rows, cols, _ptr(W), _ptr(alpha), _ptr(packed), _ptr(alpha_bf16),
                          _stream(stream)), "pq_pack_w2")


def pq_pack_w4(rows, cols, W, alpha, packed, alpha_bf16, stream=None) -> None:
    _check(lib.pq_pack_w4(rows, cols, _ptr(W), _ptr(alpha), _ptr(packed), _ptr(alpha_bf16),
                          _stream(stream)), "pq_pack_w4")


def pq_gemm_workspace_bytes(mode: int, M: int, N: int, K: int) -> int:
    return int(lib.pq_gemm_workspace_bytes(mode, M, N, K))


def gemm_workspace(mode: int, M: int, N: int, K: int, device="cuda") -> Optional[torch.Tensor]:
    """A device buffer of pq_gemm_workspace_bytes(mode, M, N, K) bytes (None
    when the shape needs none), allocated by torch for the caller to keep."""
    n = pq_gemm_workspace_bytes(mode, M, N, K)
    if n < 0:
        raise PQError(2, "pq_gemm_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def _ws(mode, M, N, K, X, workspace, stream):
    """(pointer, size, tensor) of the caller's workspace, or of one allocated
    here from torch's caching allocator, out of the launch stream's memory."""
    if workspace is None:
        dev = X.device if isinstance(X, torch.Tensor) else "cuda"
        with _memory_of(stream):
            workspace = gemm_workspace(mode, M, N, K, dev)
        if workspace is None:
            return None, 0, None
    if isinstance(workspace, tuple):        # (pointer, bytes) from a caller that keeps its own buffer
        return workspace[0], int(workspace[1]), None
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def pq_w2a16_gemm(M, N, K, X, packed, alpha_bf16, Y, stream=None, workspace=None) -> None:
    wp, wb, _keep = _ws(PQ_W2_SEQ, M, N, K, X, workspace, stream)
    _check(lib.pq_w2a16_gemm(M, N, K, _ptr(X), _ptr(packed), _ptr(alpha_bf16), _ptr(Y), wp, wb,
                             _stream(stream)), "pq_w2a16_gemm")


def pq_w4a16_gemm(M, N, K, X, packed, alpha_bf16, Y, stream=None, workspace=None) -> None:
    wp, wb, _keep = _ws(PQ_W4_LSQ, M, N, K, X, workspace, stream)
    _check(lib.pq_w4a16_gemm(M, N, K, _ptr(X), _ptr(packed), _ptr(alpha_bf16), _ptr(Y), wp, wb,
                             _stream(stream)), "pq_w4a16_gemm")


def pq_pack(mode, rows, cols, W, alpha, packed, alpha_bf16, stream=None) -> None:
    _check(lib.pq_pack(mode, rows, cols, _ptr(W), _ptr(alpha), _ptr(packed), _ptr(alpha_bf16),
                       _stream(stream)), "pq_pack")


def pq_gemm(mode, M, N, K, X, packed, alpha_bf16, Y, stream=None, workspace=None) -> None:
    wp, wb, _keep = _ws(mode, M, N, K, X, workspace, stream)
    _check(lib.pq_gemm(mode, M, N, K, _ptr(X), _ptr(packed), _ptr(alpha_bf16), _ptr(Y), wp, wb,
                       _stream(stream)), "pq_gemm")


def pq_gemm_f32a(mode, M, N, K, X, packed, alpha, Y, stream=None, workspace=None) -> None:
    wp, wb, _keep = _ws(mode, M, N, K, X, workspace, stream)
    _check(lib.pq_gemm_f32a(mode, M, N, K, _ptr(X), _ptr(packed), _ptr(alpha), _ptr(Y), wp, wb,
                            _stream(stream)), "pq_gemm_f32a")


PQ_NOALLOC_SCRATCH_BYTES = 32 << 20


def pq_gemm_noalloc(mode, M, N, K, X, packed, alpha_bf16, Y, stream=None) -> None:
    """pq_gemm with the library's fixed scratch instead of a workspace."""
    _check(lib.pq_gemm_noalloc(mode, M, N, K, _ptr(X), _ptr(packed), _ptr(alpha_bf16), _ptr(Y),
                               _stream(stream)), "pq_gemm_noalloc")


PQ_CODES_EXPORT = 2


def pq_num_levels(mode: int) -> int:
    return int(lib.pq_num_levels(mode))


def pq_level_stats(mode, rows, cols, codes, counts, entropy=None, stream=None) -> None:
    _check(lib.pq_level_stats(mode, rows, cols, _ptr(codes), _ptr(counts), _ptr(entropy), _stream(stream)),
           "pq_level_stats")


def pq_quantize_fwd_stats(mode, rows, cols, W, alpha, Wq_bf16, codes, counts, entropy=None,
                          stream=None) -> None:
    _check(lib.pq_quantize_fwd_stats(mode, rows, cols, _ptr(W), _ptr(alpha), _ptr(Wq_bf16), _ptr(codes),
                                     _ptr(counts), _ptr(entropy), _stream(stream)), "pq_quantize_fwd_stats")


def pq_weight_movement(rows, cols, W, W0, sq_diff, sq_ref, stream=None) -> None:
    _check(lib.pq_weight_movement(rows, cols, _ptr(W), _ptr(W0), _ptr(sq_diff), _ptr(sq_ref), _stream(stream)),
           "pq_weight_movement")


class MatTable:
    """A pq_mat[] descriptor table in host memory plus its device copy.

    Build it once per stack of matrices and pass it to the grouped calls;
    it keeps the device copy (a torch uint8 tensor) alive."""

    STRUCT = pq_mat
    POINTERS = ("W", "alpha", "wq_bf16", "wq_f32", "codes", "G", "dW", "dalpha", "mask_bits", "alpha_bf16")

    def __init__(self, mats: Sequence[dict], device="cuda"):
        n = len(mats)
        self.count = n
        self.host = (self.STRUCT * max(n, 1))()
        for i, m in enumerate(mats):
            d = self.host[i]
            for f in self.POINTERS:
                setattr(d, f, _ptr(m.get(f)))
            d.grad_scale = float(m.get("grad_scale", 0.0))
            d.rows = int(m["rows"])
            d.cols = int(m["cols"])
        raw = bytes(memoryview(self.host).cast("B"))[: n * ctypes.sizeof(self.STRUCT)]
        self.dev = torch.frombuffer(bytearray(raw) or bytearray(1), dtype=torch.uint8).to(device)

    @property
    def host_ptr(self) -> int:
        return ctypes.addressof(self.host)

    @property
    def dev_ptr(self) -> int:
        return self.dev.data_ptr()


def pq_quantize_fwd_grouped(mode, table: MatTable, flags=0, stream=None) -> None:
    _check(lib.pq_quantize_fwd_grouped(mode, table.count, table.host_ptr, table.dev_ptr, flags,
                                       _stream(stream)), "pq_quantize_fwd_grouped")


def pq_quantize_bwd_grouped(mode, table: MatTable, g_dtype=PQ_G_F32, stream=None) -> None:
    _check(lib.pq_quantize_bwd_grouped(mode, table.count, table.host_ptr, table.dev_ptr, g_dtype,
                                       _stream(stream)), "pq_quantize_bwd_grouped")


def pq_pack_grouped(mode, table: MatTable, stream=None) -> None:
    _check(lib.pq_pack_grouped(mode, table.count, table.host_ptr, table.dev_ptr, _stream(stream)),
           "pq_pack_grouped")


class StepTable(MatTable):
    """A pq_step_mat[] descriptor table (host + device copy) for the fused step."""

    STRUCT = pq_step_mat
    POINTERS = ("W", "alpha", "G", "mW", "vW", "m_alpha", "v_alpha", "wq_bf16", "codes", "dalpha")


def adamw_params(step, lr=2e-5, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0) -> pq_adamw:
    return pq_adamw(float(lr), float(beta1), float(beta2), float(eps), float(weight_decay), int(step))


def pq_qat_step(mode, rows, cols, W, alpha, G, g_dtype, grad_scale, mW, vW, m_alpha, v_alpha,
                hp: pq_adamw, Wq_bf16=None, codes=None, dalpha=None, stream=None) -> None:
    _check(lib.pq_qat_step(mode, rows, cols, _ptr(W), _ptr(alpha), _ptr(G), g_dtype, float(grad_scale),
                           _ptr(mW), _ptr(vW), _ptr(m_alpha), _ptr(v_alpha), ctypes.addressof(hp),
                           _ptr(Wq_bf16), _ptr(codes), _ptr(dalpha), _stream(stream)), "pq_qat_step")


def pq_qat_step_grouped(mode, table: StepTable, hp: pq_adamw, g_dtype=PQ_G_F32, stream=None) -> None:
    _check(lib.pq_qat_step_grouped(mode, table.count, table.host_ptr, table.dev_ptr, g_dtype,
                                   ctypes.addressof(hp), _stream(stream)), "pq_qat_step_grouped")


# ------------------------------------------------------------------ serving
# Rotary positions, the key-value cache and attention over it.  Sizes and
# strides come from the tensors; everything else is checked by the library.

PQ_F32, PQ_BF16, PQ_F16 = 0, 1, 2
PQ_ROPE_HALF, PQ_ROPE_INTERLEAVED = 0, 1
PQ_ROPE_PLAIN, PQ_ROPE_LINEAR, PQ_ROPE_NTK, PQ_ROPE_YARN, PQ_ROPE_BANDS = 0, 1, 2, 3, 4
PQ_KV_16, PQ_KV_8, PQ_KV_4 = 0, 1, 2
_DTYPE = {torch.float32: PQ_F32, torch.bfloat16: PQ_BF16, torch.float16: PQ_F16}


# Decode steps are short calls, so the checks below are written to cost little:
# plain conditions, each attribute of a tensor read once.


def _dtype(t: torch.Tensor, what: str) -> int:
    d = _DTYPE.get(t.dtype)
    if d is None:
        raise TypeError(f"{what}: {t.dtype} is none of float32, bfloat16, float16")
    return d


def _rows(t: torch.Tensor, what: str):
    """(token stride, head stride) in elements of t [tokens, heads, dim]."""
    st = t.stride()
    if len(st) != 3 or (st[2] != 1 and t.shape[2] != 1):
        raise ValueError(f"{what}: [tokens, heads, dim] with a contiguous last dimension wanted")
    return st[0], st[1]


def _array(t: torch.Tensor, dtype: torch.dtype, n: int, what: str) -> int:
    """The address of a contiguous index array of n elements."""
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: {n} contiguous {dtype} wanted")
    return t.data_ptr()


def pq_rope_table(max_pos, rot, base=10000.0, table=None, scaling: Optional[pq_rope_scaling] = None, stream=None,
                  device="cuda") -> torch.Tensor:
    """The (cos, sin) rows of positions 0 .. max_pos - 1: f32 [max_pos, rot / 2, 2], made here if not given."""
    if table is None:
        with _memory_of(stream):
            table = torch.empty(max_pos, rot // 2, 2, dtype=torch.float32, device=device)
        if stream is not None:          # the caller goes on to use it there
            table.record_stream(torch.cuda.current_stream())
    _check(lib.pq_rope_table(max_pos, rot, float(base), ctypes.addressof(scaling) if scaling is not None else None,
                             _array(table, torch.float32, max_pos * rot, "table"), _stream(stream)), "pq_rope_table")
    return table


def rope_scaling(kind, factor, trained=0.0, beta_fast=None, beta_slow=1.0) -> pq_rope_scaling:
    """A scaling of pq_rope_table; beta_fast defaults to the kind's usual value."""
    if beta_fast is None:
        beta_fast = 4.0 if kind == PQ_ROPE_BANDS else 32.0
    return pq_rope_scaling(int(kind), 0, float(factor), float(trained), float(beta_fast), float(beta_slow))


def _table_shape(table: torch.Tensor):
    n = table.shape
    if len(n) != 3 or n[2] != 2 or table.dtype != torch.float32 or not table.is_contiguous():
        raise ValueError("table: contiguous float32 [max_pos, rot / 2, 2] wanted")
    return n[0], 2 * n[1]


def pq_rope(x, positions, table, y=None, layout=PQ_ROPE_HALF, inverse=False, stream=None) -> None:
    """Rotate x [tokens, heads, dim] into y (None: in place); inverse=True is the gradient's rotation."""
    n, heads, dim = shape = x.shape
    xt, xh = _rows(x, "x")
    xp = x.data_ptr()
    if y is None:
        yp, yt, yh = xp, xt, xh
    else:
        if y.shape != shape or y.dtype != x.dtype:
            raise ValueError("y: the shape and type of x wanted")
        yp = y.data_ptr()
        yt, yh = _rows(y, "y")
    max_pos, rot = _table_shape(table)
    rc = lib.pq_rope(_dtype(x, "x"), n, heads, dim, rot, layout, 1 if inverse else 0, xp, xt, xh,
                     _array(positions, torch.int32, n, "positions"), table.data_ptr(), max_pos, yp, yt, yh,
                     _stream(stream))
    if rc:
        raise PQError(rc, "pq_rope")


def pq_kv_row_bytes(fmt: int, dim: int) -> int:
    return int(lib.pq_kv_row_bytes(fmt, dim))


class KVCache:
    """A paged key-value cache: the caller's arrays and their pq_kv_cache.

    k and v are [pages, heads, page_size, row] views with equal strides --
    transpose(1, 2) of [pages, page_size, heads, row] arrays for token-major
    pages -- in bf16 or f16 (PQ_KV_16, row = dim) or uint8 (PQ_KV_8, row =
    dim; PQ_KV_4, row = dim / 2); k_param and v_param are contiguous bf16
    [pages, heads, page_size, 2]."""

    def __init__(self, fmt, page_size, k, v, k_param=None, v_param=None):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k, v: [pages, heads, page_size, row] of one type, shape and strides wanted")
        pages, heads, tokens, row = k.shape
        if tokens != page_size or k.stride(3) != 1:
            raise ValueError("k, v: page_size tokens of contiguous rows wanted")
        if fmt == PQ_KV_16:
            if k.dtype not in (torch.bfloat16, torch.float16):
                raise ValueError("k, v: bfloat16 or float16 wanted")
            dim, dtype = row, _DTYPE[k.dtype]
        elif fmt in (PQ_KV_8, PQ_KV_4):
            if k.dtype != torch.uint8:
                raise ValueError("k, v: uint8 wanted")
            dim, dtype = row * (1 if fmt == PQ_KV_8 else 2), 0
            for p in (k_param, v_param):
                if p is None or p.dtype != torch.bfloat16 or tuple(p.shape) != (pages, heads, tokens, 2) or \
                        not p.is_contiguous():
                    raise ValueError("k_param, v_param: contiguous bfloat16 [pages, heads, page_size, 2] wanted")
        else:
            raise ValueError("fmt: PQ_KV_16, PQ_KV_8 or PQ_KV_4 wanted")
        self.tensors = (k, v, k_param, v_param)          # kept alive with the addresses
        self.format, self.page_size, self.heads, self.dim, self.num_pages = fmt, page_size, heads, dim, pages
        size = k.element_size()
        s = [x * size for x in k.stride()[:3]]
        self.struct = pq_kv_cache(k.data_ptr(), v.data_ptr(), _ptr(k_param), _ptr(v_param), pages, s[0], s[1], s[2],
                                  fmt, dtype, page_size, heads, dim, 0)
        self.ptr = ctypes.addressof(self.struct)

    @classmethod
    def allocate(cls, fmt, num_pages, page_size, heads, dim, dtype=torch.bfloat16, device="cuda"):
        """A zeroed cache with head-major pages."""
        row = dim if fmt != PQ_KV_4 else dim // 2
        shape = (num_pages, heads, page_size)
        kind = dtype if fmt == PQ_KV_16 else torch.uint8
        k, v = (torch.zeros(*shape, row, dtype=kind, device=device) for _ in range(2))
        if fmt == PQ_KV_16:
            return cls(fmt, page_size, k, v)
        return cls(fmt, page_size, k, v, *(torch.zeros(*shape, 2, dtype=torch.bfloat16, device=device) for _ in range(2)))


def pq_kv_append(cache: KVCache, k, v, slots, positions=None, table=None, layout=PQ_ROPE_HALF, q=None, q_out=None,
                 stream=None) -> None:
    """Write k, v [tokens, heads, dim] into the cache at slots, each token at its own (padding: -1); with a table k
    is rotated on the way, and q [tokens, q_heads, dim] is rotated into q_out (None: in place) in the same launch."""
    n, heads, dim = shape = k.shape
    kt, kh = _rows(k, "k")
    vt, vh = _rows(v, "v")
    kind = k.dtype
    if v.shape != shape or v.dtype != kind or heads != cache.heads or dim != cache.dim:
        raise ValueError("k, v: [tokens, heads, dim] of the cache and one type wanted")
    max_pos = rot = qh = qt = qs = qot = qos = 0
    pp = tp = qp = qop = None
    if table is not None:
        max_pos, rot = _table_shape(table)
        tp = table.data_ptr()
        if positions is not None:
            pp = _array(positions, torch.int32, n, "positions")
    if q is not None:
        qn, qh, qd = qshape = q.shape
        if qn != n or qd != dim or q.dtype != kind:
            raise ValueError("q: [tokens, q_heads, dim] of k's type wanted")
        qt, qs = _rows(q, "q")
        qp = q.data_ptr()
        if q_out is None:
            qop, qot, qos = qp, qt, qs
        else:
            if q_out.shape != qshape or q_out.dtype != kind:
                raise ValueError("q_out: the shape and type of q wanted")
            qot, qos = _rows(q_out, "q_out")
            qop = q_out.data_ptr()
    rc = lib.pq_kv_append(cache.ptr, _dtype(k, "k"), n, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh,
                          _array(slots, torch.int64, n, "slots"), pp, tp, max_pos, rot, layout, qp, qh, qt, qs,
                          qop, qot, qos, _stream(stream))
    if rc:
        raise PQError(rc, "pq_kv_append")


def _block_table(block_table, batch: int):
    n, st = block_table.shape, block_table.stride()
    if len(n) != 2 or n[0] != batch or (st[1] != 1 and n[1] > 1) or block_table.dtype != torch.int32:
        raise ValueError("block_table: int32 [batch, pages] wanted")
    return block_table.data_ptr(), st[0], n[1]


def pq_kv_load(cache: KVCache, block_table, starts, cu, k_out, v_out, stream=None) -> None:
    """Read tokens starts[b] .. of each sequence into rows cu[b] .. cu[b + 1] of k_out and v_out."""
    batch = cu.numel() - 1
    bp, bs, bn = _block_table(block_table, batch)
    n, heads, dim = shape = k_out.shape
    if v_out.shape != shape or v_out.dtype != k_out.dtype or heads != cache.heads or dim != cache.dim:
        raise ValueError("k_out, v_out: [tokens, heads, dim] of one type wanted")
    kt, kh = _rows(k_out, "k_out")
    vt, vh = _rows(v_out, "v_out")
    rc = lib.pq_kv_load(cache.ptr, _dtype(k_out, "k_out"), batch, n, bp, bs, bn,
                        None if starts is None else _array(starts, torch.int32, batch, "starts"),
                        _array(cu, torch.int32, batch + 1, "cu"), k_out.data_ptr(), kt, kh, v_out.data_ptr(), vt, vh,
                        _stream(stream))
    if rc:
        raise PQError(rc, "pq_kv_load")


def pq_attn_decode_workspace_bytes(cache: KVCache, batch: int, q_heads: int) -> int:
    return int(lib.pq_attn_decode_workspace_bytes(cache.ptr, batch, q_heads))


def attn_workspace(cache: KVCache, batch: int, q_heads: int, device="cuda") -> torch.Tensor:
    """A workspace for pq_attn_decode calls of up to this size, for the caller to keep."""
    n = pq_attn_decode_workspace_bytes(cache, batch, q_heads)
    if n < 0:
        raise PQError(2, "pq_attn_decode_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def pq_attn_decode(cache: KVCache, q, block_table, lens, out, lse=None, scale=None, window=0, max_len=0,
                   workspace=None, stream=None) -> None:
    """Attention of one new token per sequence, q [batch, q_heads, dim], over the cache; scale defaults to
    1 / sqrt(dim).  Without a workspace one is allocated for the call."""
    batch, q_heads, dim = shape = q.shape
    if dim != cache.dim or out.shape != shape or out.dtype != q.dtype:
        raise ValueError("q, out: [batch, q_heads, dim] of the cache and one type wanted")
    qt, qh = _rows(q, "q")
    ot, oh = _rows(out, "out")
    bp, bs, bn = _block_table(block_table, batch)
    if workspace is None:
        with _memory_of(stream):
            workspace = attn_workspace(cache, batch, q_heads, q.device)
    rc = lib.pq_attn_decode(cache.ptr, _dtype(q, "q"), batch, q_heads, q.data_ptr(), qt, qh, bp, bs, bn,
                            _array(lens, torch.int32, batch, "lens"), dim ** -0.5 if scale is None else scale, window,
                            max_len, out.data_ptr(), ot, oh,
                            None if lse is None else _array(lse, torch.float32, batch * q_heads, "lse"),
                            workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream))
    if rc:
        raise PQError(rc, "pq_attn_decode")
