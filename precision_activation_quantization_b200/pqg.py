"""Python binding of libpqg.so (C ABI in include/pqg.h).

Argument marshalling only: every step of the quantization runs in the CUDA
library.  Importing this module loads the library, building it first with nvcc
when it is missing or older than its sources, and raises if that fails; there
is no fallback implementation.

``pqg_quant``, ``pqg_scales_bytes``, ``pqg_status_string`` and friends mirror
the C entry points one to one.  ``quant`` is the torch-facing convenience: it
takes tensors, allocates outputs when not given (torch is used for device memory
and streams only), and raises ``PqgError`` on a non-OK status.  The interface
follows the sglang PR #30924 report, "[JIT] Trait-driven per_token_group_quant"
(实现拆解 item 2: one entry taking masked_m and expected_m, an allocation helper
and a scale-layout inference helper).
"""
from __future__ import annotations

import contextlib
import ctypes
import os

from . import build as _build

# ---- enums (values of include/pqg.h) ---------------------------------------
PQG_OK = 0
PQG_ERR_INVALID_ARG = -1
PQG_ERR_UNSUPPORTED = -2
PQG_ERR_ALIGNMENT = -3
PQG_ERR_CUDA = -4

PQG_BF16, PQG_FP16, PQG_E4M3, PQG_INT8, PQG_E2M1 = 0, 1, 2, 3, 4
PQG_SCALE_FP32, PQG_SCALE_UE8M0, PQG_SCALE_E4M3 = 0, 1, 2
PQG_KV_MXFP4, PQG_KV_NVFP4 = 0, 1
PQG_ROW_MAJOR, PQG_COL_MAJOR_TMA, PQG_UE8M0_PACKED, PQG_UE8M0_TILED_128x4 = 0, 1, 2, 3

IN_DTYPES = {"bf16": PQG_BF16, "fp16": PQG_FP16}
OUT_DTYPES = {"e4m3": PQG_E4M3, "int8": PQG_INT8, "e2m1": PQG_E2M1}
SCALE_FMTS = {"fp32": PQG_SCALE_FP32, "ue8m0": PQG_SCALE_UE8M0, "e4m3": PQG_SCALE_E4M3}
LAYOUTS = {"row": PQG_ROW_MAJOR, "col": PQG_COL_MAJOR_TMA, "packed": PQG_UE8M0_PACKED,
           "tile128x4": PQG_UE8M0_TILED_128x4}
KV_FORMATS = {"mxfp4": PQG_KV_MXFP4, "nvfp4": PQG_KV_NVFP4}
KV_GROUP = {"mxfp4": 32, "nvfp4": 16}

EXPORTS = ("pqg_quant", "pqg_quant_nvfp4", "pqg_quant_varlen", "pqg_rmsnorm_quant",
           "pqg_kv_write", "pqg_kv_read", "pqg_kv_attention", "pqg_kv_attention_workspace",
           "pqg_scales_bytes",
           "pqg_status_string", "pqg_last_cuda_error", "pqg_set_pdl", "pqg_launch_count",
           "pqg_version")


class pqg_kv_cache(ctypes.Structure):
    """struct pqg_kv_cache of include/pqg.h."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("global_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32)]


class PqgError(RuntimeError):
    def __init__(self, status: int, where: str = "pqg_quant"):
        self.status = status
        msg = pqg_status_string(status)
        if status == PQG_ERR_CUDA:
            msg += f" (cudaError {pqg_last_cuda_error()})"
        super().__init__(f"{where}: {msg} [{status}]")


def _load() -> ctypes.CDLL:
    path = os.environ.get("PQG_LIBRARY") or _build.build()
    lib = ctypes.CDLL(path)
    i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    lib.pqg_quant.restype = i32
    lib.pqg_quant.argtypes = [vp, vp, vp, i64, i64, i64, i32, i32, i32, i32, i32, i32, vp,
                              i64, vp]
    lib.pqg_quant_nvfp4.restype = i32
    lib.pqg_quant_nvfp4.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, i32, i32, vp, i64, vp]
    lib.pqg_quant_varlen.restype = i32
    lib.pqg_quant_varlen.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, i32, i32, i32, i32,
                                     i32, vp, vp, i64, vp]
    lib.pqg_rmsnorm_quant.restype = i32
    lib.pqg_rmsnorm_quant.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i32,
                                      ctypes.c_double, i32, i32, i32, i32, vp]
    cache = ctypes.POINTER(pqg_kv_cache)
    lib.pqg_kv_write.restype = i32
    lib.pqg_kv_write.argtypes = [cache, vp, vp, vp, i64, i64, i64, i32, vp]
    lib.pqg_kv_read.restype = i32
    lib.pqg_kv_read.argtypes = [cache, vp, i64, i64, vp, i64, vp, vp, i64, i32, vp]
    lib.pqg_kv_attention.restype = i32
    lib.pqg_kv_attention.argtypes = [cache, vp, i64, vp, i64, i64, vp, i64, i64, i64,
                                     ctypes.c_float, i64, vp, vp, vp, i64, i32, vp]
    lib.pqg_kv_attention_workspace.restype = i64
    lib.pqg_kv_attention_workspace.argtypes = [cache, i64, i64, i64, i64, i64]
    lib.pqg_scales_bytes.restype = i64
    lib.pqg_scales_bytes.argtypes = [i64, i64, i64, i32, i32, i32]
    lib.pqg_status_string.restype = ctypes.c_char_p
    lib.pqg_status_string.argtypes = [i32]
    lib.pqg_last_cuda_error.restype = i32
    lib.pqg_last_cuda_error.argtypes = []
    lib.pqg_set_pdl.restype = i32
    lib.pqg_set_pdl.argtypes = [i32]
    lib.pqg_launch_count.restype = ctypes.c_uint64
    lib.pqg_launch_count.argtypes = []
    lib.pqg_version.restype = ctypes.c_char_p
    lib.pqg_version.argtypes = []
    return lib


_lib = _load()
LIBRARY_PATH = _lib._name


# ---- the C entry points, one to one ----------------------------------------

def pqg_quant(in_ptr: int, out_ptr: int, scales_ptr: int, M: int, num_experts: int, K: int,
              group: int, in_dtype: int, out_dtype: int, scale_fmt: int, scale_layout: int,
              fuse_silu_mul: int, masked_m_ptr: int | None, expected_m: int,
              stream: int | None) -> int:
    return _lib.pqg_quant(in_ptr, out_ptr, scales_ptr, M, num_experts, K, group, in_dtype,
                          out_dtype, scale_fmt, scale_layout, fuse_silu_mul, masked_m_ptr,
                          expected_m, stream)


def pqg_quant_nvfp4(in_ptr: int, out_ptr: int, scales_ptr: int, global_scale_ptr: int, M: int,
                    num_experts: int, K: int, in_dtype: int, scale_layout: int,
                    fuse_silu_mul: int, masked_m_ptr: int | None, expected_m: int,
                    stream: int | None) -> int:
    return _lib.pqg_quant_nvfp4(in_ptr, out_ptr, scales_ptr, global_scale_ptr, M, num_experts,
                                K, in_dtype, scale_layout, fuse_silu_mul, masked_m_ptr,
                                expected_m, stream)


def pqg_quant_varlen(in_ptr: int, out_ptr: int, scales_ptr: int, global_scale_ptr: int | None,
                     M: int, num_experts: int, K: int, group: int, in_dtype: int,
                     out_dtype: int, scale_fmt: int, scale_layout: int, fuse_silu_mul: int,
                     seg_indptr_ptr: int | None, seg_lens_ptr: int | None, expected_m: int,
                     stream: int | None) -> int:
    return _lib.pqg_quant_varlen(in_ptr, out_ptr, scales_ptr, global_scale_ptr, M, num_experts,
                                 K, group, in_dtype, out_dtype, scale_fmt, scale_layout,
                                 fuse_silu_mul, seg_indptr_ptr, seg_lens_ptr, expected_m,
                                 stream)


def pqg_rmsnorm_quant(in_ptr: int, residual_ptr: int | None, weight_ptr: int,
                      residual_out_ptr: int | None, out_ptr: int, scales_ptr: int,
                      global_scale_ptr: int | None, M: int, K: int, group: int, eps: float,
                      in_dtype: int, out_dtype: int, scale_fmt: int, scale_layout: int,
                      stream: int | None) -> int:
    return _lib.pqg_rmsnorm_quant(in_ptr, residual_ptr, weight_ptr, residual_out_ptr, out_ptr,
                                  scales_ptr, global_scale_ptr, M, K, group, eps, in_dtype,
                                  out_dtype, scale_fmt, scale_layout, stream)


def pqg_kv_write(cache: pqg_kv_cache, k_ptr: int, v_ptr: int, slots_ptr: int, T: int,
                 k_stride: int, v_stride: int, in_dtype: int, stream: int | None) -> int:
    return _lib.pqg_kv_write(cache, k_ptr, v_ptr, slots_ptr, T, k_stride, v_stride, in_dtype,
                             stream)


def pqg_kv_read(cache: pqg_kv_cache, page_table_ptr: int, table_stride: int, max_pages: int,
                indptr_ptr: int, B: int, k_out_ptr: int, v_out_ptr: int, M: int, out_dtype: int,
                stream: int | None) -> int:
    return _lib.pqg_kv_read(cache, page_table_ptr, table_stride, max_pages, indptr_ptr, B,
                            k_out_ptr, v_out_ptr, M, out_dtype, stream)


def pqg_kv_attention(cache: pqg_kv_cache, q_ptr: int, q_stride: int, page_table_ptr: int,
                     table_stride: int, max_pages: int, seq_lens_ptr: int, B: int, q_len: int,
                     q_heads: int, sm_scale: float, max_len: int, out_ptr: int,
                     lse_ptr: int | None, workspace_ptr: int | None, workspace_bytes: int,
                     in_dtype: int, stream: int | None) -> int:
    return _lib.pqg_kv_attention(cache, q_ptr, q_stride, page_table_ptr, table_stride, max_pages,
                                 seq_lens_ptr, B, q_len, q_heads, sm_scale, max_len, out_ptr,
                                 lse_ptr, workspace_ptr, workspace_bytes, in_dtype, stream)


def pqg_kv_attention_workspace(cache: pqg_kv_cache, max_pages: int, B: int, q_len: int,
                               q_heads: int, max_len: int) -> int:
    return _lib.pqg_kv_attention_workspace(cache, max_pages, B, q_len, q_heads, max_len)


def pqg_scales_bytes(num_experts: int, M: int, K: int, group: int, scale_fmt: int,
                     scale_layout: int) -> int:
    return _lib.pqg_scales_bytes(num_experts, M, K, group, scale_fmt, scale_layout)


def pqg_status_string(status: int) -> str:
    return _lib.pqg_status_string(status).decode()


def pqg_last_cuda_error() -> int:
    return _lib.pqg_last_cuda_error()


def pqg_set_pdl(enable: bool) -> bool:
    return bool(_lib.pqg_set_pdl(int(bool(enable))))


def pqg_launch_count() -> int:
    return int(_lib.pqg_launch_count())


def pqg_version() -> str:
    return _lib.pqg_version().decode()


# ---- torch-facing helpers ---------------------------------------------------

def scales_spec(M: int, K: int, group: int, scale_fmt: str = "fp32", layout: str = "row",
                num_experts: int = 1):
    """(shape, torch dtype) of a contiguous scale buffer for these arguments.

    row       : [E, M, ng]            fp32 or uint8
    col       : [E, ng, M_pad]        fp32 or uint8
    packed    : [E, ceil(ng/4), M_pad] int32
    tile128x4 : [E, ceil(M/128) * ceil(ng/4) * 512] uint8
    """
    import torch
    nbytes = pqg_scales_bytes(num_experts, M, K, group, SCALE_FMTS[scale_fmt], LAYOUTS[layout])
    if nbytes < 0:
        raise PqgError(nbytes, "pqg_scales_bytes")
    ng, mpad = K // group, (M + 3) // 4 * 4
    if layout == "row":
        shape = (num_experts, M, ng)
    elif layout == "col":
        shape = (num_experts, ng, mpad)
    elif layout == "tile128x4":
        return (num_experts, (M + 127) // 128 * ((ng + 3) // 4) * 512), torch.uint8
    else:
        return (num_experts, (ng + 3) // 4, mpad), torch.int32
    return shape, (torch.float32 if scale_fmt == "fp32" else torch.uint8)


def allocate_outputs(M: int, K: int, group: int, *, num_experts: int = 1,
                     out_dtype: str = "e4m3", scale_fmt: str = "fp32", layout: str = "row",
                     device=None):
    """Allocate (out, scales) for one call with torch (device memory only).
    E2M1 codes come back as uint8 [E, M, K/2], two codes per byte."""
    import torch
    if out_dtype == "e2m1":
        out = torch.empty((num_experts, M, K // 2), dtype=torch.uint8, device=device)
    else:
        odt = torch.float8_e4m3fn if out_dtype == "e4m3" else torch.int8
        out = torch.empty((num_experts, M, K), dtype=odt, device=device)
    shape, sdt = scales_spec(M, K, group, scale_fmt, layout, num_experts)
    return out, torch.empty(shape, dtype=sdt, device=device)


def infer_scale_layout(scales, M: int, K: int, group: int) -> str:
    """Scale layout of an [M, ng]-shaped view (or packed [M, ceil(ng/4)] int32 view)
    from its strides: contiguous rows -> "row"; unit stride along M -> "col", or
    "packed" for int32.  Mirrors the stride-based inference the pages describe."""
    import torch
    ng = K // group
    if scales.dim() != 2 or scales.shape[0] != M:
        raise ValueError("expected a 2-D [M, groups] view of the scales")
    if scales.dtype == torch.int32:
        if scales.shape[1] == (ng + 3) // 4 and (M <= 1 or scales.stride(0) == 1):
            return "packed"
    elif scales.shape[1] == ng:
        if scales.stride(1) == 1 and (M <= 1 or scales.stride(0) == ng):
            return "row"
        if M <= 1 or scales.stride(0) == 1:
            return "col"
    raise ValueError("scale view matches no supported layout")


def quant(x, out=None, scales=None, *, M: int | None = None, K: int | None = None,
          group: int = 128, num_experts: int | None = None, out_dtype: str = "e4m3",
          scale_fmt: str = "fp32", layout: str = "row", fuse_silu_mul: bool = False,
          masked_m=None, expected_m: int = 0, global_scale=None, stream=None):
    """Quantize a CUDA tensor; returns (out, scales).

    ``x`` is bf16/fp16, [E, M, K] / [M, K] ([..., 2K] when ``fuse_silu_mul``).
    ``masked_m`` is an int32 CUDA tensor of E row counts (masked dispatch).
    ``out``, ``scales`` and ``masked_m`` must be contiguous: the kernel addresses
    each densely.  With the column-wise layouts ("col", "packed") ``scales`` may
    also be the [.., M_pad, columns] transposed view of its contiguous plane; any
    other non-contiguous view raises.  The call runs with ``x``'s device current,
    whichever device is current in the caller.
    NVFP4 is ``out_dtype="e2m1", scale_fmt="e4m3", group=16`` with
    ``global_scale`` a one-element fp32 CUDA tensor (pqg_quant_nvfp4).
    The kernel runs on ``stream`` (default: torch's current stream).
    """
    import torch
    if x.dtype == torch.bfloat16:
        in_dtype = PQG_BF16
    elif x.dtype == torch.float16:
        in_dtype = PQG_FP16
    else:
        raise TypeError(f"unsupported input dtype {x.dtype}")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA tensor")
    E = num_experts if num_experts is not None else (x.shape[0] if x.dim() == 3 else 1)
    width = x.shape[-1]
    K = K if K is not None else (width // 2 if fuse_silu_mul else width)
    M = M if M is not None else x.numel() // (E * width)
    if out is None or scales is None:
        o, s = allocate_outputs(M, K, group, num_experts=E, out_dtype=out_dtype,
                                scale_fmt=scale_fmt, layout=layout, device=x.device)
        out = o if out is None else out
        scales = s if scales is None else scales
    odt = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "e2m1": torch.uint8}[out_dtype]
    out_bytes = E * M * (K // 2 if out_dtype == "e2m1" else K)
    if x.numel() != E * M * width:
        raise ValueError("x does not hold E x M rows of the given width")
    if out.numel() * out.element_size() != out_bytes or out.dtype not in (odt, torch.uint8):
        raise ValueError(f"out must hold {out_bytes} bytes of codes")
    nbytes = pqg_scales_bytes(E, M, K, group, SCALE_FMTS[scale_fmt], LAYOUTS[layout])
    if nbytes >= 0 and scales.numel() * scales.element_size() != nbytes:
        raise ValueError(f"scales must be {nbytes} bytes for this layout")
    if not (out.is_cuda and scales.is_cuda and out.device == x.device == scales.device):
        raise ValueError("x, out and scales must be on the same CUDA device")
    # the kernel addresses every buffer from its first byte, densely
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    if not scales.is_contiguous():
        # only a column-wise layout can be handed over as its [.., M_pad, columns]
        # transposed view; its underlying buffer must be the dense plane
        ng = K // group
        cols = {"col": ng, "packed": (ng + 3) // 4}.get(layout)
        if (cols is None or scales.dim() < 2 or not scales.transpose(-1, -2).is_contiguous()
                or scales.shape[-1] != cols or scales.shape[-2] != (M + 3) // 4 * 4):
            raise ValueError(f"a non-contiguous scales view must be the transposed "
                             f"[M_pad, groups] view of a contiguous '{layout}' plane; "
                             f"layout '{layout}' does not match this view")
    mm_ptr = None
    if masked_m is not None:
        if (masked_m.dtype != torch.int32 or masked_m.device != x.device
                or masked_m.numel() != E or not masked_m.is_contiguous()):
            raise ValueError("masked_m must be a contiguous int32 CUDA tensor with one entry "
                             "per expert")
        mm_ptr = masked_m.data_ptr()
    if stream is None:
        stream = torch.cuda.current_stream(x.device)
    # the library sizes its grid from, and launches on, the current device
    with torch.cuda.device(x.device):
        return _launch(x, out, scales, M, E, K, group, in_dtype, out_dtype, scale_fmt, layout,
                       fuse_silu_mul, mm_ptr, expected_m, global_scale, stream)


def _launch(x, out, scales, M, E, K, group, in_dtype, out_dtype, scale_fmt, layout,
            fuse_silu_mul, mm_ptr, expected_m, global_scale, stream):
    import torch
    if scale_fmt == "e4m3":
        if (global_scale is None or global_scale.dtype != torch.float32
                or global_scale.numel() != 1 or global_scale.device != x.device):
            raise ValueError("NVFP4 needs global_scale: a one-element fp32 tensor on x's device")
        if out_dtype != "e2m1" or group != 16:
            raise ValueError("scale_fmt='e4m3' is NVFP4: out_dtype='e2m1', group=16")
        st = pqg_quant_nvfp4(x.data_ptr(), out.data_ptr(), scales.data_ptr(),
                             global_scale.data_ptr(), M, E, K, in_dtype, LAYOUTS[layout],
                             int(bool(fuse_silu_mul)), mm_ptr, int(expected_m),
                             getattr(stream, "cuda_stream", stream))
        if st != PQG_OK:
            raise PqgError(st, "pqg_quant_nvfp4")
        return out, scales
    st = pqg_quant(x.data_ptr(), out.data_ptr(), scales.data_ptr(), M, E, K, group, in_dtype,
                   OUT_DTYPES[out_dtype], SCALE_FMTS[scale_fmt], LAYOUTS[layout],
                   int(bool(fuse_silu_mul)), mm_ptr, int(expected_m),
                   getattr(stream, "cuda_stream", stream))
    if st != PQG_OK:
        raise PqgError(st)
    return out, scales


def quant_varlen(x, seg_indptr, seg_lens=None, out=None, scales=None, *, group: int = 128,
                 out_dtype: str = "e4m3", scale_fmt: str = "fp32", layout: str = "row",
                 fuse_silu_mul: bool = False, expected_m: int = 0, global_scale=None,
                 stream=None):
    """Grouped-contiguous (varlen) quantization of packed token rows; returns
    (out, scales).

    ``x`` is a contiguous bf16/fp16 CUDA tensor [M, K] ([M, 2K] when
    ``fuse_silu_mul``) holding the segments of all experts.  ``seg_indptr`` is
    an int32 CUDA tensor of E + 1 row offsets and ``seg_lens`` one of E token
    counts (or None: every row of a segment is a token).  Token rows are
    quantized into the same rows of ``out`` and of one scale plane of M rows;
    padding rows are left as they are (``torch.empty`` when allocated here).
    NVFP4 is ``out_dtype="e2m1", scale_fmt="e4m3", group=16`` with
    ``global_scale``.  The call runs with ``x``'s device current.
    """
    import torch
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"unsupported input dtype {x.dtype}")
    if not x.is_cuda or not x.is_contiguous() or x.dim() != 2:
        raise ValueError("x must be a contiguous 2-D CUDA tensor of packed rows")
    M, width = x.shape
    K = width // 2 if fuse_silu_mul else width
    E = seg_indptr.numel() - 1
    for name, t, n in (("seg_indptr", seg_indptr, E + 1), ("seg_lens", seg_lens, E)):
        if t is None:
            continue
        if (t.dtype != torch.int32 or t.device != x.device or t.numel() != n
                or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous int32 tensor of {n} entries on "
                             f"x's device")
    if E < 1:
        raise ValueError("seg_indptr needs at least two entries")
    if out is None or scales is None:
        o, sc = allocate_outputs(M, K, group, out_dtype=out_dtype, scale_fmt=scale_fmt,
                                 layout=layout, device=x.device)
        out = o[0] if out is None else out
        scales = sc[0] if scales is None else scales
    out_bytes = M * (K // 2 if out_dtype == "e2m1" else K)
    if out.numel() * out.element_size() != out_bytes or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous buffer of {out_bytes} bytes")
    nbytes = pqg_scales_bytes(1, M, K, group, SCALE_FMTS[scale_fmt], LAYOUTS[layout])
    if (nbytes >= 0 and scales.numel() * scales.element_size() != nbytes) \
            or not scales.is_contiguous():
        raise ValueError(f"scales must be a contiguous buffer of {nbytes} bytes")
    if not (out.device == scales.device == x.device):
        raise ValueError("x, out and scales must be on the same CUDA device")
    gptr = None
    if scale_fmt == "e4m3":
        if (global_scale is None or global_scale.dtype != torch.float32
                or global_scale.numel() != 1 or global_scale.device != x.device):
            raise ValueError("NVFP4 needs global_scale: a one-element fp32 tensor on x's device")
        gptr = global_scale.data_ptr()
    if stream is None:
        stream = torch.cuda.current_stream(x.device)
    in_dtype = PQG_BF16 if x.dtype == torch.bfloat16 else PQG_FP16
    with torch.cuda.device(x.device):
        st = pqg_quant_varlen(x.data_ptr(), out.data_ptr(), scales.data_ptr(), gptr, M, E, K,
                              group, in_dtype, OUT_DTYPES[out_dtype], SCALE_FMTS[scale_fmt],
                              LAYOUTS[layout], int(bool(fuse_silu_mul)), seg_indptr.data_ptr(),
                              None if seg_lens is None else seg_lens.data_ptr(),
                              int(expected_m), getattr(stream, "cuda_stream", stream))
    if st != PQG_OK:
        raise PqgError(st, "pqg_quant_varlen")
    return out, scales


def _allocating_on(stream, device):
    """Scope in which torch allocates from the pool of the stream a call runs on
    (memory of another stream's pool may still be in use there)."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        # (an ExternalStream of handle 0 would be a new stream, not the default one)
        stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                  else torch.cuda.default_stream(device))
    return torch.cuda.stream(stream)


_native = None


def native():
    """The tensor binding (csrc/pqg_torch.cpp), built first when it is missing or
    older than its sources, calling the library this module loaded."""
    global _native
    if _native is None:
        import torch  # noqa: F401  (its libraries resolve the binding's symbols)
        _build.build_binding()
        from . import _pqg_torch
        _pqg_torch.load(LIBRARY_PATH)
        _native = _pqg_torch
    return _native


def _call(function, stream, device, *args):
    """A native entry point on ``stream`` (None: torch's current stream); returns
    what it made, or raises on a non-OK status."""
    if stream is None:
        result = function(*args, None)
    else:
        with _allocating_on(stream, device):
            result = function(*args, getattr(stream, "cuda_stream", stream))
    if result[0] != PQG_OK:
        raise PqgError(result[0], result[1])
    return result[2:]


def rmsnorm_quant(x, weight, residual=None, out=None, scales=None, *, residual_out=None,
                  eps: float = 1e-6, group: int = 128, out_dtype: str = "e4m3",
                  scale_fmt: str = "fp32", layout: str = "row", global_scale=None, stream=None):
    """Residual addition, RMS norm and quantization in one pass; returns
    (out, scales, h).

    ``x`` and ``residual`` are contiguous bf16/fp16 CUDA tensors [M, K] (or
    [..., K], read as rows) and ``weight`` [K] of the same type.  h = x +
    residual, rounded to their type, comes back in ``residual_out`` (pass
    ``residual`` itself to update it in place; allocated when None); without a
    residual h is ``x`` and nothing is stored.  The norm of h times ``weight``
    is quantized by ``quant``'s rules into ``out`` [M, K] ([M, K/2] for E2M1)
    and one plane of ``scales`` in the given layout; neither is written past its
    rows.  NVFP4 is ``out_dtype="e2m1", scale_fmt="e4m3", group=16`` with
    ``global_scale``.  The call runs with ``x``'s device current.
    """
    return _call((_native or native()).rmsnorm_quant, stream, getattr(x, "device", None), x,
                 weight, residual, out, scales, residual_out, eps, group, OUT_DTYPES[out_dtype],
                 SCALE_FMTS[scale_fmt], LAYOUTS[layout], global_scale)


# ---- paged 4-bit key/value cache --------------------------------------------

class KVCache:
    """A paged 4-bit cache: its buffers and their geometry (see ``kv_cache``)."""

    __slots__ = ("k_codes", "v_codes", "k_scales", "v_scales", "global_scale", "fmt", "device",
                 "num_pages", "page_size", "kv_heads", "head_dim", "struct", "address", "index")


def kv_cache(k_codes, v_codes, k_scales, v_scales, *, fmt: str = "mxfp4",
             global_scale=None) -> KVCache:
    """A cache over existing buffers.

    Codes are uint8 CUDA tensors [num_pages, kv_heads, page_size, head_dim / 2]
    and scales [num_pages, kv_heads, head_dim / G, page_size], contiguous, with
    G = 32 for ``fmt="mxfp4"`` (UE8M0 scales) and 16 for "nvfp4" (E4M3 scales
    under ``global_scale``, two fp32 values on the device: g of the keys and g of
    the values).  The buffers belong to the caller, who keeps them alive.
    """
    import torch
    if fmt not in KV_FORMATS:
        raise ValueError(f"fmt must be one of {sorted(KV_FORMATS)}")
    c = KVCache()
    dev = k_codes.device
    if k_codes.dim() != 4:
        raise ValueError("codes must be [num_pages, kv_heads, page_size, head_dim / 2]")
    pages, heads, size, half = k_codes.shape
    want = {"k_codes": (pages, heads, size, half), "v_codes": (pages, heads, size, half)}
    want["k_scales"] = want["v_scales"] = (pages, heads, 2 * half // KV_GROUP[fmt], size)
    for name, t in (("k_codes", k_codes), ("v_codes", v_codes), ("k_scales", k_scales),
                    ("v_scales", v_scales)):
        if (t.dtype != torch.uint8 or tuple(t.shape) != want[name] or not t.is_contiguous()
                or not t.is_cuda or t.device != dev):
            raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor {want[name]} on one "
                             f"device")
        setattr(c, name, t)
    if (fmt == "nvfp4") != (global_scale is not None):
        raise ValueError("global_scale (two fp32 values) goes with fmt='nvfp4'")
    if global_scale is not None and (
            global_scale.dtype != torch.float32 or global_scale.numel() != 2
            or global_scale.device != dev or not global_scale.is_contiguous()):
        raise ValueError("global_scale must be a contiguous fp32 tensor of two values on the "
                         "cache's device")
    c.global_scale, c.fmt, c.device = global_scale, fmt, dev
    c.num_pages, c.kv_heads, c.page_size, c.head_dim = pages, heads, size, 2 * half
    c.struct = pqg_kv_cache(
        k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
        None if global_scale is None else global_scale.data_ptr(), pages, size, heads, 2 * half,
        KV_FORMATS[fmt])
    c.address, c.index = ctypes.addressof(c.struct), dev.index
    return c


def kv_allocate(num_pages: int, page_size: int, kv_heads: int, head_dim: int, *,
                fmt: str = "mxfp4", global_scale=None, device=None) -> KVCache:
    """A new cache of zeros (see ``kv_cache``)."""
    import torch
    if fmt not in KV_FORMATS:
        raise ValueError(f"fmt must be one of {sorted(KV_FORMATS)}")
    device = torch.device("cuda" if device is None else device)
    codes = (num_pages, kv_heads, page_size, head_dim // 2)
    scales = (num_pages, kv_heads, head_dim // KV_GROUP[fmt], page_size)
    k, v, ks, vs = (torch.zeros(n, dtype=torch.uint8, device=device)
                    for n in (codes, codes, scales, scales))
    return kv_cache(k, v, ks, vs, fmt=fmt, global_scale=global_scale)


def kv_write(cache: KVCache, k, v, slots, *, stream=None) -> None:
    """Quantize the keys and values of T tokens into their slots of the cache.

    ``k`` and ``v`` are bf16/fp16 CUDA tensors [T, kv_heads, head_dim]; the heads
    of a token are dense, tokens may be strided (slices of one projection's
    output).  ``slots`` [T] int32 holds page * page_size + offset; a token with a
    slot outside the cache (-1: padding) is skipped.  Slots of one call must be
    distinct.
    """
    _call((_native or native()).kv_write, stream, cache.device, cache.address, cache.index, k, v,
          slots)


def kv_read(cache: KVCache, page_table, indptr, num_tokens: int, *, dtype=None, k_out=None,
            v_out=None, stream=None):
    """The cached keys and values of B sequences as packed 16-bit rows; returns
    (k, v), each [num_tokens, kv_heads, head_dim].

    ``page_table`` [B, max_pages] int32 names the pages of each sequence and
    ``indptr`` [B + 1] int32 the row its first token goes to.  Rows of no
    sequence are left as they are (``torch.empty`` when allocated here);
    tokens of a page outside the cache read as zeros.  ``dtype`` (bf16 by
    default) is that of the tensors allocated here.
    """
    if dtype is not None:
        name = str(dtype).removeprefix("torch.")
        if name not in ("bfloat16", "float16"):
            raise TypeError(f"unsupported dtype {dtype}")
        dtype = PQG_BF16 if name == "bfloat16" else PQG_FP16
    return _call((_native or native()).kv_read, stream, cache.device, cache.address, cache.index,
                 page_table, indptr, num_tokens, dtype, k_out, v_out)


def kv_attention(q, cache: KVCache, page_table, seq_lens, *, sm_scale: float | None = None,
                 max_len: int = 0, out=None, lse=None, return_lse: bool = False, stream=None):
    """Attention of each sequence's newest tokens over the cache; returns out, or
    (out, lse) with ``return_lse`` or a given ``lse``.

    ``q`` is a bf16/fp16 CUDA tensor [B * q_len, q_heads, head_dim], the q_len
    newest tokens of a sequence together, oldest first; the heads of a token are
    dense, tokens may be strided.  ``seq_lens`` [B] int32 counts each sequence's
    cached tokens, these included: token t of q_len sees the first
    seq_lens[b] - (q_len - 1 - t) of them.  Query head h reads key/value head
    h // (q_heads / kv_heads).  ``sm_scale`` defaults to head_dim ** -0.5.
    ``out`` is like ``q`` (dense); ``lse`` [B * q_len, q_heads] fp32 holds the
    natural logarithm of each row's sum of exponentials.  A row that sees no key
    gives zeros and -inf.  ``max_len``, the longest sequence's length, is a hint
    for splitting the keys among blocks (0: the page table's capacity).
    """
    got = _call((_native or native()).kv_attention, stream, cache.device, cache.address,
                cache.index, q, page_table, seq_lens,
                cache.head_dim ** -0.5 if sm_scale is None else sm_scale, max_len, out, lse,
                bool(return_lse))
    return got if len(got) == 2 else got[0]
