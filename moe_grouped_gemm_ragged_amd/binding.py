"""ctypes binding of libgg.so (the C ABI in include/gg.h).

Argument marshalling only: shapes, dtypes and devices are checked, outputs
are allocated with ``torch.empty`` when the caller passes none (the library
itself allocates nothing), and the pointers plus the current HIP stream go to
the C entry point of the same name.  Every step of the computation runs in
the HIP kernels; there is no fallback: if the library is missing or a call
fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libgg.so")
_HEADER = os.path.join(os.path.dirname(_PKG), "include", "gg.h")
_lib = None

GG_BF16 = 0
GG_F32 = 1

STATUS = {
    0: "GG_OK",
    1: "GG_ERR_NULL_PTR",
    2: "GG_ERR_BAD_DIM",
    3: "GG_ERR_ALIGNMENT",
    4: "GG_ERR_BAD_DTYPE",
    5: "GG_ERR_LIMIT",
    6: "GG_ERR_HIP",
}


class GGError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        self.status = status
        self.status_name = STATUS.get(status, str(status))
        super().__init__(f"{fn} failed: {self.status_name}: {message}")


def library_path() -> str:
    return _LIB_PATH


def header_path() -> str:
    return _HEADER


def load():
    """Load libgg.so (built in-tree by moe_grouped_gemm_ragged_amd.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"{_LIB_PATH} is missing: build it with `python -m moe_grouped_gemm_ragged_amd.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(_LIB_PATH)
    P = ctypes.c_void_p
    I64 = ctypes.c_int64
    I32 = ctypes.c_int32
    sig = [P, P, P, P, ctypes.c_int, I64, I64, I64, I32, P]
    for name in ("gg_forward", "gg_dgrad", "gg_wgrad", "gg_masked_forward", "gg_masked_dgrad",
                 "gg_masked_wgrad", "gg_forward_silu_mul", "gg_masked_forward_silu_mul",
                 "gg_forward_nk", "gg_dgrad_nk", "gg_wgrad_nk", "gg_masked_forward_nk"):
        f = getattr(lib, name)
        f.argtypes = sig
        f.restype = ctypes.c_int
    sig_ex = sig[:-1] + [ctypes.c_float, ctypes.c_float, P]
    for name in ("gg_forward_ex", "gg_dgrad_ex", "gg_wgrad_ex", "gg_masked_forward_ex",
                 "gg_masked_dgrad_ex", "gg_masked_wgrad_ex", "gg_forward_nk_ex", "gg_dgrad_nk_ex",
                 "gg_wgrad_nk_ex", "gg_masked_forward_nk_ex"):
        f = getattr(lib, name)
        f.argtypes = sig_ex
        f.restype = ctypes.c_int
    for name in ("gg_forward_bias", "gg_masked_forward_bias"):
        f = getattr(lib, name)
        f.argtypes = [P, P, P, P, P, P, ctypes.c_int, I64, I64, I64, I32, ctypes.c_float,
                      ctypes.c_float, P]
        f.restype = ctypes.c_int
    lib.gg_offsets_from_splits.argtypes = [P, I32, I32, ctypes.c_int, P, P]
    lib.gg_offsets_from_splits.restype = ctypes.c_int
    lib.gg_route_rows_bound.argtypes = [I64, I32, I32]
    lib.gg_route_rows_bound.restype = ctypes.c_int64
    lib.gg_route_workspace_bytes.argtypes = [I64, I32]
    lib.gg_route_workspace_bytes.restype = ctypes.c_int64
    lib.gg_route.argtypes = [P, I64, I32, I32, ctypes.c_int, P, P, I64, P, P, P]
    lib.gg_route.restype = ctypes.c_int
    lib.gg_route_noalloc.argtypes = [P, I64, I32, I32, ctypes.c_int, P, P, I64, P, P]
    lib.gg_route_noalloc.restype = ctypes.c_int
    lib.gg_gather_rows.argtypes = [P, I64, I64, P, I32, P, I32, I64, P, P]
    lib.gg_gather_rows.restype = ctypes.c_int
    lib.gg_combine_rows.argtypes = [P, I64, P, P, I32, I64, I64, P, ctypes.c_int, P]
    lib.gg_combine_rows.restype = ctypes.c_int
    for name in ("gg_bias_grad", "gg_masked_bias_grad", "gg_bias_scale_grad", "gg_masked_bias_scale_grad"):
        f = getattr(lib, name)
        f.argtypes = [P, P, P, P, I64, I64, I32, P]
        f.restype = ctypes.c_int
    lib.gg_fp8_scale_bytes.argtypes = [ctypes.c_int, I64, I64, I32]
    lib.gg_fp8_scale_bytes.restype = ctypes.c_int64
    lib.gg_fp8_pack_scales.argtypes = [ctypes.c_int, P, ctypes.c_int, I64, P, I64, I64, I32, P, P, P]
    lib.gg_fp8_pack_scales.restype = ctypes.c_int
    for name in ("gg_fp8_forward", "gg_fp8_masked_forward"):
        f = getattr(lib, name)
        f.argtypes = [P, P, P, P, P, P, ctypes.c_int, I64, I64, I64, I32, P]
        f.restype = ctypes.c_int
    F32 = ctypes.c_float
    for name in ("gg_fp8_wgrad", "gg_fp8_masked_wgrad"):
        f = getattr(lib, name)
        f.argtypes = [P, P, P, P, P, ctypes.c_int, I64, I64, I64, I32, F32, F32, P]
        f.restype = ctypes.c_int
    lib.gg_rmsnorm.argtypes = [P, P, P, P, P, P, P, I64, I64, F32, P]
    lib.gg_rmsnorm_grad.argtypes = [P, P, P, P, P, P, P, I64, I64, F32, P]
    lib.gg_fp8_gather_rows.argtypes = [P, P, I64, I64, P, I32, P, I32, I64, P, P, P]
    lib.gg_combine_rows_grad.argtypes = [P, ctypes.c_int, P, I64, P, P, P, I32, P, I32, I64, I64, P, P, P]
    for name in ("gg_silu_mul_rows", "gg_masked_silu_mul_rows"):
        getattr(lib, name).argtypes = [P, P, P, P, P, P, P, I64, I64, I32, P]
    for name in ("gg_silu_mul_grad", "gg_masked_silu_mul_grad"):
        getattr(lib, name).argtypes = [P, P, P, P, P, P, I64, I64, I32, P]
    for name in ("gg_rmsnorm", "gg_rmsnorm_grad", "gg_fp8_gather_rows", "gg_combine_rows_grad", "gg_silu_mul_rows",
                 "gg_masked_silu_mul_rows", "gg_silu_mul_grad", "gg_masked_silu_mul_grad"):
        getattr(lib, name).restype = ctypes.c_int
    lib.gg_rmsnorm_grad_workspace_bytes.argtypes = [I64, I64]
    lib.gg_rmsnorm_grad_workspace_bytes.restype = ctypes.c_int64
    lib.gg_fp4_scale_bytes.argtypes = [ctypes.c_int, I64, I64, I32]
    lib.gg_fp4_scale_bytes.restype = ctypes.c_int64
    for name, args in (("gg_fp4_pack_scales", [ctypes.c_int, P, I64, P, I64, I64, I32, P, P]),
                       ("gg_fp4_quantize", [ctypes.c_int, P, P, I64, I64, I32, P, P, P]),
                       ("gg_fp4_gather_rows", [P, I64, I64, P, I32, P, I32, I64, P, P, P]),
                       ("gg_fp4_silu_mul_rows", [P, P, P, P, I64, I64, I32, P]),
                       ("gg_fp4_masked_silu_mul_rows", [P, P, P, P, I64, I64, I32, P]),
                       ("gg_fp4_dequantize", [ctypes.c_int, P, P, P, I64, I64, I32, P, P]),
                       ("gg_fp4_forward", [P, P, P, P, P, P, ctypes.c_int, I64, I64, I64, I32, P]),
                       ("gg_fp4_masked_forward", [P, P, P, P, P, P, ctypes.c_int, I64, I64, I64, I32, P]),
                       ("gg_moe_few_tokens", [P, P, P, P, P, P, ctypes.c_int, P, I64, I32, I64, I64, I32, P]),
                       ("gg_fp4_moe_few_tokens",
                        [P, P, P, P, P, P, P, P, ctypes.c_int, P, I64, I32, I64, I64, I32, P])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = ctypes.c_int
    lib.gg_moe_few_tokens_workspace_bytes.argtypes = [I64, I32, I64, I32]
    lib.gg_moe_few_tokens_workspace_bytes.restype = ctypes.c_int64
    lib.gg_status_str.argtypes = [ctypes.c_int]
    lib.gg_status_str.restype = ctypes.c_char_p
    lib.gg_last_error.argtypes = []
    lib.gg_last_error.restype = ctypes.c_char_p
    lib.gg_version.argtypes = []
    lib.gg_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def header_symbols():
    """Names of the functions include/gg.h declares."""
    with open(_HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(gg_[a-z_]+)\s*\(", text)))


def call_raw(name: str, *args) -> int:
    """Call a C entry point with raw integer pointers/sizes; returns the
    gg_status code."""
    return int(getattr(load(), name)(*args))


def last_error() -> str:
    return load().gg_last_error().decode()


# ---------------------------------------------------------------------------
# torch-level helpers
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _dtype_code(dt) -> int:
    torch = _torch()
    if dt == torch.bfloat16:
        return GG_BF16
    if dt == torch.float32:
        return GG_F32
    raise TypeError(f"unsupported output dtype {dt}; use torch.bfloat16 or torch.float32")


def _check(t, name, dtype, ndim, device):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _launch(name, dev, *args):
    """Calls an entry point on ``dev``'s current stream, with ``dev`` current
    (a kernel goes to the current device)."""
    torch = _torch()
    if dev.type != "cuda":
        raise ValueError(f"{name}: the tensors are on {dev}, expected a GPU")
    f = getattr(load(), name)
    if torch.cuda.current_device() == dev.index:
        rc = f(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            rc = f(*args, _raw_stream(dev.index))
    if rc != 0:
        raise GGError(name, rc, last_error())


def _raw_stream(index):
    """The current stream's handle without a Stream object around it (2 us of
    a small call's 10), where this torch has that."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else int(torch.cuda.current_stream(index).cuda_stream)


def _invoke(name, a, b, groups, out, out_code, m, k, n, e, device, alpha=1.0, beta=0.0):
    """Calls the plain entry point, or its *_ex form when alpha != 1 or
    beta != 0."""
    ptrs = a.data_ptr(), b.data_ptr(), groups.data_ptr(), out.data_ptr()
    if float(alpha) == 1.0 and float(beta) == 0.0:
        _launch(name, device, *ptrs, out_code, int(m), int(k), int(n), int(e))
    else:
        _launch(name + "_ex", device, *ptrs, out_code, int(m), int(k), int(n), int(e), float(alpha), float(beta))


def _need_out(out, beta):
    if float(beta) != 0.0 and out is None:
        raise ValueError("beta != 0 accumulates into `out`, which must be given")


def forward(x, w, offs, out: Optional["torch.Tensor"] = None, out_dtype=None, alpha=1.0, beta=0.0):
    """Y[rows of g] = X[rows of g] . W[g] (gg_forward).  x: bf16 [m,k];
    w: bf16 [E,k,n]; offs: int32 [E] cumulative end offsets on the device.
    Rows of ``out`` at or past offs[-1] are left untouched.  With alpha /
    beta, the written rows become alpha * product + beta * out
    (gg_forward_ex)."""
    torch = _torch()
    _need_out(out, beta)
    dev = x.device
    _check(x, "x", torch.bfloat16, 2, dev)
    _check(w, "w", torch.bfloat16, 3, dev)
    _check(offs, "offs", torch.int32, 1, dev)
    m, k = x.shape
    e, k2, n = w.shape
    if k2 != k or offs.shape[0] != e:
        raise ValueError("shape mismatch between x, w and offs")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=dev)
    _check(out, "out", out.dtype, 2, dev)
    if tuple(out.shape) != (m, n):
        raise ValueError(f"out must be [{m}, {n}]")
    _invoke("gg_forward", x, w, offs, out, _dtype_code(out.dtype), m, k, n, e, dev, alpha, beta)
    return out


def dgrad(dy, w, offs, out=None, out_dtype=None, alpha=1.0, beta=0.0):
    """dX[rows of g] = dY[rows of g] . W[g]^T (gg_dgrad).  dy: bf16 [m,n].
    alpha / beta as in forward (gg_dgrad_ex)."""
    torch = _torch()
    _need_out(out, beta)
    dev = dy.device
    _check(dy, "dy", torch.bfloat16, 2, dev)
    _check(w, "w", torch.bfloat16, 3, dev)
    _check(offs, "offs", torch.int32, 1, dev)
    m, n = dy.shape
    e, k, n2 = w.shape
    if n2 != n or offs.shape[0] != e:
        raise ValueError("shape mismatch between dy, w and offs")
    if out is None:
        out = torch.empty((m, k), dtype=out_dtype or torch.bfloat16, device=dev)
    _check(out, "out", out.dtype, 2, dev)
    if tuple(out.shape) != (m, k):
        raise ValueError(f"out must be [{m}, {k}]")
    _invoke("gg_dgrad", dy, w, offs, out, _dtype_code(out.dtype), m, k, n, e, dev, alpha, beta)
    return out


def wgrad(x, dy, offs, out=None, out_dtype=None, alpha=1.0, beta=0.0):
    """dW[g] = X[rows of g]^T . dY[rows of g] for every expert (gg_wgrad);
    all of ``out`` [E,k,n] is written, empty experts get +0.0.  beta = 1
    accumulates into ``out`` (e.g. an fp32 main-grad; gg_wgrad_ex)."""
    torch = _torch()
    _need_out(out, beta)
    dev = x.device
    _check(x, "x", torch.bfloat16, 2, dev)
    _check(dy, "dy", torch.bfloat16, 2, dev)
    _check(offs, "offs", torch.int32, 1, dev)
    m, k = x.shape
    m2, n = dy.shape
    e = offs.shape[0]
    if m2 != m:
        raise ValueError("x and dy must have the same number of rows")
    if out is None:
        out = torch.empty((e, k, n), dtype=out_dtype or torch.float32, device=dev)
    _check(out, "out", out.dtype, 3, dev)
    if tuple(out.shape) != (e, k, n):
        raise ValueError(f"out must be [{e}, {k}, {n}]")
    _invoke("gg_wgrad", x, dy, offs, out, _dtype_code(out.dtype), m, k, n, e, dev, alpha, beta)
    return out


def masked_forward(x, w, masked_m, out=None, out_dtype=None, alpha=1.0, beta=0.0):
    """Y[e, r] = X[e, r] . W[e] for r < masked_m[e] (gg_masked_forward).
    x: bf16 [E, max_m, k]; inactive rows are neither read nor written.
    alpha / beta as in forward (gg_masked_forward_ex)."""
    torch = _torch()
    _need_out(out, beta)
    dev = x.device
    _check(x, "x", torch.bfloat16, 3, dev)
    _check(w, "w", torch.bfloat16, 3, dev)
    _check(masked_m, "masked_m", torch.int32, 1, dev)
    e, max_m, k = x.shape
    e2, k2, n = w.shape
    if e2 != e or k2 != k or masked_m.shape[0] != e:
        raise ValueError("shape mismatch between x, w and masked_m")
    if out is None:
        out = torch.empty((e, max_m, n), dtype=out_dtype or torch.bfloat16, device=dev)
    _check(out, "out", out.dtype, 3, dev)
    if tuple(out.shape) != (e, max_m, n):
        raise ValueError(f"out must be [{e}, {max_m}, {n}]")
    _invoke("gg_masked_forward", x, w, masked_m, out, _dtype_code(out.dtype), max_m, k, n, e, dev,
            alpha, beta)
    return out


def masked_dgrad(dy, w, masked_m, out=None, out_dtype=None, alpha=1.0, beta=0.0):
    """dX[e, r] = dY[e, r] . W[e]^T for r < masked_m[e] (gg_masked_dgrad).
    dy: bf16 [E, max_m, n]; w: bf16 [E, k, n]; only active rows of ``out``
    [E, max_m, k] are written."""
    torch = _torch()
    _need_out(out, beta)
    dev = dy.device
    _check(dy, "dy", torch.bfloat16, 3, dev)
    _check(w, "w", torch.bfloat16, 3, dev)
    _check(masked_m, "masked_m", torch.int32, 1, dev)
    e, max_m, n = dy.shape
    e2, k, n2 = w.shape
    if e2 != e or n2 != n or masked_m.shape[0] != e:
        raise ValueError("shape mismatch between dy, w and masked_m")
    if out is None:
        out = torch.empty((e, max_m, k), dtype=out_dtype or torch.bfloat16, device=dev)
    _check(out, "out", out.dtype, 3, dev)
    if tuple(out.shape) != (e, max_m, k):
        raise ValueError(f"out must be [{e}, {max_m}, {k}]")
    _invoke("gg_masked_dgrad", dy, w, masked_m, out, _dtype_code(out.dtype), max_m, k, n, e, dev,
            alpha, beta)
    return out


def masked_wgrad(x, dy, masked_m, out=None, out_dtype=None, alpha=1.0, beta=0.0):
    """dW[e] = X[e, :a]^T . dY[e, :a], a = masked_m[e] clamped, for every
    expert (gg_masked_wgrad); all of ``out`` [E, k, n] is written."""
    torch = _torch()
    _need_out(out, beta)
    dev = x.device
    _check(x, "x", torch.bfloat16, 3, dev)
    _check(dy, "dy", torch.bfloat16, 3, dev)
    _check(masked_m, "masked_m", torch.int32, 1, dev)
    e, max_m, k = x.shape
    e2, max_m2, n = dy.shape
    if e2 != e or max_m2 != max_m or masked_m.shape[0] != e:
        raise ValueError("shape mismatch between x, dy and masked_m")
    if out is None:
        out = torch.empty((e, k, n), dtype=out_dtype or torch.float32, device=dev)
    _check(out, "out", out.dtype, 3, dev)
    if tuple(out.shape) != (e, k, n):
        raise ValueError(f"out must be [{e}, {k}, {n}]")
    _invoke("gg_masked_wgrad", x, dy, masked_m, out, _dtype_code(out.dtype), max_m, k, n, e, dev,
            alpha, beta)
    return out


def forward_silu_mul(x, w13, offs, out=None, out_dtype=None):
    """out[i, c] = silu(G)[i, c] * U[i, c] with [G | U] = X[rows of g] .
    W13[g] (gg_forward_silu_mul).  x: bf16 [m, k]; w13: bf16 [E, k, 2I]
    (gate columns, then up); returns [m, I]."""
    torch = _torch()
    dev = x.device
    _check(x, "x", torch.bfloat16, 2, dev)
    _check(w13, "w13", torch.bfloat16, 3, dev)
    _check(offs, "offs", torch.int32, 1, dev)
    m, k = x.shape
    e, k2, n = w13.shape
    if k2 != k or offs.shape[0] != e or n % 2:
        raise ValueError("shape mismatch between x, w13 and offs")
    if out is None:
        out = torch.empty((m, n // 2), dtype=out_dtype or torch.bfloat16, device=dev)
    _check(out, "out", out.dtype, 2, dev)
    if tuple(out.shape) != (m, n // 2):
        raise ValueError(f"out must be [{m}, {n // 2}]")
    _invoke("gg_forward_silu_mul", x, w13, offs, out, _dtype_code(out.dtype), m, k, n, e, dev)
    return out


def masked_forward_silu_mul(x, w13, masked_m, out=None, out_dtype=None):
    """The masked layout's gate/up forward with the SiLU-mul activation
    (gg_masked_forward_silu_mul): x bf16 [E, max_m, k] -> [E, max_m, I]."""
    torch = _torch()
    dev = x.device
    _check(x, "x", torch.bfloat16, 3, dev)
    _check(w13, "w13", torch.bfloat16, 3, dev)
    _check(masked_m, "masked_m", torch.int32, 1, dev)
    e, max_m, k = x.shape
    e2, k2, n = w13.shape
    if e2 != e or k2 != k or masked_m.shape[0] != e or n % 2:
        raise ValueError("shape mismatch between x, w13 and masked_m")
    if out is None:
        out = torch.empty((e, max_m, n // 2), dtype=out_dtype or torch.bfloat16, device=dev)
    _check(out, "out", out.dtype, 3, dev)
    if tuple(out.shape) != (e, max_m, n // 2):
        raise ValueError(f"out must be [{e}, {max_m}, {n // 2}]")
    _invoke("gg_masked_forward_silu_mul", x, w13, masked_m, out, _dtype_code(out.dtype), max_m, k, n,
            e, dev)
    return out


# ---------------------------------------------------------------------------
# producing the grouped layout
# ---------------------------------------------------------------------------

def offsets_from_splits(m_splits, min_alignment=1, pad_empty=False, out=None):
    """int32 end offsets from int64 per-expert row counts on the device
    (gg_offsets_from_splits), each count padded to min_alignment."""
    torch = _torch()
    dev = m_splits.device
    _check(m_splits, "m_splits", torch.int64, 1, dev)
    e = m_splits.shape[0]
    if out is None:
        out = torch.empty(e, dtype=torch.int32, device=dev)
    _check(out, "out", torch.int32, 1, dev)
    _launch("gg_offsets_from_splits", dev, m_splits.data_ptr(), int(e), int(min_alignment), 1 if pad_empty else 0,
            out.data_ptr())
    return out


def route_rows_bound(slots, num_groups, min_alignment=1) -> int:
    v = int(load().gg_route_rows_bound(int(slots), int(num_groups), int(min_alignment)))
    if v < 0:
        raise ValueError("invalid arguments for gg_route_rows_bound")
    return v


def route(expert_of_slot, num_groups, min_alignment=1, pad_empty=False, rows_cap=None):
    """Token slots -> grouped layout (gg_route).  expert_of_slot: int32
    [tokens, topk] (or flat) expert ids.  Returns (offs int32 [E], row_slot
    int32 [rows_cap], slot_row int32 [slots]); row_slot past offs[-1] is
    uninitialised."""
    torch = _torch()
    dev = expert_of_slot.device
    if expert_of_slot.dtype != torch.int32 or not expert_of_slot.is_contiguous():
        raise TypeError("expert_of_slot must be a contiguous int32 tensor")
    slots = expert_of_slot.numel()
    cap = route_rows_bound(slots, num_groups, min_alignment) if rows_cap is None else int(rows_cap)
    offs = torch.empty(num_groups, dtype=torch.int32, device=dev)
    row_slot = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    slot_row = torch.empty(max(slots, 1), dtype=torch.int32, device=dev)
    ws = torch.empty(int(load().gg_route_workspace_bytes(slots, num_groups)), dtype=torch.uint8, device=dev)
    _launch("gg_route", dev, expert_of_slot.data_ptr(), int(slots), int(num_groups), int(min_alignment),
            1 if pad_empty else 0, offs.data_ptr(), row_slot.data_ptr(), int(cap), slot_row.data_ptr(), ws.data_ptr())
    return offs, row_slot[:cap], slot_row[:slots]


def gather_rows(src, row_slot, topk, offs, out=None):
    """Grouped rows from token rows (gg_gather_rows): src [tokens, ...]
    (any dtype, rows a multiple of 16 bytes); returns [len(row_slot), ...]."""
    torch = _torch()
    dev = src.device
    if not src.is_contiguous():
        raise ValueError("src must be contiguous")
    tokens = src.shape[0]
    row_bytes = src[0].numel() * src.element_size() if tokens else src.shape[1:].numel() * src.element_size()
    rows_cap = row_slot.shape[0]
    if out is None:
        out = torch.empty((rows_cap, *src.shape[1:]), dtype=src.dtype, device=dev)
    _launch("gg_gather_rows", dev, src.data_ptr(), int(tokens), int(row_bytes), row_slot.data_ptr(), int(topk),
            offs.data_ptr(), int(offs.shape[0]), int(rows_cap), out.data_ptr())
    return out


def combine_rows(y, slot_row, topk, weights=None, out=None, out_dtype=None):
    """out[t] = sum_k w[t, k] y[slot_row[t topk + k]] (gg_combine_rows): y
    bf16 [rows, n]; weights fp32 [tokens, topk] or None."""
    torch = _torch()
    dev = y.device
    _check(y, "y", torch.bfloat16, 2, dev)
    rows_cap, n = y.shape
    slots = slot_row.numel()
    tokens = slots // topk
    if out is None:
        out = torch.empty((tokens, n), dtype=out_dtype or torch.bfloat16, device=dev)
    _launch("gg_combine_rows", dev, y.data_ptr(), int(n), slot_row.data_ptr(),
            None if weights is None else weights.data_ptr(), int(topk), int(tokens), int(rows_cap), out.data_ptr(),
            _dtype_code(out.dtype))
    return out


# ---------------------------------------------------------------------------
# grouped bias with a per-token factor
# ---------------------------------------------------------------------------

def _bias_call(name, x, w, groups, bias, bias_scale, out, m, k, n, e, dev, alpha, beta):
    torch = _torch()
    _check(bias, "bias", torch.bfloat16, 2, dev)
    if tuple(bias.shape) != (e, n):
        raise ValueError(f"bias must be [{e}, {n}]")
    if bias_scale is not None:
        if bias_scale.dtype != torch.float32 or bias_scale.device != dev or not bias_scale.is_contiguous():
            raise TypeError("bias_scale must be a contiguous float32 tensor on the device")
    _launch(name, dev, x.data_ptr(), w.data_ptr(), groups.data_ptr(), bias.data_ptr(),
            None if bias_scale is None else bias_scale.data_ptr(), out.data_ptr(), _dtype_code(out.dtype), int(m),
            int(k), int(n), int(e), float(alpha), float(beta))


def forward_bias(x, w, offs, bias, bias_scale=None, out=None, out_dtype=None, alpha=1.0, beta=0.0):
    """Y[i] = alpha X[i] W[g] + beta Y[i] + s[i] bias[g] on the rows of each
    expert (gg_forward_bias).  bias: bf16 [E, n]; bias_scale: fp32 with at
    least offs[-1] entries (the logical tokens), or None for 1."""
    torch = _torch()
    _need_out(out, beta)
    dev = x.device
    _check(x, "x", torch.bfloat16, 2, dev)
    _check(w, "w", torch.bfloat16, 3, dev)
    _check(offs, "offs", torch.int32, 1, dev)
    m, k = x.shape
    e, k2, n = w.shape
    if k2 != k or offs.shape[0] != e:
        raise ValueError("shape mismatch between x, w and offs")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=dev)
    _check(out, "out", out.dtype, 2, dev)
    if tuple(out.shape) != (m, n):
        raise ValueError(f"out must be [{m}, {n}]")
    _bias_call("gg_forward_bias", x, w, offs, bias, bias_scale, out, m, k, n, e, dev, alpha, beta)
    return out


def masked_forward_bias(x, w, masked_m, bias, bias_scale=None, out=None, out_dtype=None, alpha=1.0,
                        beta=0.0):
    """The masked forward plus s[e, r] bias[e] on active rows
    (gg_masked_forward_bias); bias_scale: fp32 [E, max_m] or None."""
    torch = _torch()
    _need_out(out, beta)
    dev = x.device
    _check(x, "x", torch.bfloat16, 3, dev)
    _check(w, "w", torch.bfloat16, 3, dev)
    _check(masked_m, "masked_m", torch.int32, 1, dev)
    e, max_m, k = x.shape
    e2, k2, n = w.shape
    if e2 != e or k2 != k or masked_m.shape[0] != e:
        raise ValueError("shape mismatch between x, w and masked_m")
    if out is None:
        out = torch.empty((e, max_m, n), dtype=out_dtype or torch.bfloat16, device=dev)
    _check(out, "out", out.dtype, 3, dev)
    if tuple(out.shape) != (e, max_m, n):
        raise ValueError(f"out must be [{e}, {max_m}, {n}]")
    _bias_call("gg_masked_forward_bias", x, w, masked_m, bias, bias_scale, out, max_m, k, n, e, dev,
               alpha, beta)
    return out


def bias_grad(dy, groups, bias_scale=None, masked=False, out=None):
    """dbias[g] = sum_{i in g} s[i] dY[i] (gg_bias_grad / gg_masked_bias_grad):
    dy bf16 [m, n] or [E, max_m, n]; returns fp32 [E, n]."""
    torch = _torch()
    dev = dy.device
    _check(dy, "dy", torch.bfloat16, 3 if masked else 2, dev)
    _check(groups, "groups", torch.int32, 1, dev)
    e = groups.shape[0]
    rows, n = (dy.shape[1], dy.shape[2]) if masked else (dy.shape[0], dy.shape[1])
    if out is None:
        out = torch.empty((e, n), dtype=torch.float32, device=dev)
    _check(out, "out", torch.float32, 2, dev)
    name = "gg_masked_bias_grad" if masked else "gg_bias_grad"
    _launch(name, dev, dy.data_ptr(), groups.data_ptr(), None if bias_scale is None else bias_scale.data_ptr(),
            out.data_ptr(), int(rows), int(n), int(e))
    return out


def bias_scale_grad(dy, groups, bias, masked=False, out=None):
    """ds[i] = <bias[g], dY[i]> on the rows an expert owns
    (gg_bias_scale_grad / gg_masked_bias_scale_grad); returns fp32 [rows]
    (other entries as ``out`` held them; NaN when allocated here)."""
    torch = _torch()
    dev = dy.device
    _check(dy, "dy", torch.bfloat16, 3 if masked else 2, dev)
    _check(groups, "groups", torch.int32, 1, dev)
    _check(bias, "bias", torch.bfloat16, 2, dev)
    e = groups.shape[0]
    rows, n = (dy.shape[1], dy.shape[2]) if masked else (dy.shape[0], dy.shape[1])
    total = e * rows if masked else rows
    if out is None:
        out = torch.full((total,), float("nan"), dtype=torch.float32, device=dev)
    _check(out, "out", torch.float32, 1, dev)
    name = "gg_masked_bias_scale_grad" if masked else "gg_bias_scale_grad"
    _launch(name, dev, dy.data_ptr(), groups.data_ptr(), bias.data_ptr(), out.data_ptr(), int(rows), int(n), int(e))
    return out


# ---------------------------------------------------------------------------
# [E, N, K] weight layout
# ---------------------------------------------------------------------------

def forward_nk(x, w, offs, out=None, out_dtype=None, alpha=1.0, beta=0.0):
    """Y = X W[g]^T with W [E, n, k] (gg_forward_nk).  x: bf16 [m, k]."""
    torch = _torch()
    _need_out(out, beta)
    dev = x.device
    _check(x, "x", torch.bfloat16, 2, dev)
    _check(w, "w", torch.bfloat16, 3, dev)
    _check(offs, "offs", torch.int32, 1, dev)
    m, k = x.shape
    e, n, k2 = w.shape
    if k2 != k or offs.shape[0] != e:
        raise ValueError("shape mismatch between x, w and offs")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=dev)
    _check(out, "out", out.dtype, 2, dev)
    if tuple(out.shape) != (m, n):
        raise ValueError(f"out must be [{m}, {n}]")
    _invoke("gg_forward_nk", x, w, offs, out, _dtype_code(out.dtype), m, k, n, e, dev, alpha, beta)
    return out


def dgrad_nk(dy, w, offs, out=None, out_dtype=None, alpha=1.0, beta=0.0):
    """dX = dY W[g] with W [E, n, k] (gg_dgrad_nk).  dy: bf16 [m, n]."""
    torch = _torch()
    _need_out(out, beta)
    dev = dy.device
    _check(dy, "dy", torch.bfloat16, 2, dev)
    _check(w, "w", torch.bfloat16, 3, dev)
    _check(offs, "offs", torch.int32, 1, dev)
    m, n = dy.shape
    e, n2, k = w.shape
    if n2 != n or offs.shape[0] != e:
        raise ValueError("shape mismatch between dy, w and offs")
    if out is None:
        out = torch.empty((m, k), dtype=out_dtype or torch.bfloat16, device=dev)
    _check(out, "out", out.dtype, 2, dev)
    if tuple(out.shape) != (m, k):
        raise ValueError(f"out must be [{m}, {k}]")
    _invoke("gg_dgrad_nk", dy, w, offs, out, _dtype_code(out.dtype), m, k, n, e, dev, alpha, beta)
    return out


def wgrad_nk(x, dy, offs, out=None, out_dtype=None, alpha=1.0, beta=0.0):
    """dW[g] = dY[rows of g]^T X[rows of g], dW as [E, n, k] (gg_wgrad_nk)."""
    torch = _torch()
    _need_out(out, beta)
    dev = x.device
    _check(x, "x", torch.bfloat16, 2, dev)
    _check(dy, "dy", torch.bfloat16, 2, dev)
    _check(offs, "offs", torch.int32, 1, dev)
    m, k = x.shape
    m2, n = dy.shape
    e = offs.shape[0]
    if m2 != m:
        raise ValueError("x and dy must have the same rows")
    if out is None:
        out = torch.empty((e, n, k), dtype=out_dtype or torch.float32, device=dev)
    _check(out, "out", out.dtype, 3, dev)
    if tuple(out.shape) != (e, n, k):
        raise ValueError(f"out must be [{e}, {n}, {k}]")
    _invoke("gg_wgrad_nk", x, dy, offs, out, _dtype_code(out.dtype), m, k, n, e, dev, alpha, beta)
    return out


def masked_forward_nk(x, w, masked_m, out=None, out_dtype=None, alpha=1.0, beta=0.0):
    """The masked forward with W [E, n, k] (gg_masked_forward_nk)."""
    torch = _torch()
    _need_out(out, beta)
    dev = x.device
    _check(x, "x", torch.bfloat16, 3, dev)
    _check(w, "w", torch.bfloat16, 3, dev)
    _check(masked_m, "masked_m", torch.int32, 1, dev)
    e, max_m, k = x.shape
    e2, n, k2 = w.shape
    if e2 != e or k2 != k or masked_m.shape[0] != e:
        raise ValueError("shape mismatch between x, w and masked_m")
    if out is None:
        out = torch.empty((e, max_m, n), dtype=out_dtype or torch.bfloat16, device=dev)
    _check(out, "out", out.dtype, 3, dev)
    if tuple(out.shape) != (e, max_m, n):
        raise ValueError(f"out must be [{e}, {max_m}, {n}]")
    _invoke("gg_masked_forward_nk", x, w, masked_m, out, _dtype_code(out.dtype), max_m, k, n, e, dev,
            alpha, beta)
    return out


# ---------------------------------------------------------------------------
# fp8 (e4m3) block-scaled forward
# ---------------------------------------------------------------------------

GG_FP8_ACT_RAGGED = 0
GG_FP8_ACT_MASKED = 1
GG_FP8_WEIGHT = 2


def fp8_scale_bytes(layout: int, rows: int, k: int, num_groups: int) -> int:
    """Bytes of packed scales (gg_fp8_scale_bytes)."""
    v = int(load().gg_fp8_scale_bytes(int(layout), int(rows), int(k), int(num_groups)))
    if v < 0:
        raise ValueError("invalid arguments for gg_fp8_scale_bytes")
    return v


def fp8_pack_scales(layout: int, scales, groups, rows: int, k: int, num_groups: int,
                    out=None, bad_count=None):
    """Packed E8M0 scales of one operand (gg_fp8_pack_scales).  scales: fp32
    or uint8 (E8M0 bytes) with one scale per (row, k-block) in its last dim
    (rows flattened: [m, G], [E, max_m, G] or [E, n, G]; G may be padded);
    groups: the int32 end offsets / masked_m (ignored for weights);
    bad_count: optional int32 [1] device tensor the kernel adds the number of
    active non-UE8M0 scales to.  Returns the packed uint8 tensor."""
    torch = _torch()
    dev = scales.device
    if scales.dtype not in (torch.float32, torch.uint8):
        raise TypeError("scales must be float32 or uint8 (E8M0 bytes)")
    if not scales.is_contiguous():
        raise ValueError("scales must be contiguous")
    if groups is not None:
        _check(groups, "groups", torch.int32, 1, dev)
    nbytes = fp8_scale_bytes(layout, rows, k, num_groups)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(out, "out", torch.uint8, 1, dev)
    if out.numel() < nbytes:
        raise ValueError(f"out must hold {nbytes} bytes")
    if bad_count is not None:
        _check(bad_count, "bad_count", torch.int32, 1, dev)
    _launch("gg_fp8_pack_scales", dev, int(layout), scales.data_ptr(), 1 if scales.dtype == torch.float32 else 0,
            int(scales.shape[-1]), None if groups is None else groups.data_ptr(), int(rows), int(k), int(num_groups),
            out.data_ptr(), None if bad_count is None else bad_count.data_ptr())
    return out


def _fp8_call(name, x, xs, w, ws, groups, out, m, k, n, e, dev):
    _launch(name, dev, x.data_ptr(), xs.data_ptr(), w.data_ptr(), ws.data_ptr(), groups.data_ptr(), out.data_ptr(),
            _dtype_code(out.dtype), int(m), int(k), int(n), int(e))


def fp8_forward(x, x_scales, w, w_scales, offs, out=None, out_dtype=None):
    """Y[rows of g] = sum_k x sx w[g] sw over 128-value scale blocks
    (gg_fp8_forward).  x: uint8 e4m3 [m, k]; w: uint8 e4m3 [E, n, k];
    x_scales / w_scales: packed by fp8_pack_scales (GG_FP8_ACT_RAGGED with
    the same offs / GG_FP8_WEIGHT); offs: int32 [E] end offsets."""
    torch = _torch()
    dev = x.device
    _check(x, "x", torch.uint8, 2, dev)
    _check(w, "w", torch.uint8, 3, dev)
    _check(offs, "offs", torch.int32, 1, dev)
    _check(x_scales, "x_scales", torch.uint8, 1, dev)
    _check(w_scales, "w_scales", torch.uint8, 1, dev)
    m, k = x.shape
    e, n, k2 = w.shape
    if k2 != k or offs.shape[0] != e:
        raise ValueError("shape mismatch between x, w and offs")
    if x_scales.numel() < fp8_scale_bytes(GG_FP8_ACT_RAGGED, m, k, e) or \
            w_scales.numel() < fp8_scale_bytes(GG_FP8_WEIGHT, n, k, e):
        raise ValueError("packed scales are smaller than fp8_scale_bytes requires")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=dev)
    _check(out, "out", out.dtype, 2, dev)
    if tuple(out.shape) != (m, n):
        raise ValueError(f"out must be [{m}, {n}]")
    _fp8_call("gg_fp8_forward", x, x_scales, w, w_scales, offs, out, m, k, n, e, dev)
    return out


def fp8_masked_forward(x, x_scales, w, w_scales, masked_m, out=None, out_dtype=None):
    """The masked fp8 forward (gg_fp8_masked_forward): x uint8 [E, max_m, k],
    x_scales packed with GG_FP8_ACT_MASKED and the same masked_m."""
    torch = _torch()
    dev = x.device
    _check(x, "x", torch.uint8, 3, dev)
    _check(w, "w", torch.uint8, 3, dev)
    _check(masked_m, "masked_m", torch.int32, 1, dev)
    _check(x_scales, "x_scales", torch.uint8, 1, dev)
    _check(w_scales, "w_scales", torch.uint8, 1, dev)
    e, max_m, k = x.shape
    e2, n, k2 = w.shape
    if e2 != e or k2 != k or masked_m.shape[0] != e:
        raise ValueError("shape mismatch between x, w and masked_m")
    if x_scales.numel() < fp8_scale_bytes(GG_FP8_ACT_MASKED, max_m, k, e) or \
            w_scales.numel() < fp8_scale_bytes(GG_FP8_WEIGHT, n, k, e):
        raise ValueError("packed scales are smaller than fp8_scale_bytes requires")
    if out is None:
        out = torch.empty((e, max_m, n), dtype=out_dtype or torch.bfloat16, device=dev)
    _check(out, "out", out.dtype, 3, dev)
    if tuple(out.shape) != (e, max_m, n):
        raise ValueError(f"out must be [{e}, {max_m}, {n}]")
    _fp8_call("gg_fp8_masked_forward", x, x_scales, w, w_scales, masked_m, out, max_m, k, n, e, dev)
    return out


# ---------------------------------------------------------------------------
# norm, 8-bit gather, combine gradient, SiLU-mul rows
# ---------------------------------------------------------------------------

def _shaped(t, name, dtype, shape, device, like=None):
    """``t`` checked against a shape (of up to 3 dimensions), or a new tensor
    of it (that ``like`` has too, where there is one: the cheapest call)."""
    torch = _torch()
    if t is None:
        if like is not None:
            return torch.empty_like(like)
        # (with its strides: 0.4 us less than torch.empty, of a small call's 9 to 13)
        strides = (shape[1], 1) if len(shape) == 2 else (1,) if len(shape) == 1 else (shape[1] * shape[2], shape[2], 1)
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)
    # everything at once where all is well (half the time of naming what is not)
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype and t.device == device
            and t.is_contiguous()):
        return t
    _check(t, name, dtype, len(shape), device)
    raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rmsnorm(x, gamma, residual, eps, y, y8, scales, h):
    torch = _torch()
    dev = x.device
    rows, n = x.shape
    _shaped(gamma, "gamma", torch.bfloat16, (n,), dev)
    if residual is not None:
        _shaped(residual, "residual", torch.bfloat16, (rows, n), dev)
        h = _shaped(h, "h_out", torch.bfloat16, (rows, n), dev, like=x)
    elif h is not None:
        raise ValueError("h_out without a residual: h is x itself")
    _launch("gg_rmsnorm", dev, _ptr(x), _ptr(residual), _ptr(gamma), _ptr(h), _ptr(y), _ptr(y8), _ptr(scales), rows,
            n, float(eps))
    return h


def rmsnorm(x, gamma, residual=None, eps=1e-6, out=None, h_out=None):
    """y = RMSNorm(x + residual) * gamma (gg_rmsnorm): bf16 [rows, n], gamma
    bf16 [n].  Returns (y, h) with h = x + residual in bf16 (``h_out``, which
    may be ``residual`` or ``x``), or h = None without a residual."""
    torch = _torch()
    _check(x, "x", torch.bfloat16, 2, x.device)
    y = _shaped(out, "out", torch.bfloat16, x.shape, x.device, like=x)
    h = _rmsnorm(x, gamma, residual, eps, y, None, None, h_out)
    return y, h


def fp8_rmsnorm(x, gamma, residual=None, eps=1e-6, out=None, out_scales=None, h_out=None, with_bf16=False,
                y_out=None):
    """rmsnorm with y as e4m3 rows: uint8 codes [rows, n] and E8M0 bytes
    [rows, n / 128] (n a multiple of 128).  Returns (codes, scales, h), or
    (codes, scales, h, y) with the bf16 y too (``with_bf16``, or a buffer for
    it)."""
    torch = _torch()
    dev = x.device
    _check(x, "x", torch.bfloat16, 2, dev)
    rows, n = x.shape
    if n % 128:
        raise ValueError("x must be [rows, n] with n a multiple of 128")
    y8 = _shaped(out, "out", torch.uint8, (rows, n), dev)
    scales = _shaped(out_scales, "out_scales", torch.uint8, (rows, n // 128), dev)
    y = None
    if with_bf16 or y_out is not None:
        y = _shaped(y_out, "y_out", torch.bfloat16, x.shape, dev, like=x)
    h = _rmsnorm(x, gamma, residual, eps, y, y8, scales, h_out)
    return (y8, scales, h) if y is None else (y8, scales, h, y)


def rmsnorm_grad_workspace_bytes(rows, n) -> int:
    v = int(load().gg_rmsnorm_grad_workspace_bytes(int(rows), int(n)))
    if v < 0:
        raise ValueError("invalid arguments for gg_rmsnorm_grad_workspace_bytes")
    return v


def rmsnorm_grad(dy, h, gamma, dh=None, eps=1e-6, out=None, dgamma=None, workspace=None):
    """Gradient of rmsnorm at h (gg_rmsnorm_grad): dy, h bf16 [rows, n]; dh:
    the gradient that reaches h through the residual stream, or None.  Returns
    (dx bf16 [rows, n] -- of x and of residual alike -- and dgamma fp32 [n])."""
    torch = _torch()
    dev = dy.device
    _check(dy, "dy", torch.bfloat16, 2, dev)
    rows, n = dy.shape
    _shaped(h, "h", torch.bfloat16, (rows, n), dev)
    _shaped(gamma, "gamma", torch.bfloat16, (n,), dev)
    if dh is not None:
        _shaped(dh, "dh", torch.bfloat16, (rows, n), dev)
    dx = _shaped(out, "out", torch.bfloat16, (rows, n), dev, like=dy)
    dgamma = _shaped(dgamma, "dgamma", torch.float32, (n,), dev)
    need = rmsnorm_grad_workspace_bytes(rows, n)
    if workspace is None:
        workspace = _shaped(None, "workspace", torch.uint8, (need,), dev)
    _check(workspace, "workspace", torch.uint8, 1, dev)
    if workspace.numel() < need:
        raise ValueError(f"workspace must hold {need} bytes")
    _launch("gg_rmsnorm_grad", dev, _ptr(dy), _ptr(h), _ptr(gamma), _ptr(dh), _ptr(dx), _ptr(dgamma), _ptr(workspace),
            rows, n, float(eps))
    return dx, dgamma


def fp8_gather_rows(src, scales, row_slot, topk, offs, out=None, out_scales=None):
    """e4m3 rows and their scales sorted by expert (gg_fp8_gather_rows): src
    uint8 [tokens, k], scales uint8 E8M0 [tokens, k / 128]; row_slot and offs
    from ``route``.  Returns (codes [len(row_slot), k], packed scales) as
    ``fp8_forward`` takes them; rows past offs[-1] are left untouched."""
    torch = _torch()
    dev = src.device
    _check(src, "src", torch.uint8, 2, dev)
    tokens, k = src.shape
    if k % 128:
        raise ValueError("src must be [tokens, k] with k a multiple of 128")
    _shaped(scales, "scales", torch.uint8, (tokens, k // 128), dev)
    _check(row_slot, "row_slot", torch.int32, 1, dev)
    _check(offs, "offs", torch.int32, 1, dev)
    cap, e = row_slot.shape[0], offs.shape[0]
    out = _shaped(out, "out", torch.uint8, (cap, k), dev)
    out_scales = _shaped(out_scales, "out_scales", torch.uint8, (fp8_scale_bytes(GG_FP8_ACT_RAGGED, cap, k, e),), dev)
    _launch("gg_fp8_gather_rows", dev, _ptr(src), _ptr(scales), tokens, k, _ptr(row_slot), int(topk), _ptr(offs), e,
            cap, _ptr(out), _ptr(out_scales))
    return out, out_scales


def combine_rows_grad(dout, y, slot_row, row_slot, offs, topk, weights=None, out=None, with_weights=True,
                      dweights=None):
    """Gradient of combine_rows (gg_combine_rows_grad): dout bf16 or fp32
    [tokens, n], y bf16 [rows, n] (None without ``with_weights``), and the
    routing.  Returns (dy bf16 [len(row_slot), n], dweights fp32 [tokens,
    topk] or None); rows of dy past offs[-1] are left untouched."""
    torch = _torch()
    dev = dout.device
    if dout.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"dout must be bfloat16 or float32, got {dout.dtype}")
    _check(dout, "dout", dout.dtype, 2, dev)
    tokens, n = dout.shape
    topk = int(topk)
    _shaped(slot_row, "slot_row", torch.int32, (tokens * topk,), dev)
    _check(row_slot, "row_slot", torch.int32, 1, dev)
    _check(offs, "offs", torch.int32, 1, dev)
    cap, e = row_slot.shape[0], offs.shape[0]
    if weights is not None:
        _shaped(weights, "weights", torch.float32, (tokens, topk), dev)
    dw = None
    if with_weights:
        if y is None:
            raise ValueError("the gradient of the weights needs y")
        _shaped(y, "y", torch.bfloat16, (cap, n), dev)
        dw = _shaped(dweights, "dweights", torch.float32, (tokens, topk), dev)
    elif dweights is not None:
        raise ValueError("dweights without with_weights")
    out = _shaped(out, "out", torch.bfloat16, (cap, n), dev)
    _launch("gg_combine_rows_grad", dev, _ptr(dout), _dtype_code(dout.dtype), _ptr(y) if with_weights else None, n,
            _ptr(slot_row), _ptr(row_slot), _ptr(offs), e, _ptr(weights), topk, tokens, cap, _ptr(out), _ptr(dw))
    return out, dw


def _grouped(t, name, dtype, groups, masked):
    """Checks grouped rows [m, width] or [E, max_m, width]; returns (their
    leading dimensions, m or max_m, width)."""
    torch = _torch()
    _check(t, name, dtype, 3 if masked else 2, t.device)
    _check(groups, "groups", torch.int32, 1, t.device)
    if masked and t.shape[0] != groups.shape[0]:
        raise ValueError(f"{name} and groups must have the same number of experts")
    return tuple(t.shape[:-1]), t.shape[-2], t.shape[-1]


def _silu_mul_rows(h, lead, m, n, groups, masked, keep, a, a8, a8s, kept, kept_scales):
    torch = _torch()
    if keep or kept is not None or kept_scales is not None:
        if n % 256:
            raise ValueError("e4m3 rows need I = n / 2 a multiple of 128")
        kept = _shaped(kept, "kept", torch.uint8, (*lead, n), h.device)
        kept_scales = _shaped(kept_scales, "kept_scales", torch.uint8, (*lead, n // 128), h.device)
    _launch("gg_masked_silu_mul_rows" if masked else "gg_silu_mul_rows", h.device, _ptr(h), _ptr(groups), _ptr(a),
            _ptr(a8), _ptr(a8s), _ptr(kept), _ptr(kept_scales), m, n, groups.shape[0])
    return () if kept is None else (kept, kept_scales)


def silu_mul_rows(h, groups, masked=False, keep=False, out=None, kept=None, kept_scales=None):
    """a = silu(gate) * up of grouped rows h bf16 [m, 2I] (masked: [E, max_m,
    2I]; gate columns first), rows an expert owns only (gg_silu_mul_rows).
    ``keep`` (or a buffer for it) also writes h as e4m3 rows for
    ``fp8_silu_mul_grad``: returns (a, kept, kept_scales) then, else a."""
    torch = _torch()
    lead, m, n = _grouped(h, "h", torch.bfloat16, groups, masked)
    if n % 16:
        raise ValueError("h must have 2 I columns with I a multiple of 8")
    a = _shaped(out, "out", torch.bfloat16, (*lead, n // 2), h.device)
    kept = _silu_mul_rows(h, lead, m, n, groups, masked, keep, a, None, None, kept, kept_scales)
    return (a, *kept) if kept else a


def fp8_silu_mul_rows(h, groups, masked=False, keep=False, out=None, out_scales=None, kept=None, kept_scales=None):
    """silu_mul_rows with a as e4m3 rows (I a multiple of 128): returns (codes,
    scales) or (codes, scales, kept, kept_scales)."""
    torch = _torch()
    lead, m, n = _grouped(h, "h", torch.bfloat16, groups, masked)
    if n % 256:
        raise ValueError("e4m3 rows need I = n / 2 a multiple of 128")
    i = n // 2
    a8 = _shaped(out, "out", torch.uint8, (*lead, i), h.device)
    a8s = _shaped(out_scales, "out_scales", torch.uint8, (*lead, i // 128), h.device)
    return (a8, a8s, *_silu_mul_rows(h, lead, m, n, groups, masked, keep, None, a8, a8s, kept, kept_scales))


def _silu_mul_grad(da, h, h_scales, groups, masked, with_act, out, act):
    torch = _torch()
    lead, m, i = _grouped(da, "da", torch.bfloat16, groups, masked)
    dev = da.device
    _shaped(h, "h", torch.bfloat16 if h_scales is None else torch.uint8, (*lead, 2 * i), dev)
    if h_scales is not None:
        if i % 128:
            raise ValueError("e4m3 rows need I a multiple of 128")
        _shaped(h_scales, "h_scales", torch.uint8, (*lead, 2 * i // 128), dev)
    dh = _shaped(out, "out", torch.bfloat16, (*lead, 2 * i), dev)
    if with_act or act is not None:
        act = _shaped(act, "act", torch.bfloat16, (*lead, i), dev)
    _launch("gg_masked_silu_mul_grad" if masked else "gg_silu_mul_grad", dev, _ptr(da), _ptr(h), _ptr(h_scales),
            _ptr(groups), _ptr(dh), _ptr(act), m, 2 * i, groups.shape[0])
    return dh if act is None else (dh, act)


def silu_mul_grad(da, h, groups, masked=False, with_act=False, out=None, act=None):
    """Gradient of silu_mul_rows (gg_silu_mul_grad): da bf16 [m, I], h bf16
    [m, 2I] (masked: with a leading E).  Returns dh bf16 [m, 2I], or (dh, a)
    with the activation formed again (``with_act``, or a buffer for it)."""
    return _silu_mul_grad(da, h, None, groups, masked, with_act, out, act)


def fp8_silu_mul_grad(da, kept, kept_scales, groups, masked=False, with_act=False, out=None, act=None):
    """silu_mul_grad from the rows ``silu_mul_rows`` kept in 8 bits."""
    if kept_scales is None:
        raise ValueError("kept_scales is required")
    return _silu_mul_grad(da, kept, kept_scales, groups, masked, with_act, out, act)


# ---------------------------------------------------------------------------
# weight gradient from e4m3 activations
# ---------------------------------------------------------------------------

def _fp8_wgrad(name, layout, x, x_scales, dy, groups, out, out_dtype, alpha, beta):
    torch = _torch()
    _need_out(out, beta)
    masked = layout == GG_FP8_ACT_MASKED
    lead, m, k = _grouped(x, "x", torch.uint8, groups, masked)
    dev = x.device
    _check(dy, "dy", torch.bfloat16, len(lead) + 1, dev)
    if tuple(dy.shape[:-1]) != lead:
        raise ValueError("x and dy must have the same rows")
    if k % 128:
        raise ValueError("x must have a multiple of 128 columns")
    e, n = groups.shape[0], dy.shape[-1]
    _check(x_scales, "x_scales", torch.uint8, 1, dev)
    if x_scales.numel() < fp8_scale_bytes(layout, m, k, e):
        raise ValueError("packed scales are smaller than fp8_scale_bytes requires")
    out = _shaped(out, "out", (out_dtype or torch.float32) if out is None else out.dtype, (e, k, n), dev)
    _launch(name, dev, _ptr(x), _ptr(x_scales), _ptr(dy), _ptr(groups), _ptr(out), _dtype_code(out.dtype), m, k, n, e,
            float(alpha), float(beta))
    return out


def fp8_wgrad(x, x_scales, dy, offs, out=None, out_dtype=None, alpha=1.0, beta=0.0):
    """dW[g] = (x sx)[rows of g]^T . dY[rows of g] (gg_fp8_wgrad) from the
    operand pair of ``fp8_forward``: x uint8 e4m3 [m, k], x_scales packed
    (GG_FP8_ACT_RAGGED, same offs); dy bf16 [m, n].  All of ``out`` [E, k, n]
    (fp32 unless said otherwise) is written; alpha / beta as in wgrad."""
    return _fp8_wgrad("gg_fp8_wgrad", GG_FP8_ACT_RAGGED, x, x_scales, dy, offs, out, out_dtype, alpha, beta)


def fp8_masked_wgrad(x, x_scales, dy, masked_m, out=None, out_dtype=None, alpha=1.0, beta=0.0):
    """fp8_wgrad on the masked layout: x uint8 [E, max_m, k], x_scales packed
    with GG_FP8_ACT_MASKED and the same masked_m; dy bf16 [E, max_m, n]."""
    return _fp8_wgrad("gg_fp8_masked_wgrad", GG_FP8_ACT_MASKED, x, x_scales, dy, masked_m, out, out_dtype, alpha, beta)


# ---------------------------------------------------------------------------
# 4-bit rows and weights
# ---------------------------------------------------------------------------

GG_FP4_ACT_RAGGED = 0
GG_FP4_ACT_MASKED = 1
GG_FP4_WEIGHT = 2


# (sizes of sizes: asked once for each, a small call would spend 2 us of its 15 on them)
@functools.lru_cache(maxsize=1024)
def fp4_scale_bytes(layout: int, rows: int, k: int, num_groups: int) -> int:
    """Bytes of packed scales (gg_fp4_scale_bytes)."""
    v = int(load().gg_fp4_scale_bytes(int(layout), int(rows), int(k), int(num_groups)))
    if v < 0:
        raise ValueError("invalid arguments for gg_fp4_scale_bytes")
    return v


def _fp4_rows(layout, t, name, dtype, groups):
    """Checks rows in one of the layouts; returns (their leading dimensions,
    rows as the library counts them, width, experts)."""
    if layout not in (GG_FP4_ACT_RAGGED, GG_FP4_ACT_MASKED, GG_FP4_WEIGHT):
        raise ValueError(f"unknown layout {layout}")
    ragged = layout == GG_FP4_ACT_RAGGED
    _check(t, name, dtype, 2 if ragged else 3, t.device)
    if layout == GG_FP4_WEIGHT:
        if groups is not None:
            raise ValueError("weights take no groups")
        return tuple(t.shape[:2]), t.shape[1], t.shape[2], t.shape[0]
    _check(groups, "groups", _torch().int32, 1, t.device)
    if not ragged and t.shape[0] != groups.shape[0]:
        raise ValueError(f"{name} and groups must have the same number of experts")
    return tuple(t.shape[:-1]), t.shape[-2], t.shape[-1], groups.shape[0]


def _packed4(scales, name, layout, rows, k, experts, device):
    """Checks packed scales against the bytes they need, or makes them."""
    torch = _torch()
    need = fp4_scale_bytes(layout, rows, k, experts)
    if scales is None:
        return _shaped(None, name, torch.uint8, (need,), device)
    _check(scales, name, torch.uint8, 1, device)
    if scales.numel() < need:
        raise ValueError(f"{name} must hold {need} bytes")
    return scales


def fp4_pack_scales(layout: int, scales, groups=None, out=None):
    """Packed scales of one operand from E8M0 bytes (gg_fp4_pack_scales):
    scales uint8 [m, k / 32] (ragged), [E, max_m, k / 32] or [E, n, k / 32];
    groups: the int32 end offsets / masked_m (None for weights)."""
    torch = _torch()
    _, rows, blocks, e = _fp4_rows(layout, scales, "scales", torch.uint8, groups)
    out = _packed4(out, "out", layout, rows, 32 * blocks, e, scales.device)
    _launch("gg_fp4_pack_scales", scales.device, int(layout), _ptr(scales), blocks, _ptr(groups), rows, 32 * blocks, e,
            _ptr(out))
    return out


def fp4_quantize(layout: int, x, groups=None, out=None, out_scales=None):
    """4-bit rows of x (gg_fp4_quantize): bf16 [m, k], or [E, max_m, k] or
    weights [E, n, k] by ``layout``, k a multiple of 32.  Returns (codes uint8
    [..., k / 2], packed scales); rows no expert owns are left untouched."""
    torch = _torch()
    lead, rows, k, e = _fp4_rows(layout, x, "x", torch.bfloat16, groups)
    if k % 32:
        raise ValueError("x must have a multiple of 32 columns")
    out = _shaped(out, "out", torch.uint8, (*lead, k // 2), x.device)
    out_scales = _packed4(out_scales, "out_scales", layout, rows, k, e, x.device)
    _launch("gg_fp4_quantize", x.device, int(layout), _ptr(x), _ptr(groups), rows, k, e, _ptr(out), _ptr(out_scales))
    return out, out_scales


def fp4_dequantize(layout: int, codes, scales, groups=None, out=None):
    """bf16 values of 4-bit rows (gg_fp4_dequantize): codes uint8 [..., k / 2]
    and their packed scales; rows no expert owns are left untouched."""
    torch = _torch()
    lead, rows, half, e = _fp4_rows(layout, codes, "codes", torch.uint8, groups)
    if half % 16:
        raise ValueError("codes must have a multiple of 16 columns (32 values)")
    if scales is None:
        raise ValueError("scales are required")
    _packed4(scales, "scales", layout, rows, 2 * half, e, codes.device)
    out = _shaped(out, "out", torch.bfloat16, (*lead, 2 * half), codes.device)
    _launch("gg_fp4_dequantize", codes.device, int(layout), _ptr(codes), _ptr(scales), _ptr(groups), rows, 2 * half, e,
            _ptr(out))
    return out


def fp4_gather_rows(src, row_slot, topk, offs, out=None, out_scales=None):
    """Token rows sorted by expert into 4-bit rows (gg_fp4_gather_rows): src
    bf16 [tokens, k]; row_slot and offs from ``route``.  Returns (codes
    [len(row_slot), k / 2], packed scales) as ``fp4_forward`` takes them; rows
    past offs[-1] are left untouched."""
    torch = _torch()
    dev = src.device
    _check(src, "src", torch.bfloat16, 2, dev)
    tokens, k = src.shape
    if k % 32:
        raise ValueError("src must have a multiple of 32 columns")
    _check(row_slot, "row_slot", torch.int32, 1, dev)
    _check(offs, "offs", torch.int32, 1, dev)
    cap, e = row_slot.shape[0], offs.shape[0]
    out = _shaped(out, "out", torch.uint8, (cap, k // 2), dev)
    out_scales = _packed4(out_scales, "out_scales", GG_FP4_ACT_RAGGED, cap, k, e, dev)
    _launch("gg_fp4_gather_rows", dev, _ptr(src), tokens, k, _ptr(row_slot), int(topk), _ptr(offs), e, cap, _ptr(out),
            _ptr(out_scales))
    return out, out_scales


def fp4_silu_mul_rows(h, groups, masked=False, out=None, out_scales=None):
    """4-bit rows of silu(gate) * up (gg_fp4_silu_mul_rows): h bf16 [m, 2I]
    (masked: [E, max_m, 2I]; gate columns first), I a multiple of 32.  Returns
    (codes uint8 [..., I / 2], packed scales)."""
    torch = _torch()
    lead, m, n = _grouped(h, "h", torch.bfloat16, groups, masked)
    if n % 64:
        raise ValueError("h must have 2 I columns with I a multiple of 32")
    out = _shaped(out, "out", torch.uint8, (*lead, n // 4), h.device)
    out_scales = _packed4(out_scales, "out_scales", GG_FP4_ACT_MASKED if masked else GG_FP4_ACT_RAGGED, m, n // 2,
                          groups.shape[0], h.device)
    _launch("gg_fp4_masked_silu_mul_rows" if masked else "gg_fp4_silu_mul_rows", h.device, _ptr(h), _ptr(groups),
            _ptr(out), _ptr(out_scales), m, n, groups.shape[0])
    return out, out_scales


def _fp4_forward(name, layout, x, x_scales, w, w_scales, groups, out, out_dtype):
    torch = _torch()
    lead, m, half, e = _fp4_rows(layout, x, "x", torch.uint8, groups)
    dev = x.device
    _check(w, "w", torch.uint8, 3, dev)
    n = w.shape[1]
    if w.shape[0] != e or w.shape[2] != half:
        raise ValueError("shape mismatch between x, w and groups")
    if half % 16:
        raise ValueError("x must have a multiple of 16 columns (32 values)")
    if x_scales is None or w_scales is None:
        raise ValueError("x_scales and w_scales are required")
    _packed4(x_scales, "x_scales", layout, m, 2 * half, e, dev)
    _packed4(w_scales, "w_scales", GG_FP4_WEIGHT, n, 2 * half, e, dev)
    out = _shaped(out, "out", (out_dtype or torch.bfloat16) if out is None else out.dtype, (*lead, n), dev)
    _launch(name, dev, _ptr(x), _ptr(x_scales), _ptr(w), _ptr(w_scales), _ptr(groups), _ptr(out),
            _dtype_code(out.dtype), m, 2 * half, n, e)
    return out


def fp4_forward(x, x_scales, w, w_scales, offs, out=None, out_dtype=None):
    """Y[rows of g] = sum_k x sx w[g] sw (gg_fp4_forward).  x: 4-bit rows
    uint8 [m, k / 2] with packed scales (GG_FP4_ACT_RAGGED, the same offs); w:
    uint8 [E, n, k / 2] with packed scales (GG_FP4_WEIGHT)."""
    return _fp4_forward("gg_fp4_forward", GG_FP4_ACT_RAGGED, x, x_scales, w, w_scales, offs, out, out_dtype)


def fp4_masked_forward(x, x_scales, w, w_scales, masked_m, out=None, out_dtype=None):
    """The masked 4-bit forward (gg_fp4_masked_forward): x uint8 [E, max_m,
    k / 2], x_scales packed with GG_FP4_ACT_MASKED and the same masked_m."""
    return _fp4_forward("gg_fp4_masked_forward", GG_FP4_ACT_MASKED, x, x_scales, w, w_scales, masked_m, out, out_dtype)


# ---------------------------------------------------------------------------
# the expert layer for a few tokens
# ---------------------------------------------------------------------------

FEW_TOKENS_MAX = 64
FEW_SLOTS_MAX = 512


@functools.lru_cache(maxsize=1024)
def moe_few_tokens_workspace_bytes(tokens, topk, inter, num_groups) -> int:
    v = int(load().gg_moe_few_tokens_workspace_bytes(int(tokens), int(topk), int(inter), int(num_groups)))
    if v < 0:
        raise ValueError("invalid arguments for gg_moe_few_tokens_workspace_bytes")
    return v


def _few_tokens(name, x, experts, weights, w13, s13, w2, s2, wdtype, per, out, out_dtype, workspace):
    torch = _torch()
    dev = x.device
    _check(x, "x", torch.bfloat16, 2, dev)
    tokens, hidden = x.shape
    _check(experts, "experts", torch.int32, 2, dev)
    if experts.shape[0] != tokens:
        raise ValueError("experts must be [tokens, topk]")
    topk = experts.shape[1]
    if weights is not None:
        _shaped(weights, "weights", torch.float32, (tokens, topk), dev)
    _check(w13, "w13", wdtype, 3, dev)
    _check(w2, "w2", wdtype, 3, dev)
    e, rows, width = w13.shape
    inter = rows // 2
    if rows % 2 or width * per != hidden or inter % per or w2.shape != (e, hidden, inter // per):
        raise ValueError("shape mismatch between x, w13 and w2")
    ptrs = (w13.data_ptr(), w2.data_ptr())
    if per == 2:
        if hidden % 32 or inter % 32:
            raise ValueError("hidden and inter must be multiples of 32")
        if s13 is None or s2 is None:
            raise ValueError("w13_scales and w2_scales are required")
        _packed4(s13, "w13_scales", GG_FP4_WEIGHT, rows, hidden, e, dev)
        _packed4(s2, "w2_scales", GG_FP4_WEIGHT, hidden, inter, e, dev)
        ptrs = (ptrs[0], s13.data_ptr(), ptrs[1], s2.data_ptr())
    need = moe_few_tokens_workspace_bytes(tokens, topk, inter, e)
    if workspace is None:
        workspace = _shaped(None, "workspace", torch.uint8, (need,), dev)
    else:
        _check(workspace, "workspace", torch.uint8, 1, dev)
        if workspace.numel() < need:
            raise ValueError(f"workspace must hold {need} bytes")
    if out is None and (out_dtype is None or out_dtype == torch.bfloat16):
        out, code = torch.empty_like(x), GG_BF16
    else:
        out = _shaped(out, "out", out_dtype if out is None else out.dtype, (tokens, hidden), dev)
        code = _dtype_code(out.dtype)
    _launch(name, dev, x.data_ptr(), experts.data_ptr(), _ptr(weights), *ptrs, out.data_ptr(), code,
            workspace.data_ptr(), tokens, topk, hidden, inter, e)
    return out


def moe_few_tokens(x, experts, w13, w2, weights=None, out=None, out_dtype=None, workspace=None):
    """The expert layer for up to 64 tokens (gg_moe_few_tokens): x bf16
    [tokens, hidden]; experts int32 [tokens, topk] (out of range: dropped);
    w13 bf16 [E, 2I, hidden] (gate rows first), w2 bf16 [E, hidden, I];
    weights fp32 [tokens, topk] or None for 1.  Returns [tokens, hidden]."""
    torch = _torch()
    return _few_tokens("gg_moe_few_tokens", x, experts, weights, w13, None, w2, None, torch.bfloat16, 1, out, out_dtype,
                       workspace)


def fp4_moe_few_tokens(x, experts, w13, w13_scales, w2, w2_scales, weights=None, out=None, out_dtype=None,
                       workspace=None):
    """moe_few_tokens with 4-bit weights (gg_fp4_moe_few_tokens): w13 uint8
    [E, 2I, hidden / 2], w2 uint8 [E, hidden, I / 2] with their packed scales
    (GG_FP4_WEIGHT), as ``fp4_forward`` takes them."""
    torch = _torch()
    return _few_tokens("gg_fp4_moe_few_tokens", x, experts, weights, w13, w13_scales, w2, w2_scales, torch.uint8, 2, out,
                       out_dtype, workspace)
