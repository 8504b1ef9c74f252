"""ctypes binding of libqlora_nf4.so (argument marshalling only).

Every function here checks tensor shapes, dtypes and devices, passes raw device
pointers and the current HIP stream to the C ABI declared in include/qlora_nf4.h,
and raises on a non-zero return. No arithmetic on the data happens in Python.
The library must be built (``python -m bit_nf4_quantized_05_amd.build``); a
missing library is an error, never a fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora_nf4.so")

_c_i64 = ctypes.c_int64
_c_int = ctypes.c_int
_c_float = ctypes.c_float
_c_double = ctypes.c_double
_c_vp = ctypes.c_void_p

# name -> (restype, argtypes); mirrors include/qlora_nf4.h
SIGNATURES = {
    "qn_version": (_c_int, []),
    "qn_last_error": (ctypes.c_char_p, []),
    "qn_codebook": (_c_int, [_c_vp]),
    "qn_nf4_sizes": (_c_int, [_c_i64, _c_i64, _c_vp, _c_vp, _c_vp]),
    "nf4_quantize_workspace_bytes": (_c_i64, [_c_i64, _c_i64]),
    "nf4_quantize": (_c_int, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp]),
    "nf4_double_dequant": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp]),
    "qlora_linear_workspace_bytes": (_c_i64, [_c_i64, _c_i64, _c_i64, _c_int]),
    "qlora_linear_fwd_workspace_bytes": (_c_i64, [_c_i64, _c_i64, _c_i64, _c_int]),
    "qlora_linear_bwd_x_workspace_bytes": (_c_i64, [_c_i64, _c_i64, _c_i64, _c_int]),
    "qlora_linear_fwd": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_int, _c_float,
                                  _c_vp, _c_i64, _c_i64, _c_vp, _c_i64, _c_vp, _c_i64, _c_vp]),
    "qlora_linear_bwd_x": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_int, _c_float,
                                    _c_vp, _c_i64, _c_i64, _c_vp, _c_i64, _c_vp, _c_i64, _c_vp]),
    "qlora_lora_grads_workspace_bytes": (_c_i64, [_c_i64, _c_i64, _c_i64, _c_int]),
    "qlora_lora_grads": (_c_int, [_c_vp, _c_vp, _c_int, _c_float, _c_vp, _c_i64, _c_vp, _c_i64, _c_i64, _c_i64,
                                  _c_i64, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp]),
    "qn_nf4_sizes_ex": (_c_int, [_c_i64, _c_i64, _c_int, _c_vp, _c_vp, _c_vp]),
    "nf4_quantize_ex": (_c_int, [_c_vp, _c_i64, _c_i64, _c_int, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp]),
    "nf4_double_dequant_ex": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_vp, _c_vp]),
    "qlora_set_fwd_gemm": (_c_int, [_c_int]),
    "qlora_set_ax_wait": (_c_int, [_c_int]),
    "qlora_linear_fwd_ex": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_vp, _c_vp, _c_int,
                                     _c_float, _c_vp, _c_i64, _c_i64, _c_vp, _c_i64, _c_vp, _c_i64, _c_vp]),
    "qlora_linear_fwd_noalloc": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_vp, _c_vp, _c_int,
                                          _c_float, _c_vp, _c_i64, _c_i64, _c_vp, _c_i64, _c_vp]),
    "qlora_linear_bwd_x_ex": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_vp, _c_vp, _c_int,
                                       _c_float, _c_vp, _c_i64, _c_i64, _c_vp, _c_i64, _c_vp, _c_i64, _c_vp]),
    "int8_quantize": (_c_int, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp]),
    "int8_dequant": (_c_int, [_c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp]),
    "qlr_linear_workspace_bytes": (_c_i64, [_c_i64, _c_i64, _c_i64, _c_int]),
    "qlr_linear_fwd": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_int, _c_vp, _c_vp, _c_int,
                                _c_vp, _c_vp, _c_int, _c_float, _c_vp, _c_i64, _c_i64, _c_vp, _c_i64, _c_vp, _c_i64,
                                _c_vp]),
    "qlora_multi_plan_bytes": (_c_i64, [_c_i64, _c_int]),
    "qlora_multi_plan": (_c_int, [_c_vp, _c_i64, _c_int, _c_vp, _c_i64, _c_vp]),
    "qlora_multi_fwd_workspace_bytes": (_c_i64, [_c_i64, _c_i64, _c_i64, _c_int, _c_int]),
    "qlora_multi_bwd_workspace_bytes": (_c_i64, [_c_i64, _c_i64, _c_i64, _c_int, _c_int]),
    "qlora_multi_fwd": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_vp, _c_vp, _c_vp, _c_int,
                                 _c_int, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp, _c_i64, _c_vp]),
    "qlora_multi_bwd": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_vp, _c_vp, _c_vp, _c_int,
                                 _c_int, _c_vp, _c_i64, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp,
                                 _c_vp, _c_i64, _c_vp]),
    "qlora_adamw_blocks": (_c_i64, [_c_vp, _c_int]),
    "qlora_adamw_table_bytes": (_c_i64, [_c_vp, _c_int]),
    "qlora_adamw_table": (_c_i64, [_c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_int, _c_vp]),
    "qlora_adamw_step": (_c_int, [_c_vp, _c_int, _c_i64, _c_int, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_double,
                                  _c_vp, _c_double, _c_double, _c_double, _c_double, _c_vp, ctypes.c_uint32, _c_vp]),
    "qlora_adamw_moments": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_vp]),
    "qn_profile_enable": (_c_int, [_c_int]),
    "qn_profile_read": (_c_int, [_c_vp, _c_int, _c_vp, _c_vp, _c_int]),
    "qn_profile_durations": (_c_int, [ctypes.c_char_p, _c_vp, _c_int]),
}

# second-level formats: the QN_DQ_* codes of the header
DQ_CODES = {"int8": 0, "fp8": 1, "none": 2}

_lib = None


class QLoRAError(RuntimeError):
    pass


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise QLoRAError(f"{LIB_PATH} is missing: build it with `python -m bit_nf4_quantized_05_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _check(rc: int, what: str) -> None:
    if rc != 0:
        msg = lib().qn_last_error().decode(errors="replace")
        raise QLoRAError(f"{what} failed with {rc}: {msg}")


# the current stream's handle without a Stream object around it (3.4 us less per call), where
# this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev: torch.device) -> int:
    if _raw_stream is None or dev.type != "cuda" or dev.index is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return _raw_stream(dev.index)


def _ptr(t: torch.Tensor) -> int:
    return t.data_ptr()


def _rows(t: torch.Tensor, dtype, shape, name: str, device) -> int:
    """Checks a [rows, cols] activation that may be a view into a wider array: unit
    column stride, any row stride >= cols; returns the row stride (elements)."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 2 or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    rows, cols = shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the columns must be contiguous")
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{name}: row stride {ld} is smaller than the row length {cols}")
    return ld


def _need(t: torch.Tensor, dtype, shape, name: str, device) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")


@dataclass
class NF4Weight:
    """An NF4 weight with its block constants as produced by ``quantize``.

    dq names the second level: "int8" (default) or "fp8" (qconst holds E4M3 code
    bytes), both with qscale [n_g] and qmean [1]; or "none", where qscale [n_b]
    holds the float32 block absmax and qconst, qmean are empty."""
    codes: torch.Tensor    # uint8 [n_b * 32]
    qconst: torch.Tensor   # int8 [n_b] (empty for "none")
    qscale: torch.Tensor   # float32 [n_g] ([n_b] for "none")
    qmean: torch.Tensor    # float32 [1] (empty for "none")
    d_out: int
    d_in: int
    dq: str = "int8"

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.qconst, self.qscale, self.qmean))


def version() -> int:
    return lib().qn_version()


def codebook() -> list:
    buf = (ctypes.c_float * 16)()
    _check(lib().qn_codebook(ctypes.addressof(buf)), "qn_codebook")
    return list(buf)


def _dq_code(dq: str) -> int:
    if dq not in DQ_CODES:
        raise ValueError(f"dq must be one of {sorted(DQ_CODES)}, got {dq!r}")
    return DQ_CODES[dq]


def nf4_sizes(d_out: int, d_in: int, dq: str = "int8"):
    """(codes bytes, qconst entries, qscale entries) for format dq."""
    cb, nq, ns = _c_i64(), _c_i64(), _c_i64()
    _check(lib().qn_nf4_sizes_ex(d_out, d_in, _dq_code(dq), ctypes.addressof(cb), ctypes.addressof(nq),
                                 ctypes.addressof(ns)), "qn_nf4_sizes_ex")
    return cb.value, nq.value, ns.value


def quantize_workspace_bytes(d_out: int, d_in: int) -> int:
    return lib().nf4_quantize_workspace_bytes(d_out, d_in)


def linear_workspace_bytes(d_out: int, d_in: int, d_seq: int, r: int) -> int:
    """Bytes enough for both the forward and the input-gradient call."""
    return lib().qlora_linear_workspace_bytes(d_out, d_in, d_seq, r)


def linear_fwd_workspace_bytes(d_out: int, d_in: int, d_seq: int, r: int) -> int:
    return lib().qlora_linear_fwd_workspace_bytes(d_out, d_in, d_seq, r)


def linear_bwd_x_workspace_bytes(d_out: int, d_in: int, d_seq: int, r: int) -> int:
    return lib().qlora_linear_bwd_x_workspace_bytes(d_out, d_in, d_seq, r)


def alloc_weight(d_out: int, d_in: int, device, dq: str = "int8") -> NF4Weight:
    cb, nq, ns = nf4_sizes(d_out, d_in, dq)
    return NF4Weight(torch.empty(cb, dtype=torch.uint8, device=device),
                     torch.empty(nq, dtype=torch.int8, device=device),
                     torch.empty(ns, dtype=torch.float32, device=device),
                     torch.empty(0 if dq == "none" else 1, dtype=torch.float32, device=device), d_out, d_in, dq)


def quantize(W: torch.Tensor, out: NF4Weight | None = None, workspace: torch.Tensor | None = None,
             dq: str = "int8") -> NF4Weight:
    """nf4_quantize_ex on a float32 [d_out, d_in] CUDA tensor, second level dq."""
    if W.dim() != 2:
        raise ValueError("W must be 2-D [d_out, d_in]")
    d_out, d_in = W.shape
    _need(W, torch.float32, (d_out, d_in), "W", W.device)
    q = out if out is not None else alloc_weight(d_out, d_in, W.device, dq)
    if q.dq != dq:
        raise ValueError(f"out holds format {q.dq!r}, asked for {dq!r}")
    need = quantize_workspace_bytes(d_out, d_in)
    ws = workspace if workspace is not None else torch.empty(need, dtype=torch.uint8, device=W.device)
    rc = lib().nf4_quantize_ex(_ptr(W), d_out, d_in, _dq_code(dq), _ptr(q.codes), _ptr(q.qconst), _ptr(q.qscale),
                               _ptr(q.qmean), _ptr(ws), ws.numel() * ws.element_size(), _stream(W.device))
    _check(rc, "nf4_quantize_ex")
    return q


def double_dequant(q: NF4Weight, out: torch.Tensor | None = None) -> torch.Tensor:
    """nf4_double_dequant_ex -> bfloat16 [d_out, d_in]."""
    o = out if out is not None else torch.empty(q.d_out, q.d_in, dtype=torch.bfloat16, device=q.device)
    _need(o, torch.bfloat16, (q.d_out, q.d_in), "out", q.device)
    rc = lib().nf4_double_dequant_ex(_ptr(q.codes), _ptr(q.qconst), _ptr(q.qscale), _ptr(q.qmean), q.d_out, q.d_in,
                                     _dq_code(q.dq), _ptr(o), _stream(q.device))
    _check(rc, "nf4_double_dequant_ex")
    return o


def _linear(fn_name: str, q: NF4Weight, A: torch.Tensor, B: torch.Tensor, s: float, inp: torch.Tensor,
            in_dim: int, out_dim: int, out: torch.Tensor | None, workspace: torch.Tensor | None,
            ws_bytes_fn) -> torch.Tensor:
    dev = q.device
    r = A.shape[0]
    _need(A, torch.bfloat16, (r, q.d_in), "A", dev)
    _need(B, torch.bfloat16, (q.d_out, r), "B", dev)
    if inp.dim() != 2 or inp.shape[1] != in_dim:
        raise ValueError(f"input must be [d_seq, {in_dim}]")
    d_seq = inp.shape[0]
    ld_in = _rows(inp, torch.bfloat16, (d_seq, in_dim), "input", dev)
    o = out if out is not None else torch.empty(d_seq, out_dim, dtype=torch.bfloat16, device=dev)
    ld_out = _rows(o, torch.bfloat16, (d_seq, out_dim), "out", dev)
    need = ws_bytes_fn(q.d_out, q.d_in, d_seq, r)
    ws = workspace if workspace is not None else torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    rc = getattr(lib(), fn_name)(_ptr(q.codes), _ptr(q.qconst), _ptr(q.qscale), _ptr(q.qmean), q.d_out, q.d_in,
                                 _dq_code(q.dq), _ptr(A), _ptr(B), r, float(s), _ptr(inp), ld_in, d_seq, _ptr(o),
                                 ld_out, _ptr(ws), ws.numel() * ws.element_size(), _stream(dev))
    _check(rc, fn_name)
    return o


def linear_fwd(q: NF4Weight, A: torch.Tensor, B: torch.Tensor, s: float, X: torch.Tensor,
               out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """qlora_linear_fwd: Y [d_seq, d_out] = X W_hat^T + s (X A^T) B^T. X and out may be
    row views of wider arrays (unit column stride)."""
    return _linear("qlora_linear_fwd_ex", q, A, B, s, X, q.d_in, q.d_out, out, workspace,
                   linear_fwd_workspace_bytes)


# forms of the forward product for more than 64 tokens (qlora_set_fwd_gemm)
FWD_GEMM_AUTO, FWD_GEMM_STAGED, FWD_GEMM_FUSED = 0, 1, 2


def set_fwd_gemm(form: int) -> int:
    """qlora_set_fwd_gemm: process-wide choice of how the forward GEMM meets W_hat (staged in
    the workspace or formed inside the GEMM); returns the previous choice."""
    rc = lib().qlora_set_fwd_gemm(int(form))
    if rc < 0:
        raise ValueError(f"unknown forward GEMM form {form}")
    return rc


def set_ax_wait(polls: int) -> int:
    """qlora_set_ax_wait: polls a persistent one-token GEMV workgroup makes for each
    published A x slice before forming the slices itself; returns the previous value."""
    rc = lib().qlora_set_ax_wait(int(polls))
    if rc < 0:
        raise ValueError(f"polls must be >= 0, got {polls}")
    return rc


def linear_fwd_noalloc(q: NF4Weight, A: torch.Tensor, B: torch.Tensor, s: float, X: torch.Tensor,
                       out: torch.Tensor | None = None) -> torch.Tensor:
    """qlora_linear_fwd_noalloc: the forward for 1..64 tokens with no workspace (the library's
    static per-device scratch instead). Calls that overlap on one device race."""
    dev = q.device
    r = A.shape[0]
    _need(A, torch.bfloat16, (r, q.d_in), "A", dev)
    _need(B, torch.bfloat16, (q.d_out, r), "B", dev)
    if X.dim() != 2 or X.shape[1] != q.d_in:
        raise ValueError(f"input must be [d_seq, {q.d_in}]")
    d_seq = X.shape[0]
    ldx = _rows(X, torch.bfloat16, (d_seq, q.d_in), "input", dev)
    o = out if out is not None else torch.empty(d_seq, q.d_out, dtype=torch.bfloat16, device=dev)
    ldy = _rows(o, torch.bfloat16, (d_seq, q.d_out), "out", dev)
    rc = lib().qlora_linear_fwd_noalloc(_ptr(q.codes), _ptr(q.qconst), _ptr(q.qscale), _ptr(q.qmean), q.d_out,
                                        q.d_in, _dq_code(q.dq), _ptr(A), _ptr(B), r, float(s), _ptr(X), ldx, d_seq,
                                        _ptr(o), ldy, _stream(dev))
    _check(rc, "qlora_linear_fwd_noalloc")
    return o


def linear_bwd_x(q: NF4Weight, A: torch.Tensor, B: torch.Tensor, s: float, dY: torch.Tensor,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """qlora_linear_bwd_x: dX [d_seq, d_in] = dY W_hat + s (dY B) A. dY and out may be row
    views of wider arrays."""
    return _linear("qlora_linear_bwd_x_ex", q, A, B, s, dY, q.d_out, q.d_in, out, workspace,
                   linear_bwd_x_workspace_bytes)


def lora_grads_workspace_bytes(d_out: int, d_in: int, d_seq: int, r: int) -> int:
    return lib().qlora_lora_grads_workspace_bytes(d_out, d_in, d_seq, r)


def lora_grads(A: torch.Tensor, B: torch.Tensor, s: float, X: torch.Tensor, dY: torch.Tensor,
               dA: torch.Tensor | None = None, dB: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None):
    """qlora_lora_grads: (dA [r, d_in], dB [d_out, r]) float32 adapter gradients."""
    dev = A.device
    r, d_in = A.shape
    d_out = B.shape[0]
    _need(A, torch.bfloat16, (r, d_in), "A", dev)
    _need(B, torch.bfloat16, (d_out, r), "B", dev)
    if X.dim() != 2 or dY.dim() != 2 or X.shape[0] != dY.shape[0]:
        raise ValueError("X [d_seq, d_in] and dY [d_seq, d_out] must share d_seq")
    d_seq = X.shape[0]
    ldx = _rows(X, torch.bfloat16, (d_seq, d_in), "X", dev)
    lddy = _rows(dY, torch.bfloat16, (d_seq, d_out), "dY", dev)
    ga = dA if dA is not None else torch.empty(r, d_in, dtype=torch.float32, device=dev)
    gb = dB if dB is not None else torch.empty(d_out, r, dtype=torch.float32, device=dev)
    _need(ga, torch.float32, (r, d_in), "dA", dev)
    _need(gb, torch.float32, (d_out, r), "dB", dev)
    need = lora_grads_workspace_bytes(d_out, d_in, d_seq, r)
    ws = workspace if workspace is not None else torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    rc = lib().qlora_lora_grads(_ptr(A), _ptr(B), r, float(s), _ptr(X), ldx, _ptr(dY), lddy, d_out, d_in, d_seq,
                                _ptr(ga), _ptr(gb), _ptr(ws), ws.numel() * ws.element_size(), _stream(dev))
    _check(rc, "qlora_lora_grads")
    return ga, gb


def profile_enable(on: bool = True) -> None:
    """Start (clearing old records) or stop per-kernel event timing in the library."""
    _check(lib().qn_profile_enable(1 if on else 0), "qn_profile_enable")


def profile_read(cap: int = 64) -> dict:
    """{kernel name: (launches, total ms)} of the kernels timed since profile_enable."""
    name_len = 96
    names = ctypes.create_string_buffer(name_len * cap)
    launches = (ctypes.c_int64 * cap)()
    total = (ctypes.c_double * cap)()
    n = lib().qn_profile_read(ctypes.addressof(names), name_len, ctypes.addressof(launches),
                              ctypes.addressof(total), cap)
    if n < 0:
        _check(n, "qn_profile_read")
    out = {}
    for i in range(min(n, cap)):
        nm = names.raw[i * name_len:(i + 1) * name_len].split(b"\0", 1)[0].decode()
        out[nm] = (int(launches[i]), float(total[i]))
    return out


def profile_durations(name: str, cap: int = 4096) -> list:
    """Milliseconds of each launch of kernel `name` timed since profile_enable, in order."""
    buf = (ctypes.c_float * cap)()
    n = lib().qn_profile_durations(name.encode(), ctypes.addressof(buf), cap)
    if n < 0:
        _check(n, "qn_profile_durations")
    return [float(buf[i]) for i in range(min(n, cap))]


# ---- quantised low-rank factors (W ~ Q + L R with L, R at 4 or 8 bits) ----------

@dataclass
class QFactor:
    """A low-rank factor [rows, cols] kept at 4 bits (NF4 codes, float32 a_j per block
    of 64) or 8 bits (absmax INT8 per block of 64, float32 a_j)."""
    bits: int
    codes: torch.Tensor    # uint8 [n_b * 32] (4 bits) or int8 [n_b * 64] (8 bits)
    scale: torch.Tensor    # float32 [n_b]
    rows: int
    cols: int


def int8_quantize(W: torch.Tensor):
    """int8_quantize on a float32 [rows, cols] CUDA tensor -> (q int8 [n_b*64], absmax float32 [n_b])."""
    if W.dim() != 2:
        raise ValueError("W must be 2-D")
    rows, cols = W.shape
    _need(W, torch.float32, (rows, cols), "W", W.device)
    n_b = -(-rows * cols // 64)
    q = torch.empty(n_b * 64, dtype=torch.int8, device=W.device)
    a = torch.empty(n_b, dtype=torch.float32, device=W.device)
    _check(lib().int8_quantize(_ptr(W), rows, cols, _ptr(q), _ptr(a), _stream(W.device)), "int8_quantize")
    return q, a


def int8_dequant(q: torch.Tensor, absmax: torch.Tensor, rows: int, cols: int) -> torch.Tensor:
    """int8_dequant -> bfloat16 [rows, cols]."""
    n_b = -(-rows * cols // 64)
    _need(q, torch.int8, (n_b * 64,), "q", q.device)
    _need(absmax, torch.float32, (n_b,), "absmax", q.device)
    o = torch.empty(rows, cols, dtype=torch.bfloat16, device=q.device)
    _check(lib().int8_dequant(_ptr(q), _ptr(absmax), rows, cols, _ptr(o), _stream(q.device)), "int8_dequant")
    return o


def quantize_factor(M: torch.Tensor, bits: int) -> QFactor:
    """A factor at 4 bits (nf4_quantize_ex without a second level) or 8 bits (int8_quantize)."""
    rows, cols = M.shape
    if bits == 4:
        q = quantize(M, dq="none")
        return QFactor(4, q.codes, q.qscale, rows, cols)
    if bits == 8:
        c, a = int8_quantize(M)
        return QFactor(8, c, a, rows, cols)
    raise ValueError("bits must be 4 or 8")


def dequant_factor(f: QFactor) -> torch.Tensor:
    """bfloat16 [rows, cols] of a quantised factor."""
    if f.bits == 4:
        empty_q = torch.empty(0, dtype=torch.int8, device=f.codes.device)
        empty_m = torch.empty(0, dtype=torch.float32, device=f.codes.device)
        return double_dequant(NF4Weight(f.codes, empty_q, f.scale, empty_m, f.rows, f.cols, "none"))
    return int8_dequant(f.codes, f.scale, f.rows, f.cols)


def qlr_linear_workspace_bytes(d_out: int, d_in: int, d_seq: int, r: int) -> int:
    return lib().qlr_linear_workspace_bytes(d_out, d_in, d_seq, r)


def qlr_linear_fwd(q: NF4Weight, Af: QFactor, Bf: QFactor, s: float, X: torch.Tensor,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """qlr_linear_fwd: Y [d_seq, d_out] = X Q_hat^T + s (X A_hat^T) B_hat^T with A [r, d_in]
    and B [d_out, r] quantised (W ~ Q + L R with B = R^T, A = L^T)."""
    dev = q.device
    r = Af.rows
    if (Af.rows, Af.cols) != (r, q.d_in) or (Bf.rows, Bf.cols) != (q.d_out, r):
        raise ValueError("factor shapes must be A [r, d_in] and B [d_out, r]")
    if X.dim() != 2 or X.shape[1] != q.d_in:
        raise ValueError(f"input must be [d_seq, {q.d_in}]")
    d_seq = X.shape[0]
    ldx = _rows(X, torch.bfloat16, (d_seq, q.d_in), "input", dev)
    o = out if out is not None else torch.empty(d_seq, q.d_out, dtype=torch.bfloat16, device=dev)
    ldy = _rows(o, torch.bfloat16, (d_seq, q.d_out), "out", dev)
    need = qlr_linear_workspace_bytes(q.d_out, q.d_in, d_seq, r)
    ws = workspace if workspace is not None else torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    rc = lib().qlr_linear_fwd(_ptr(q.codes), _ptr(q.qconst), _ptr(q.qscale), _ptr(q.qmean), q.d_out, q.d_in,
                              _dq_code(q.dq), Af.bits, _ptr(Af.codes), _ptr(Af.scale), Bf.bits, _ptr(Bf.codes),
                              _ptr(Bf.scale), r, float(s), _ptr(X), ldx, d_seq, _ptr(o), ldy, _ptr(ws),
                              ws.numel() * ws.element_size(), _stream(dev))
    _check(rc, "qlr_linear_fwd")
    return o


# ---- many adapters on one layer ---------------------------------------------------

MULTI_RANK_STEP = 16          # ranks of a pool come in this step
MULTI_MAX_ADAPTERS = 1024


@dataclass(frozen=True)
class AdapterPool:
    """Adapters of one layer side by side: A bfloat16 [n, r, d_in], B bfloat16
    [n, d_out, r], s float32 [n] (each adapter's LoRA scale); n <= 1024, r a multiple of 16
    up to 256. Checked when it is made; the tensors' contents may change, the tensors may not be replaced.
    ``alloc_pool`` and ``set`` make one from adapters of any rank up to r."""
    A: torch.Tensor
    B: torch.Tensor
    s: torch.Tensor
    n: int = field(init=False)
    r: int = field(init=False)
    d_in: int = field(init=False)
    d_out: int = field(init=False)
    device: torch.device = field(init=False)

    def __post_init__(self):
        A, B, s = self.A, self.B, self.s
        if A.dim() != 3 or B.dim() != 3:
            raise ValueError("expected A [n, r, d_in] and B [n, d_out, r]")
        (n, r, d_in), d_out, dev = A.shape, B.shape[1], A.device
        _need(A, torch.bfloat16, (n, r, d_in), "pool.A", dev)
        _need(B, torch.bfloat16, (n, d_out, r), "pool.B", dev)
        _need(s, torch.float32, (n,), "pool.s", dev)
        if not 1 <= n <= MULTI_MAX_ADAPTERS:
            raise ValueError(f"a pool holds 1 to {MULTI_MAX_ADAPTERS} adapters, not {n}")
        if not MULTI_RANK_STEP <= r <= 256 or r % MULTI_RANK_STEP:
            raise ValueError(f"a pool's rank is a multiple of {MULTI_RANK_STEP} up to 256, not {r}")
        for name, v in (("n", n), ("r", r), ("d_in", d_in), ("d_out", d_out), ("device", dev)):
            object.__setattr__(self, name, v)

    def set(self, i: int, A: torch.Tensor, B: torch.Tensor, s: float) -> None:
        """Puts an adapter (A [k, d_in], B [d_out, k], k <= r, scale s) at place i; ranks
        past k are zeros."""
        k = A.shape[0]
        if A.shape != (k, self.d_in) or B.shape != (self.d_out, k) or not 1 <= k <= self.r:
            raise ValueError(f"expected A [k, {self.d_in}] and B [{self.d_out}, k] with k <= {self.r}")
        self.A[i].zero_()
        self.B[i].zero_()
        self.A[i, :k] = A
        self.B[i, :, :k] = B
        self.s[i] = s


def alloc_pool(n: int, r: int, d_out: int, d_in: int, device) -> AdapterPool:
    """A pool of n adapters of rank up to r (rounded up to a multiple of 16), all zero."""
    if not 1 <= n <= MULTI_MAX_ADAPTERS or not 1 <= r <= 256:
        raise ValueError(f"n must be in [1, {MULTI_MAX_ADAPTERS}] and r in [1, 256]")
    rp = -(-r // MULTI_RANK_STEP) * MULTI_RANK_STEP
    return AdapterPool(torch.zeros(n, rp, d_in, dtype=torch.bfloat16, device=device),
                       torch.zeros(n, d_out, rp, dtype=torch.bfloat16, device=device),
                       torch.zeros(n, dtype=torch.float32, device=device))


@dataclass(frozen=True)
class MultiPlan:
    """A batch's plan (``multi_plan``): good for every layer with n adapters in its pool."""
    buf: torch.Tensor
    d_seq: int
    n: int


def multi_plan(ids: torch.Tensor, n: int, out: MultiPlan | None = None) -> MultiPlan:
    """qlora_multi_plan: the plan of a batch whose token t has adapter ids[t] (int32
    [d_seq]; a value outside [0, n): none). out: a plan of the same sizes to write again."""
    if ids.dim() != 1:
        raise ValueError("ids must be 1-D [d_seq]")
    d_seq = ids.shape[0]
    _need(ids, torch.int32, (d_seq,), "ids", ids.device)
    need = lib().qlora_multi_plan_bytes(d_seq, n)
    if out is None:
        out = MultiPlan(torch.empty(max(need, 1), dtype=torch.uint8, device=ids.device), d_seq, n)
    elif (out.d_seq, out.n) != (d_seq, n) or out.buf.device != ids.device:
        raise ValueError(f"out is a plan for {out.d_seq} tokens and {out.n} adapters")
    _check(lib().qlora_multi_plan(_ptr(ids), d_seq, n, _ptr(out.buf), out.buf.numel(), _stream(ids.device)),
           "qlora_multi_plan")
    return out


def multi_linear_fwd_workspace_bytes(d_out: int, d_in: int, d_seq: int, r: int, n: int) -> int:
    return lib().qlora_multi_fwd_workspace_bytes(d_out, d_in, d_seq, r, n)


def multi_linear_bwd_workspace_bytes(d_out: int, d_in: int, d_seq: int, r: int, n: int) -> int:
    return lib().qlora_multi_bwd_workspace_bytes(d_out, d_in, d_seq, r, n)


def _multi_check(q: NF4Weight, pool: AdapterPool, plan: MultiPlan, d_seq: int, dev) -> None:
    if pool.d_in != q.d_in or pool.d_out != q.d_out or pool.device != dev:
        raise ValueError(f"the pool is for a {pool.d_out} x {pool.d_in} layer on {pool.device}, "
                         f"not {q.d_out} x {q.d_in} on {dev}")
    if plan.d_seq != d_seq or plan.n != pool.n or plan.buf.device != dev:
        raise ValueError(f"the plan is for {plan.d_seq} tokens and {plan.n} adapters on {plan.buf.device}, "
                         f"not {d_seq} and {pool.n} on {dev}")


def _multi_workspace(workspace: torch.Tensor | None, need, d_out, d_in, d_seq, pool: AdapterPool, dev) -> torch.Tensor:
    if workspace is None:
        return torch.empty(max(need(d_out, d_in, d_seq, pool.r, pool.n), 1), dtype=torch.uint8, device=dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected contiguous memory on {dev}")
    return workspace


def _multi_output(t: torch.Tensor, shape, name: str, dev, *inputs: torch.Tensor) -> int:
    """Row stride of an output that is none of the inputs (they are read while it is written)."""
    ld = _rows(t, torch.bfloat16, shape, name, dev)
    if any(t.data_ptr() == x.data_ptr() for x in inputs):
        raise ValueError(f"{name} is an input of the call")
    return ld


def multi_linear_fwd(q: NF4Weight, pool: AdapterPool, plan: MultiPlan, X: torch.Tensor,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """qlora_multi_fwd: Y[t] = W_hat x_t + s_a B_a (A_a x_t), a the adapter of token t in the
    plan. X [d_seq, d_in] and out [d_seq, d_out] may be row views of wider arrays."""
    dev = q.codes.device
    d_out, d_in = q.d_out, q.d_in
    if X.dim() != 2 or X.shape[1] != d_in:
        raise ValueError(f"input must be [d_seq, {d_in}]")
    d_seq = X.shape[0]
    _multi_check(q, pool, plan, d_seq, dev)
    ldx = _rows(X, torch.bfloat16, X.shape, "input", dev)
    if out is None:
        o, ldy = X.new_empty((d_seq, d_out)), d_out
    else:
        o, ldy = out, _multi_output(out, (d_seq, d_out), "out", dev, X)
    ws = _multi_workspace(workspace, multi_linear_fwd_workspace_bytes, d_out, d_in, d_seq, pool, dev)
    rc = lib().qlora_multi_fwd(q.codes.data_ptr(), q.qconst.data_ptr(), q.qscale.data_ptr(), q.qmean.data_ptr(), d_out,
                               d_in, _dq_code(q.dq), pool.A.data_ptr(), pool.B.data_ptr(), pool.s.data_ptr(), pool.n,
                               pool.r, X.data_ptr(), ldx, d_seq, plan.buf.data_ptr(), o.data_ptr(), ldy, ws.data_ptr(),
                               ws.nbytes, _stream(dev))
    if rc:
        _check(rc, "qlora_multi_fwd")
    return o


def multi_linear_bwd(q: NF4Weight, pool: AdapterPool, plan: MultiPlan, X: torch.Tensor, dY: torch.Tensor,
                     dX: torch.Tensor | None = None, dA: torch.Tensor | None = None, dB: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None):
    """qlora_multi_bwd: (dX bfloat16 [d_seq, d_in], dA float32 [n, r, d_in], dB float32
    [n, d_out, r]) of ``multi_linear_fwd`` for the loss gradient dY."""
    dev = q.codes.device
    d_out, d_in, n, r = q.d_out, q.d_in, pool.n, pool.r
    if X.dim() != 2 or dY.dim() != 2 or X.shape[0] != dY.shape[0]:
        raise ValueError("X [d_seq, d_in] and dY [d_seq, d_out] must share d_seq")
    d_seq = X.shape[0]
    _multi_check(q, pool, plan, d_seq, dev)
    ldx = _rows(X, torch.bfloat16, (d_seq, d_in), "X", dev)
    lddy = _rows(dY, torch.bfloat16, (d_seq, d_out), "dY", dev)
    if dX is None:
        gx, lddx = X.new_empty((d_seq, d_in)), d_in
    else:
        gx, lddx = dX, _multi_output(dX, (d_seq, d_in), "dX", dev, X, dY)
    ga = dA if dA is not None else torch.empty(n, r, d_in, dtype=torch.float32, device=dev)
    gb = dB if dB is not None else torch.empty(n, d_out, r, dtype=torch.float32, device=dev)
    if dA is not None:
        _need(ga, torch.float32, (n, r, d_in), "dA", dev)
    if dB is not None:
        _need(gb, torch.float32, (n, d_out, r), "dB", dev)
    ws = _multi_workspace(workspace, multi_linear_bwd_workspace_bytes, d_out, d_in, d_seq, pool, dev)
    rc = lib().qlora_multi_bwd(q.codes.data_ptr(), q.qconst.data_ptr(), q.qscale.data_ptr(), q.qmean.data_ptr(), d_out,
                               d_in, _dq_code(q.dq), pool.A.data_ptr(), pool.B.data_ptr(), pool.s.data_ptr(), n, r,
                               X.data_ptr(), ldx, dY.data_ptr(), lddy, d_seq, plan.buf.data_ptr(), gx.data_ptr(), lddx,
                               ga.data_ptr(), gb.data_ptr(), ws.data_ptr(), ws.nbytes, _stream(dev))
    if rc:
        _check(rc, "qlora_multi_bwd")
    return gx, ga, gb


# ---- AdamW over many tensors -----------------------------------------------------

ADAMW_BLOCK = 256     # elements per state block
_STATES_8, _GRAD_BF16, _PARAM_BF16 = 1, 2, 4


@dataclass
class AdamWState:
    """The tensors of an AdamW step, their moments and the device table that lists them,
    as made by ``adamw_state``. Tensor i's moments are the elements [offsets[i],
    offsets[i] + numel) of m and v (values with bits 32, codes with bits 8: ``adamw_moments``
    gives their values). The tensors are kept, not copied; ``set_grads`` names other
    gradient tensors."""
    params: list
    grads: list
    copies: list | None
    bits: int
    m: torch.Tensor                 # float32 or uint8 [256 * blocks]
    v: torch.Tensor
    m_scale: torch.Tensor | None    # float32 [blocks] (bits 8)
    v_scale: torch.Tensor | None
    offsets: list
    blocks: int
    flags: int
    table: torch.Tensor             # uint8, device
    n_chunks: int

    @property
    def device(self) -> torch.device:
        return self.m.device

    def set_grads(self, grads) -> None:
        """Uses these gradients (same shapes and type) from the next step on the current stream
        on, captured steps included; the table is filled again in place (a copy from the host,
        so keep gradient buffers where possible)."""
        grads = list(grads)
        if _adamw_flags(self.params, grads, self.copies, self.bits) != self.flags:
            raise TypeError("the gradients' type must stay the same")
        host, self.n_chunks = _adamw_table(self.params, grads, self.copies, self.flags)
        self.table.copy_(host)
        self.grads = grads


def _adamw_flags(params, grads, copies, bits) -> int:
    if bits not in (8, 32):
        raise ValueError("bits must be 8 or 32")
    if not params:
        raise ValueError("no tensors")
    if len(grads) != len(params) or (copies is not None and len(copies) != len(params)):
        raise ValueError("params, grads and copies must have the same length")
    dev, pt, gt = params[0].device, params[0].dtype, grads[0].dtype
    for t, name in ((pt, "params"), (gt, "grads")):
        if t not in (torch.float32, torch.bfloat16):
            raise TypeError(f"{name}: expected float32 or bfloat16, got {t}")
    for i, p in enumerate(params):
        _need(p, pt, p.shape, f"params[{i}]", dev)
        _need(grads[i], gt, p.shape, f"grads[{i}]", dev)
        if copies is not None and copies[i] is not None:
            _need(copies[i], torch.bfloat16, p.shape, f"copies[{i}]", dev)
    return ((_STATES_8 if bits == 8 else 0) | (_GRAD_BF16 if gt == torch.bfloat16 else 0) |
            (_PARAM_BF16 if pt == torch.bfloat16 else 0))


def _adamw_own_memory(params, copies) -> None:
    """Every written element belongs to one tensor (a bfloat16 parameter may be its own copy)."""
    spans = [(p.data_ptr(), p.data_ptr() + p.nbytes, f"params[{i}]") for i, p in enumerate(params)]
    spans += [(c.data_ptr(), c.data_ptr() + c.nbytes, f"copies[{i}]") for i, c in enumerate(copies or [])
              if c is not None and (c.data_ptr(), c.dtype) != (params[i].data_ptr(), params[i].dtype)]
    spans = sorted(s for s in spans if s[1] > s[0])
    for (_, end, a), (start, _, b) in zip(spans, spans[1:]):
        if start < end:
            raise ValueError(f"{a} and {b} share memory: one step would update it twice")


def _adamw_table(params, grads, copies, flags):
    """(the table in host memory, its chunks)."""
    k = len(params)
    n = (_c_i64 * k)(*[p.numel() for p in params])
    ptrs = [(ctypes.c_void_p * k)(*[t.data_ptr() if t is not None and t.numel() else None for t in ts])
            for ts in (params, grads, copies if copies is not None else [None] * k)]
    need = lib().qlora_adamw_table_bytes(ctypes.addressof(n), k)
    if need < 0:
        _check(int(need), "qlora_adamw_table_bytes")
    host = torch.empty(need, dtype=torch.uint8)
    chunks = lib().qlora_adamw_table(*[ctypes.addressof(p) for p in ptrs], ctypes.addressof(n), k, flags, _ptr(host))
    if chunks < 0:
        _check(int(chunks), "qlora_adamw_table")
    return host, int(chunks)


def adamw_state(params, grads, copies=None, bits: int = 32) -> AdamWState:
    """State of an AdamW step over these tensors (float32 or bfloat16, contiguous; the
    gradients of the same shapes, float32 or bfloat16), moments of 32 or 8 bits, all zero.
    copies: bfloat16 tensors (or None entries) that receive the new parameters."""
    params, grads = list(params), list(grads)
    copies = list(copies) if copies is not None else None
    flags = _adamw_flags(params, grads, copies, bits)
    _adamw_own_memory(params, copies)
    dev = params[0].device
    offsets, blocks = [], 0
    for p in params:
        offsets.append(blocks * ADAMW_BLOCK)
        blocks += -(-p.numel() // ADAMW_BLOCK)
    dt = torch.uint8 if bits == 8 else torch.float32
    m = torch.zeros(blocks * ADAMW_BLOCK, dtype=dt, device=dev)
    scales = [torch.zeros(blocks, dtype=torch.float32, device=dev) for _ in range(2)] if bits == 8 else [None, None]
    table, n_chunks = _adamw_table(params, grads, copies, flags)
    return AdamWState(params, grads, copies, bits, m, torch.zeros_like(m), *scales, offsets, blocks, flags,
                      table.to(dev), n_chunks)


def _scalar(t: torch.Tensor, dtype, name: str, device) -> int:
    if t.dtype != dtype or t.numel() != 1 or t.device != device:
        raise ValueError(f"{name}: expected one {dtype} on {device}")
    return t.data_ptr()


def adamw_step(state: AdamWState, step, lr, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               weight_decay: float = 0.01, grad_scale: torch.Tensor | None = None, seed: int = 0) -> None:
    """qlora_adamw_step: one AdamW step in place over all tensors of the state. step (1 for
    the first) and lr may be one-element device tensors (int64, float32), read when the step
    runs, for calls captured in a graph (a device step below 1 changes nothing); grad_scale is a one-element float32 device tensor
    that multiplies the gradients."""
    dev = state.device
    step_dev = _scalar(step, torch.int64, "step", dev) if isinstance(step, torch.Tensor) else None
    lr_dev = _scalar(lr, torch.float32, "lr", dev) if isinstance(lr, torch.Tensor) else None
    gs = _scalar(grad_scale, torch.float32, "grad_scale", dev) if grad_scale is not None else None
    s8 = state.bits == 8
    rc = lib().qlora_adamw_step(_ptr(state.table), len(state.params), state.n_chunks, state.flags, _ptr(state.m),
                                _ptr(state.v), _ptr(state.m_scale) if s8 else None,
                                _ptr(state.v_scale) if s8 else None, 0 if step_dev else step, step_dev,
                                0.0 if lr_dev else lr, lr_dev, beta1, beta2, eps, weight_decay, gs,
                                seed & 0xFFFFFFFF, _stream(dev))
    _check(rc, "qlora_adamw_step")


def adamw_moments(state: AdamWState, m: torch.Tensor | None = None, v: torch.Tensor | None = None):
    """(m, v) as float32 [256 * blocks]: the state's own tensors with bits 32, the values of
    the codes with bits 8 (into m and v if given)."""
    if state.bits == 32:
        return state.m, state.v
    n = state.blocks * ADAMW_BLOCK
    mo = m if m is not None else torch.empty(n, dtype=torch.float32, device=state.device)
    vo = v if v is not None else torch.empty(n, dtype=torch.float32, device=state.device)
    _need(mo, torch.float32, (n,), "m", state.device)
    _need(vo, torch.float32, (n,), "v", state.device)
    _check(lib().qlora_adamw_moments(_ptr(state.m), _ptr(state.m_scale), _ptr(state.v), _ptr(state.v_scale),
                                     state.blocks, _ptr(mo), _ptr(vo), _stream(state.device)), "qlora_adamw_moments")
    return mo, vo
