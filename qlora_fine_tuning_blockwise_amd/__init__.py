"""QLoRA frozen-base hot path for MI355X (gfx950): blockwise NF4 quantization
with double quantization, dequantization to bf16, and the QLoRA linear layer
(forward and backward), as hand-written HIP kernels behind a C ABI.

The functions below carry the names of the C entry points
(include/qlora_amd.h). They only marshal arguments: torch supplies device
memory and the current stream, and every step of the computation runs in
libqlora_amd.so. Tensors must be contiguous and on a ROCm device.

The row operators (qlora_embed_*, qlora_norm_*, qlora_distill_*,
qlora_add_norm_*, qlora_head_loss_*) take matrices whose rows are contiguous, at
any row stride (views of wider or longer tensors), and run on the device of
their tensors whichever is current.
Without `stream` they use that device's current stream; with it, what they
allocate belongs to that stream. A given output may not share memory with an
input or another output (the library refuses the call); only qlora_norm_fwd's
y may be x itself, and qlora_add_norm_fwd's h x or the residual. The clipping of
the gradients (qlora_grad_norm, qlora_grad_scale) takes contiguous tensors, one
by one or as a list that the program keeps (qlora_tensor_list).
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _lib

__all__ = [
    "qlora_strerror", "qlora_nf4_sizes", "qlora_codebook", "qlora_codebook_quotient_thresholds",
    "qlora_codebook_id", "qlora_setup_id", "qlora_nf4_check",
    "qlora_workspace_bytes", "qlora_quantize_nf4_dq", "qlora_dequant_bf16",
    "qlora_linear_fwd", "qlora_linear_bwd", "qlora_linear_fwd_noalloc", "qlora_gemm_bf16_nt", "qlora_merge_lora", "qlora_adamw_step",
    "qlora_embed_fwd", "qlora_embed_bwd", "qlora_embed_bwd_workspace_bytes",
    "qlora_norm_fwd", "qlora_norm_bwd", "qlora_norm_bwd_workspace_bytes",
    "qlora_distill_fwd", "qlora_distill_bwd", "qlora_distill_fwd_workspace_bytes",
    "qlora_add_norm_fwd", "qlora_add_norm_bwd",
    "qlora_head_loss_fwd", "qlora_head_loss_bwd", "qlora_head_loss_fwd_workspace_bytes",
    "qlora_head_loss_bwd_workspace_bytes",
    "qlora_tensor_list", "qlora_grad_norm", "qlora_grad_norm_workspace_bytes", "qlora_grad_scale",
    "TensorList", "NORM_LAYER", "NORM_RMS",
    "NF4Weight", "DQ_INT8", "DQ_UINT8", "DQ_E4M3", "LAYOUT_ROWS", "LAYOUT_KSLAB32",
]


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _need(t, name, shape, dtypes, device):
    """Checks one tensor argument before its pointer crosses the C ABI (the
    library cannot see buffer sizes): shape, dtype, contiguity and device."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not isinstance(dtypes, tuple):
        dtypes = (dtypes,)
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(dt) -> int:
    if dt == torch.float32:
        return _lib.DTYPE_F32
    if dt == torch.bfloat16:
        return _lib.DTYPE_BF16
    raise ValueError(f"unsupported dtype {dt}")


DQ_INT8, DQ_UINT8, DQ_E4M3 = _lib.DQ_INT8, _lib.DQ_UINT8, _lib.DQ_E4M3
LAYOUT_ROWS, LAYOUT_KSLAB32 = _lib.LAYOUT_ROWS, _lib.LAYOUT_KSLAB32
NORM_LAYER, NORM_RMS = _lib.NORM_LAYER, _lib.NORM_RMS


class NF4Weight:
    """A quantized [N, K] weight: its three device buffers and the metadata of
    the C descriptor (struct qlora_nf4): the second-level format of the
    absmax codes (DQ_INT8, DQ_UINT8, DQ_E4M3), the storage format version and
    the setup id of the library that quantized it. qlora_quantize_nf4_dq
    fills the metadata; a weight restored from storage carries the stored
    values, and the library rejects it if they do not match its own."""

    def __init__(self, codes, absmax_q, absmax_scale, N: int, K: int, dq_format: int = DQ_INT8,
                 format_version: int = 0, setup_id: int = 0):
        self.codes, self.absmax_q, self.absmax_scale = codes, absmax_q, absmax_scale
        self.N, self.K = int(N), int(K)
        self.dq_format = int(dq_format)
        self.format_version = int(format_version)
        self.setup_id = int(setup_id)

    def nbytes(self) -> int:
        return self.codes.numel() + self.absmax_q.numel() + 4 * self.absmax_scale.numel()

    @property
    def device(self):
        return self.codes.device

    def _check_buffers(self):
        cb, qb, sb = qlora_nf4_sizes(self.N, self.K)
        dev = self.codes.device
        _need(self.codes, "codes", (cb,), torch.uint8, dev)
        _need(self.absmax_q, "absmax_q", (qb,), torch.int8, dev)
        _need(self.absmax_scale, "absmax_scale", (sb // 4,), torch.float32, dev)

    def desc(self) -> "ctypes.pointer":
        """The C descriptor of this weight (buffers checked first)."""
        self._check_buffers()
        d = _lib.NF4Desc(self.N, self.K, self.codes.data_ptr(), self.absmax_q.data_ptr(),
                         self.absmax_scale.data_ptr(), self.dq_format, self.format_version,
                         self.setup_id, 0)
        return ctypes.pointer(d)


def qlora_strerror(status: int) -> str:
    return _lib.strerror(status)


def qlora_nf4_sizes(N: int, K: int):
    cb, qb, sb = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _lib.check(_lib.load().qlora_nf4_sizes(N, K, ctypes.byref(cb), ctypes.byref(qb),
                                           ctypes.byref(sb)), "qlora_nf4_sizes")
    return cb.value, qb.value, sb.value


def qlora_codebook():
    lv = np.zeros(16, np.float32)
    th = np.zeros(15, np.float32)
    _lib.check(_lib.load().qlora_codebook(lv.ctypes.data_as(ctypes.c_void_p),
                                          th.ctypes.data_as(ctypes.c_void_p)), "qlora_codebook")
    return lv, th


def qlora_codebook_quotient_thresholds():
    tq = np.zeros(15, np.float32)
    _lib.check(_lib.load().qlora_codebook_quotient_thresholds(tq.ctypes.data_as(ctypes.c_void_p)),
               "qlora_codebook_quotient_thresholds")
    return tq


def qlora_nf4_check(w: NF4Weight) -> int:
    """Status of the library's host check of w's descriptor (0 = usable)."""
    return int(_lib.load().qlora_nf4_check(w.desc()))


def qlora_setup_id(dq_format: int) -> int:
    return int(_lib.load().qlora_setup_id(int(dq_format)))


def qlora_codebook_id() -> int:
    return int(_lib.load().qlora_codebook_id())


def qlora_workspace_bytes(op: int, M: int, N: int, K: int, r: int) -> int:
    return int(_lib.load().qlora_workspace_bytes(op, M, N, K, r))


def _alloc_nf4(N, K, device):
    cb, qb, sb = qlora_nf4_sizes(N, K)
    return (torch.empty(cb, dtype=torch.uint8, device=device),
            torch.empty(qb, dtype=torch.int8, device=device),
            torch.empty(sb // 4, dtype=torch.float32, device=device))


def qlora_quantize_nf4_dq(W: torch.Tensor, out: NF4Weight | None = None, stream=None,
                          dq_format: int | None = None) -> NF4Weight:
    """Quantize a [N, K] fp32 or bf16 device tensor to NF4 + double-quantized
    constants in second-level format dq_format (default: out's format, else
    DQ_INT8). The returned weight carries the descriptor metadata the library
    wrote."""
    if W.dim() != 2:
        raise ValueError("qlora_quantize_nf4_dq: W must be [N, K]")
    N, K = W.shape
    _need(W, "W", (N, K), (torch.float32, torch.bfloat16), W.device)
    if dq_format is None:
        dq_format = out.dq_format if out is not None else DQ_INT8
    if out is None:
        out = NF4Weight(*_alloc_nf4(N, K, W.device), N, K, dq_format)
    if (out.N, out.K) != (N, K):
        raise ValueError("qlora_quantize_nf4_dq: out has another shape")
    out.dq_format = int(dq_format)
    d = out.desc()
    st = _lib.load().qlora_quantize_nf4_dq(_ptr(W), _dtype_code(W.dtype), N, K, out.dq_format, d,
                                           _stream(stream))
    _lib.check(st, "qlora_quantize_nf4_dq")
    out.format_version, out.setup_id = int(d.contents.format_version), int(d.contents.setup_id)
    return out


def qlora_dequant_bf16(w: NF4Weight, out: torch.Tensor | None = None, stream=None,
                       layout: int = LAYOUT_ROWS) -> torch.Tensor:
    """w_hat as bf16: [N, K] (LAYOUT_ROWS) or [K/32, N, 32] (LAYOUT_KSLAB32)."""
    shape = (w.N, w.K) if layout == LAYOUT_ROWS else (w.K // 32, w.N, 32)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=w.device)
    if out.numel() != w.N * w.K:
        raise ValueError("qlora_dequant_bf16: out must hold N*K elements")
    _need(out, "out", tuple(out.shape), torch.bfloat16, w.device)
    st = _lib.load().qlora_dequant_bf16(w.desc(), _ptr(out), int(layout), _stream(stream))
    _lib.check(st, "qlora_dequant_bf16")
    return out


def _workspace(op, M, N, K, r, device, workspace):
    need = qlora_workspace_bytes(op, M, N, K, r)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    if workspace.dtype != torch.uint8 or workspace.dim() != 1 or not workspace.is_contiguous() \
            or workspace.device != device:
        raise ValueError("workspace: a contiguous 1-D uint8 tensor on the weight's device")
    return workspace


def qlora_linear_fwd(w: NF4Weight, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                     alpha: float, y: torch.Tensor | None = None, y_dtype=torch.float32,
                     u_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None, lean: bool = False) -> torch.Tensor:
    """y = x W_hat^T + (alpha/r) (x A) B. x [M,K] bf16, A [K,r] bf16, B [r,N] bf16.
    The route follows the workspace size (an allocated one is sized for the
    fast route, or for the lean route that holds no bf16 copy of the weight
    when `lean`)."""
    M = x.shape[0]
    r = A.shape[1]
    dev = w.device
    _need(x, "x", (M, w.K), torch.bfloat16, dev)
    _need(A, "A", (w.K, r), torch.bfloat16, dev)
    _need(B, "B", (r, w.N), torch.bfloat16, dev)
    if y is None:
        y = torch.empty((M, w.N), dtype=y_dtype, device=dev)
    _need(y, "y", (M, w.N), (torch.float32, torch.bfloat16), dev)
    _need(u_out, "u_out", (M, r), torch.float32, dev)
    workspace = _workspace(_lib.OP_FWD_LEAN if lean else _lib.OP_FWD, M, w.N, w.K, r, dev,
                           workspace)
    st = _lib.load().qlora_linear_fwd(
        w.desc(), _ptr(x), M, _ptr(A), _ptr(B), r, float(alpha), _ptr(y), _dtype_code(y.dtype),
        _ptr(u_out), _ptr(workspace), workspace.numel(), _stream(stream))
    _lib.check(st, "qlora_linear_fwd")
    return y


def qlora_linear_fwd_noalloc(w: NF4Weight, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                             alpha: float, y: torch.Tensor, u_out: torch.Tensor | None = None,
                             stream=None) -> torch.Tensor:
    """qlora_linear_fwd with the library's own device array as the workspace:
    the call allocates nothing (y and u_out are the caller's)."""
    M = x.shape[0]
    r = A.shape[1]
    dev = w.device
    _need(x, "x", (M, w.K), torch.bfloat16, dev)
    _need(A, "A", (w.K, r), torch.bfloat16, dev)
    _need(B, "B", (r, w.N), torch.bfloat16, dev)
    _need(y, "y", (M, w.N), (torch.float32, torch.bfloat16), dev)
    _need(u_out, "u_out", (M, r), torch.float32, dev)
    st = _lib.load().qlora_linear_fwd_noalloc(
        w.desc(), _ptr(x), M, _ptr(A), _ptr(B), r, float(alpha), _ptr(y), _dtype_code(y.dtype),
        _ptr(u_out), _stream(stream))
    _lib.check(st, "qlora_linear_fwd_noalloc")
    return y


def qlora_linear_bwd(w: NF4Weight, x: torch.Tensor | None, dY: torch.Tensor, A: torch.Tensor,
                     B: torch.Tensor, alpha: float, u_saved: torch.Tensor | None = None,
                     want_dx: bool = True, dx_dtype=torch.float32, grad_dtype=torch.float32,
                     want_grads: bool = True, workspace: torch.Tensor | None = None,
                     stream=None, lean: bool = False):
    """Returns (dX or None, dA or None, dB or None). With lean=True (and no
    workspace given) the call gets the smallest workspace it accepts, so from
    512 rows on dX is computed without a bf16 copy of the weight."""
    M = dY.shape[0]
    r = A.shape[1]
    dev = w.device
    _need(dY, "dY", (M, w.N), torch.bfloat16, dev)
    _need(x, "x", (M, w.K), torch.bfloat16, dev)
    _need(A, "A", (w.K, r), torch.bfloat16, dev)
    _need(B, "B", (r, w.N), torch.bfloat16, dev)
    _need(u_saved, "u_saved", (M, r), torch.float32, dev)
    dX = torch.empty((M, w.K), dtype=dx_dtype, device=dev) if want_dx else None
    dA = torch.empty((w.K, r), dtype=grad_dtype, device=dev) if want_grads else None
    dB = torch.empty((r, w.N), dtype=grad_dtype, device=dev) if want_grads else None
    workspace = _workspace(_lib.OP_BWD_LEAN if lean else _lib.OP_BWD, M, w.N, w.K, r, dev,
                           workspace)
    st = _lib.load().qlora_linear_bwd(
        w.desc(), _ptr(x), _ptr(dY), M, _ptr(A), _ptr(B), r, float(alpha), _ptr(u_saved),
        _ptr(dX), _dtype_code(dx_dtype), _ptr(dA), _ptr(dB), _dtype_code(grad_dtype),
        _ptr(workspace), workspace.numel(), _stream(stream))
    _lib.check(st, "qlora_linear_bwd")
    return dX, dA, dB


def qlora_gemm_bf16_nt(a: torch.Tensor, b: torch.Tensor, e: torch.Tensor, f: torch.Tensor,
                       y: torch.Tensor | None = None, y_dtype=torch.float32,
                       stream=None, b_layout: int = LAYOUT_ROWS) -> torch.Tensor:
    """y = a b^T + e [f|f]^T. a [M,K], b [N,K] (LAYOUT_ROWS) or [K/32,N,32]
    (LAYOUT_KSLAB32), e [M,2r], f [N,r], all bf16."""
    M, K = a.shape
    if b_layout == LAYOUT_ROWS:
        N = b.shape[0]
        b_ok = b.shape == (N, K)
    else:
        N = b.shape[1]
        b_ok = b.shape == (K // 32, N, 32)
    r = f.shape[1]
    if not b_ok or e.shape != (M, 2 * r) or f.shape[0] != N:
        raise ValueError("qlora_gemm_bf16_nt: inconsistent shapes")
    if y is None:
        y = torch.empty((M, N), dtype=y_dtype, device=a.device)
    st = _lib.load().qlora_gemm_bf16_nt(_ptr(a), K, _ptr(b), K, int(b_layout), _ptr(e), _ptr(f), M,
                                        N, K, r, _ptr(y), _dtype_code(y.dtype), _stream(stream))
    _lib.check(st, "qlora_gemm_bf16_nt")
    return y


def qlora_merge_lora(A: torch.Tensor, B: torch.Tensor, alpha: float, w: NF4Weight | None = None,
                     W: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """merged = base + (alpha/r) (A B)^T as fp32 [N, K]; base = the dequantized
    NF4 weight w, or the bf16 weight W. Requantize with qlora_quantize_nf4_dq."""
    if (w is None) == (W is None):
        raise ValueError("qlora_merge_lora: give exactly one of w (NF4) and W (bf16)")
    N, K = (w.N, w.K) if w is not None else W.shape
    r = A.shape[1]
    dev = A.device
    if out is None:
        out = torch.empty((N, K), dtype=torch.float32, device=dev)
    need = qlora_workspace_bytes(_lib.OP_MERGE, 0, N, K, r)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _need(W, "W", (N, K), torch.bfloat16, dev)
    _need(A, "A", (K, r), torch.bfloat16, dev)
    _need(B, "B", (r, N), torch.bfloat16, dev)
    _need(out, "out", (N, K), torch.float32, dev)
    st = _lib.load().qlora_merge_lora(w.desc() if w is not None else None, _ptr(W), N, K,
                                      _ptr(A), _ptr(B), r, float(alpha), _ptr(out),
                                      _ptr(workspace), workspace.numel(), _stream(stream))
    _lib.check(st, "qlora_merge_lora")
    return out


def _one_factor(t, name):
    if t.numel() != 1 or t.dtype != torch.float32 or t.device.type != "cuda":
        raise ValueError(f"{name}: one fp32 value on the device")


def qlora_adamw_step(param: torch.Tensor, grad: torch.Tensor, exp_avg: torch.Tensor,
                     exp_avg_sq: torch.Tensor, step: int, lr: float, beta1: float = 0.9,
                     beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
                     param_bf16: torch.Tensor | None = None, stream=None,
                     grad_factor: torch.Tensor | None = None) -> None:
    """One AdamW step in place on flat fp32 master values, moments and an
    optional bf16 copy; grad is bf16 or fp32. The arrays may be device tensors
    or pinned host tensors (the paged state); the step runs on the GPU.
    grad_factor: one fp32 value on the device that the gradient is multiplied
    by, such as the second of qlora_grad_norm's result."""
    n = param.numel()
    for name, t, dt in (("param", param, torch.float32), ("exp_avg", exp_avg, torch.float32),
                        ("exp_avg_sq", exp_avg_sq, torch.float32),
                        ("param_bf16", param_bf16, torch.bfloat16)):
        if t is not None and (t.dtype != dt or t.numel() != n):
            raise ValueError(f"qlora_adamw_step: {name} must be {dt} with {n} elements")
    if grad.numel() != n:
        raise ValueError("qlora_adamw_step: grad must have as many elements as param")
    if grad_factor is not None:
        _one_factor(grad_factor, "grad_factor")
        st = _lib.load().qlora_adamw_step_scaled(
            _ptr(param), _ptr(grad), _dtype_code(grad.dtype), _ptr(grad_factor), _ptr(exp_avg),
            _ptr(exp_avg_sq), _ptr(param_bf16), n, float(lr), float(beta1), float(beta2), float(eps),
            float(weight_decay), int(step), _stream(stream))
        _lib.check(st, "qlora_adamw_step_scaled")
        return
    st = _lib.load().qlora_adamw_step(_ptr(param), _ptr(grad), _dtype_code(grad.dtype),
                                      _ptr(exp_avg), _ptr(exp_avg_sq), _ptr(param_bf16), n,
                                      float(lr), float(beta1), float(beta2), float(eps),
                                      float(weight_decay), int(step), _stream(stream))
    _lib.check(st, "qlora_adamw_step")


# ------------------------------------------------------------ row operators
_FLOATS = {torch.float32: _lib.DTYPE_F32, torch.bfloat16: _lib.DTYPE_BF16}
_INDEXES = {torch.int32: _lib.DTYPE_I32, torch.int64: _lib.DTYPE_I64}
_F32 = (torch.float32,)
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _elsewhere(dev, stream):
    """Whether a row operator has to change the current device or stream for
    tensors on dev."""
    return stream is not None or dev.type != "cuda" or dev.index != _device_now()


def _place(dev, stream):
    """Context in which a row operator on dev allocates and launches."""
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a ROCm device, got {dev}")
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"stream on {stream.device}, tensors on {dev}")
    return torch.cuda.stream(stream)


def _at(t):
    return None if t is None else t.data_ptr()


# The handle of a device's current stream. torch's own short way to it (0.1 us
# against 1.9 us for current_stream(), of about 8 us for a whole small call)
# is taken where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _here(dev):
    if _raw_stream is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _matrix(t, name, shape, device, codes=False) -> int:
    """Row stride of a [rows, width] fp32 or bf16 matrix (or one of 8-bit codes)
    whose rows are contiguous; shape and device checked."""
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in _FLOATS and not codes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected fp32 or bf16")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    M, N = shape
    ld, step = t.stride()
    if step != 1 and N > 1 and M > 0:
        raise ValueError(f"{name}: rows must be contiguous")
    if M <= 1:
        return max(N, 1)
    if ld < N:
        raise ValueError(f"{name}: row stride {ld} below the width {N}")
    return ld


def _vector(t, name, shape, dtypes, device):
    """_need for an argument that is there, without its conversions: on a
    small call the checks are a part of its time."""
    if t.shape != shape or t.dtype not in dtypes or t.device != device or not t.is_contiguous():
        _need(t, name, shape, tuple(dtypes), device)


def _new(like, M, N, dtype):
    """A matrix on like's device, in its type by default, and its row stride."""
    if dtype is None:
        dtype = like.dtype
    elif dtype not in _FLOATS:
        raise ValueError(f"dtype {dtype}, expected fp32 or bf16")
    return like.new_empty((M, N), dtype=dtype), max(N, 1)


def _indexes(t, name, shape, device) -> int:
    _vector(t, name, shape, _INDEXES, device)
    return _INDEXES[t.dtype]


def _bytes(workspace, need, device):
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    if workspace.dtype != torch.uint8 or workspace.dim() != 1 or not workspace.is_contiguous() \
            or workspace.device != device:
        raise ValueError("workspace: a contiguous 1-D uint8 tensor on the tensors' device")
    return workspace


def _two_dims(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: must have two dimensions, has {t.dim()}")
    return t.shape


def qlora_embed_bwd_workspace_bytes(M: int, D: int) -> int:
    return int(_lib.load().qlora_embed_bwd_workspace_bytes(M, D))


def qlora_norm_bwd_workspace_bytes(M: int, N: int) -> int:
    return int(_lib.load().qlora_norm_bwd_workspace_bytes(M, N))


def qlora_distill_fwd_workspace_bytes(M: int, V: int) -> int:
    return int(_lib.load().qlora_distill_fwd_workspace_bytes(M, V))


def qlora_embed_fwd(W: torch.Tensor, ids: torch.Tensor, scale: float = 1.0,
                    out: torch.Tensor | None = None, out_dtype=None, stream=None) -> torch.Tensor:
    """out[m] = scale * W[ids[m]]: W [V,D] fp32 or bf16, ids [M] int32 or
    int64 (an id outside of [0, V) gives zeros), out [M,D] (W's dtype by
    default)."""
    V, D = _two_dims(W, "W")
    dev = W.device
    M = ids.numel()
    ldw = _matrix(W, "W", (V, D), dev)
    ids_dtype = _indexes(ids, "ids", (M,), dev)
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return qlora_embed_fwd(W, ids, scale, out, out_dtype)
    if out is None:
        out, ldo = _new(W, M, D, out_dtype)
    else:
        ldo = _matrix(out, "out", (M, D), dev)
    st = _lib.load().qlora_embed_fwd(_at(W), ldw, _FLOATS[W.dtype], V, D, _at(ids), ids_dtype,
                                     M, scale, _at(out), ldo, _FLOATS[out.dtype], _here(dev))
    if st:
        _lib.check(st, "qlora_embed_fwd")
    return out


def qlora_embed_bwd(dY: torch.Tensor, ids: torch.Tensor, V: int, scale: float = 1.0,
                    grad_dtype=torch.float32, dW: torch.Tensor | None = None,
                    accumulate: bool = False, workspace: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """The dense gradient of the table: dW[v] = scale * sum of dY's rows with
    id v, [V,D] (grad_dtype, or a given dW's); with accumulate the sums are
    added to the given dW."""
    M, D = _two_dims(dY, "dY")
    dev = dY.device
    ldy = _matrix(dY, "dY", (M, D), dev)
    ids_dtype = _indexes(ids, "ids", (M,), dev)
    if accumulate and dW is None:
        raise ValueError("qlora_embed_bwd: accumulate needs dW")
    _need(dW, "dW", (V, D), tuple(_FLOATS), dev)
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return qlora_embed_bwd(dY, ids, V, scale, grad_dtype, dW, accumulate, workspace)
    if dW is None:
        dW, _ = _new(dY, V, D, grad_dtype)
    workspace = _bytes(workspace, qlora_embed_bwd_workspace_bytes(M, D), dev)
    st = _lib.load().qlora_embed_bwd(_at(dY), ldy, _FLOATS[dY.dtype], _at(ids), ids_dtype, M, V,
                                     D, scale, _at(dW), _FLOATS[dW.dtype], int(accumulate),
                                     _at(workspace), workspace.numel(), _here(dev))
    if st:
        _lib.check(st, "qlora_embed_bwd")
    return dW


def _norm_vectors(N, dev, *named):
    """Dtype code of the affine vectors (they share one; fp32 without any)."""
    code = None
    for t, name in named:
        if t is None:
            continue
        _vector(t, name, (N,), _FLOATS, dev)
        if code is not None and code != _FLOATS[t.dtype]:
            raise ValueError(f"{name}: the affine vectors must share one dtype")
        code = _FLOATS[t.dtype]
    return _lib.DTYPE_F32 if code is None else code


def qlora_norm_fwd(x: torch.Tensor, gamma: torch.Tensor | None = None,
                   beta: torch.Tensor | None = None, eps: float = 1e-5, norm: int = NORM_LAYER,
                   y: torch.Tensor | None = None, y_dtype=None,
                   stats_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Layer norm (NORM_LAYER) or its form without the mean (NORM_RMS) of the
    rows of x [M,N]; y in x's dtype by default. stats_out: fp32 [2,M], receives
    the rows' means and reciprocal standard deviations for the backward."""
    M, N = _two_dims(x, "x")
    dev = x.device
    ldx = _matrix(x, "x", (M, N), dev)
    w_dtype = _norm_vectors(N, dev, (gamma, "gamma"), (beta, "beta"))
    if stats_out is not None:
        _vector(stats_out, "stats_out", (2, M), _F32, dev)
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return qlora_norm_fwd(x, gamma, beta, eps, norm, y, y_dtype, stats_out)
    if y is None:
        y, ldy = _new(x, M, N, y_dtype)
    else:
        ldy = _matrix(y, "y", (M, N), dev)
    st = _lib.load().qlora_norm_fwd(_at(x), ldx, _FLOATS[x.dtype], M, N, norm, _at(gamma),
                                    _at(beta), w_dtype, eps, _at(y), ldy, _FLOATS[y.dtype],
                                    _at(stats_out), _here(dev))
    if st:
        _lib.check(st, "qlora_norm_fwd")
    return y


def qlora_norm_bwd(dY: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor | None = None,
                   eps: float = 1e-5, norm: int = NORM_LAYER, stats: torch.Tensor | None = None,
                   want_dx: bool = True, want_dgamma: bool = True, want_dbeta: bool = True,
                   dx_dtype=None, grad_dtype=torch.float32, workspace: torch.Tensor | None = None,
                   stream=None):
    """Returns (dX or None, dgamma or None, dbeta or None) of the norm: dX in
    x's dtype by default. stats: the forward's stats_out, or None to recompute
    them."""
    M, N = _two_dims(x, "x")
    dev = x.device
    ldx = _matrix(x, "x", (M, N), dev)
    ldy = _matrix(dY, "dY", (M, N), dev)
    w_dtype = _norm_vectors(N, dev, (gamma, "gamma"))
    if stats is not None:
        _vector(stats, "stats", (2, M), _F32, dev)
    dx_dtype = x.dtype if dx_dtype is None else dx_dtype
    if dx_dtype not in _FLOATS or grad_dtype not in _FLOATS:
        raise ValueError("qlora_norm_bwd: gradients are fp32 or bf16")
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return qlora_norm_bwd(dY, x, gamma, eps, norm, stats, want_dx, want_dgamma, want_dbeta,
                                  dx_dtype, grad_dtype, workspace)
    dX = torch.empty((M, N), dtype=dx_dtype, device=dev) if want_dx else None
    dgamma = torch.empty(N, dtype=grad_dtype, device=dev) if want_dgamma else None
    dbeta = torch.empty(N, dtype=grad_dtype, device=dev) if want_dbeta else None
    need = qlora_norm_bwd_workspace_bytes(M, N) if want_dgamma or want_dbeta else 0
    if need or workspace is not None:
        workspace = _bytes(workspace, need, dev)
    st = _lib.load().qlora_norm_bwd(_at(dY), ldy, _FLOATS[dY.dtype], _at(x), ldx,
                                    _FLOATS[x.dtype], M, N, norm, _at(gamma), w_dtype, eps,
                                    _at(stats), _at(dX), N, _FLOATS[dx_dtype], _at(dgamma),
                                    _at(dbeta), _FLOATS[grad_dtype], _at(workspace),
                                    0 if workspace is None else workspace.numel(), _here(dev))
    if st:
        _lib.check(st, "qlora_norm_bwd")
    return dX, dgamma, dbeta


def _top(logits, top_ids, top_logits):
    M, V = _two_dims(logits, "logits")
    k = _two_dims(top_ids, "top_ids")[1]
    dev = logits.device
    ldz = _matrix(logits, "logits", (M, V), dev)
    ids_dtype = _indexes(top_ids, "top_ids", (M, k), dev)
    _vector(top_logits, "top_logits", (M, k), _FLOATS, dev)
    return (_at(logits), ldz, _FLOATS[logits.dtype], M, V, _at(top_ids), ids_dtype,
            _at(top_logits), _FLOATS[top_logits.dtype], k)


def qlora_distill_fwd(logits: torch.Tensor, top_ids: torch.Tensor, top_logits: torch.Tensor,
                      temperature: float = 1.0, loss: torch.Tensor | None = None,
                      stats_out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Loss of each row (fp32 [M]): the divergence of softmax(logits / T) from
    the teacher's softmax over its top logits, times T^2. logits [M,V] fp32 or
    bf16; top_ids [M,k] int32 or int64 (an id outside of [0, V) is no entry),
    top_logits [M,k]. stats_out: fp32 [2,M] for the backward."""
    heads = _top(logits, top_ids, top_logits)
    M, V, dev = heads[3], heads[4], logits.device
    if stats_out is not None:
        _vector(stats_out, "stats_out", (2, M), _F32, dev)
    _need(loss, "loss", (M,), torch.float32, dev)
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return qlora_distill_fwd(logits, top_ids, top_logits, temperature, loss, stats_out,
                                     workspace)
    if loss is None:
        loss = torch.empty(M, dtype=torch.float32, device=dev)
    need = qlora_distill_fwd_workspace_bytes(M, V)
    if need or workspace is not None:
        workspace = _bytes(workspace, need, dev)
    st = _lib.load().qlora_distill_fwd(*heads, temperature, _at(loss), _at(stats_out),
                                       _at(workspace),
                                       0 if workspace is None else workspace.numel(), _here(dev))
    if st:
        _lib.check(st, "qlora_distill_fwd")
    return loss


def qlora_distill_bwd(logits: torch.Tensor, top_ids: torch.Tensor, top_logits: torch.Tensor,
                      dloss: torch.Tensor, stats: torch.Tensor, temperature: float = 1.0,
                      dlogits: torch.Tensor | None = None, grad_dtype=None,
                      stream=None) -> torch.Tensor:
    """Gradient of the rows' losses with respect to the logits, [M,V] (the
    logits' dtype by default), for the rows' gradients dloss (fp32 [M]) and the
    forward's stats_out."""
    heads = _top(logits, top_ids, top_logits)
    M, V, dev = heads[3], heads[4], logits.device
    _vector(stats, "stats", (2, M), _F32, dev)
    _vector(dloss, "dloss", (M,), _F32, dev)
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return qlora_distill_bwd(logits, top_ids, top_logits, dloss, stats, temperature, dlogits,
                                     grad_dtype)
    if dlogits is None:
        dlogits, ldg = _new(logits, M, V, grad_dtype)
    else:
        ldg = _matrix(dlogits, "dlogits", (M, V), dev)
    st = _lib.load().qlora_distill_bwd(*heads, temperature, _at(stats), _at(dloss),
                                       _at(dlogits), ldg, _FLOATS[dlogits.dtype], _here(dev))
    if st:
        _lib.check(st, "qlora_distill_bwd")
    return dlogits


# ------------------------------------------------------- the close of a step
def qlora_add_norm_fwd(x: torch.Tensor, residual: torch.Tensor | None = None,
                       gamma: torch.Tensor | None = None, beta: torch.Tensor | None = None,
                       eps: float = 1e-5, norm: int = NORM_LAYER, h: torch.Tensor | None = None,
                       y: torch.Tensor | None = None, y_dtype=None,
                       scales_out: torch.Tensor | None = None,
                       stats_out: torch.Tensor | None = None, stream=None):
    """h = x + residual in the residual's dtype, and y = the norm of h (as
    qlora_norm_fwd; in x's dtype by default). y_dtype torch.float8_e4m3fn: codes
    of 8 bits with one scale a row, written to scales_out (fp32 [M], needed then).
    h may be given, also as x or residual itself. stats_out: fp32 [2,M]. Without a
    residual h is x. Returns (y, h)."""
    M, N = _two_dims(x, "x")
    dev = x.device
    ldx = _matrix(x, "x", (M, N), dev)
    ldr = ldh = max(N, 1)
    if residual is not None:
        ldr = _matrix(residual, "residual", (M, N), dev)
    elif h is not None:
        raise ValueError("qlora_add_norm_fwd: h needs a residual")
    w_dtype = _norm_vectors(N, dev, (gamma, "gamma"), (beta, "beta"))
    if stats_out is not None:
        _vector(stats_out, "stats_out", (2, M), _F32, dev)
    if y is not None:
        y_dtype = y.dtype
    elif y_dtype is None:
        y_dtype = x.dtype
    codes = y_dtype == torch.float8_e4m3fn
    if not codes and y_dtype not in _FLOATS:
        raise ValueError(f"qlora_add_norm_fwd: y of {y_dtype}, expected fp32, bf16 or float8_e4m3fn")
    if codes != (scales_out is not None):
        raise ValueError("qlora_add_norm_fwd: scales_out goes with y of float8_e4m3fn")
    if codes:
        _vector(scales_out, "scales_out", (M,), _F32, dev)
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return qlora_add_norm_fwd(x, residual, gamma, beta, eps, norm, h, y, y_dtype, scales_out,
                                      stats_out)
    if residual is not None:
        if h is None:
            h, ldh = _new(residual, M, N, None)
        else:
            ldh = _matrix(h, "h", (M, N), dev)
            if h.dtype != residual.dtype:
                raise ValueError(f"h: dtype {h.dtype}, the residual's is {residual.dtype}")
    if y is None:
        y, ldy = x.new_empty((M, N), dtype=y_dtype), max(N, 1)
    else:
        ldy = _matrix(y, "y", (M, N), dev, codes)
    st = _lib.load().qlora_add_norm_fwd(
        _at(x), ldx, _FLOATS[x.dtype], _at(residual), ldr,
        0 if residual is None else _FLOATS[residual.dtype], M, N, norm, _at(gamma), _at(beta),
        w_dtype, eps, _at(h), ldh, _at(y), ldy, _lib.DTYPE_E4M3 if codes else _FLOATS[y_dtype],
        _at(scales_out), _at(stats_out), _here(dev))
    if st:
        _lib.check(st, "qlora_add_norm_fwd")
    return y, x if residual is None else h


def qlora_add_norm_bwd(dY: torch.Tensor, h: torch.Tensor, dH: torch.Tensor | None = None,
                       gamma: torch.Tensor | None = None, eps: float = 1e-5,
                       norm: int = NORM_LAYER, stats: torch.Tensor | None = None,
                       want_dx: bool = True, want_dgamma: bool = True, want_dbeta: bool = True,
                       dx_dtype=None, grad_dtype=torch.float32, dX: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None):
    """Returns (dX or None, dgamma or None, dbeta or None) of the norm behind a
    residual addition: dX, the gradient of x and of the residual, is the norm's
    plus dH, the gradient that reaches h by itself. dX has dH's dtype (h's without
    dH) unless dx_dtype or dX says another, which dH must then have too."""
    M, N = _two_dims(h, "h")
    dev = h.device
    ldh = _matrix(h, "h", (M, N), dev)
    ldy = _matrix(dY, "dY", (M, N), dev)
    lddh = lddx = max(N, 1)
    if dX is not None:
        lddx = _matrix(dX, "dX", (M, N), dev)
        dx_dtype = dX.dtype
    if dx_dtype is None:
        dx_dtype = h.dtype if dH is None else dH.dtype
    if dH is not None:
        lddh = _matrix(dH, "dH", (M, N), dev)
        if dH.dtype != dx_dtype:
            raise ValueError(f"dH: dtype {dH.dtype}, dX has {dx_dtype}")
    w_dtype = _norm_vectors(N, dev, (gamma, "gamma"))
    if stats is not None:
        _vector(stats, "stats", (2, M), _F32, dev)
    if dx_dtype not in _FLOATS or grad_dtype not in _FLOATS:
        raise ValueError("qlora_add_norm_bwd: gradients are fp32 or bf16")
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return qlora_add_norm_bwd(dY, h, dH, gamma, eps, norm, stats, want_dx, want_dgamma,
                                      want_dbeta, dx_dtype, grad_dtype, dX, workspace)
    if dX is None and want_dx:
        dX = torch.empty((M, N), dtype=dx_dtype, device=dev)
    dgamma = torch.empty(N, dtype=grad_dtype, device=dev) if want_dgamma else None
    dbeta = torch.empty(N, dtype=grad_dtype, device=dev) if want_dbeta else None
    need = qlora_norm_bwd_workspace_bytes(M, N) if want_dgamma or want_dbeta else 0
    if need or workspace is not None:
        workspace = _bytes(workspace, need, dev)
    st = _lib.load().qlora_add_norm_bwd(
        _at(dY), ldy, _FLOATS[dY.dtype], _at(dH), lddh, _at(h), ldh, _FLOATS[h.dtype], M, N, norm,
        _at(gamma), w_dtype, eps, _at(stats), _at(dX) if want_dx else None, lddx, _FLOATS[dx_dtype],
        _at(dgamma), _at(dbeta), _FLOATS[grad_dtype], _at(workspace),
        0 if workspace is None else workspace.numel(), _here(dev))
    if st:
        _lib.check(st, "qlora_add_norm_bwd")
    return dX if want_dx else None, dgamma, dbeta


def qlora_head_loss_fwd_workspace_bytes(M: int, V: int, K: int, w_copy: bool = False) -> int:
    return int(_lib.load().qlora_head_loss_fwd_workspace_bytes(M, V, K, int(w_copy)))


def qlora_head_loss_bwd_workspace_bytes(M: int, V: int, K: int, w_copy: bool = False,
                                        dx_dtype=torch.bfloat16, grad_dtype=None) -> int:
    """For dX of dx_dtype and dW of grad_dtype (None: not wanted)."""
    code = lambda dt: -1 if dt is None else _dtype_code(dt)  # noqa: E731
    return int(_lib.load().qlora_head_loss_bwd_workspace_bytes(M, V, K, int(w_copy), code(dx_dtype),
                                                               code(grad_dtype)))


def _head(x, W, labels):
    """The shared arguments of both directions, and whether W is copied (not read
    in place)."""
    M, K = _two_dims(x, "x")
    V = _two_dims(W, "W")[0]
    dev = x.device
    ldx, ldw = _matrix(x, "x", (M, K), dev), _matrix(W, "W", (V, K), dev)
    for t, name in ((x, "x"), (W, "W")):
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name}: dtype {t.dtype}, expected bf16")
    ids_dtype = _indexes(labels, "labels", (M,), dev)
    at = W.data_ptr()
    copy = K % 32 != 0 or ldw % 8 != 0 or ldw > 1 << 20 or at % 16 != 0
    return (_at(x), ldx, at, ldw, M, V, K, _at(labels), ids_dtype), copy


def qlora_head_loss_fwd(x: torch.Tensor, W: torch.Tensor, labels: torch.Tensor, scale: float = 1.0,
                        loss: torch.Tensor | None = None, stats_out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Softmax cross entropy of each row (fp32 [M]) with the logits scale * x W^T,
    which are not kept: x [M,K], W [V,K] bf16, labels [M] int32 or int64 (outside
    of [0, V): no loss, and no work). stats_out: fp32 [2,M] for the backward."""
    head, copy = _head(x, W, labels)
    M, V, K, dev = head[4], head[5], head[6], x.device
    if stats_out is not None:
        _vector(stats_out, "stats_out", (2, M), _F32, dev)
    _need(loss, "loss", (M,), torch.float32, dev)
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return qlora_head_loss_fwd(x, W, labels, scale, loss, stats_out, workspace)
    if loss is None:
        loss = torch.empty(M, dtype=torch.float32, device=dev)
    workspace = _bytes(workspace, qlora_head_loss_fwd_workspace_bytes(M, V, K, copy), dev)
    st = _lib.load().qlora_head_loss_fwd(*head, scale, _at(loss), _at(stats_out), _at(workspace),
                                         workspace.numel(), _here(dev))
    if st:
        _lib.check(st, "qlora_head_loss_fwd")
    return loss


def qlora_head_loss_bwd(x: torch.Tensor, W: torch.Tensor, labels: torch.Tensor,
                        dloss: torch.Tensor, stats: torch.Tensor, scale: float = 1.0,
                        want_dx: bool = True, want_dw: bool = True, dx_dtype=torch.bfloat16,
                        grad_dtype=torch.bfloat16, dX: torch.Tensor | None = None,
                        dW: torch.Tensor | None = None, accumulate: bool = False,
                        workspace: torch.Tensor | None = None, stream=None):
    """Returns (dX or None, dW or None) of the rows' losses for their gradients
    dloss (fp32 [M]) and the forward's stats_out: dX [M,K] in dx_dtype, dW [V,K]
    in grad_dtype (or as they are given); with accumulate the sums are added to
    the given dW."""
    head, copy = _head(x, W, labels)
    M, V, K, dev = head[4], head[5], head[6], x.device
    _vector(stats, "stats", (2, M), _F32, dev)
    _vector(dloss, "dloss", (M,), _F32, dev)
    lddx = K
    if dX is not None:
        lddx, dx_dtype = _matrix(dX, "dX", (M, K), dev), dX.dtype
    if accumulate and want_dw and dW is None:
        raise ValueError("qlora_head_loss_bwd: accumulate needs dW")
    if dW is not None:
        _vector(dW, "dW", (V, K), tuple(_FLOATS), dev)
        grad_dtype = dW.dtype
    if dx_dtype not in _FLOATS or grad_dtype not in _FLOATS:
        raise ValueError("qlora_head_loss_bwd: gradients are fp32 or bf16")
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return qlora_head_loss_bwd(x, W, labels, dloss, stats, scale, want_dx, want_dw, dx_dtype,
                                       grad_dtype, dX, dW, accumulate, workspace)
    if not want_dx:
        dX = None
    elif dX is None:
        dX = torch.empty((M, K), dtype=dx_dtype, device=dev)
    if not want_dw:
        dW = None
    elif dW is None:
        dW = torch.empty((V, K), dtype=grad_dtype, device=dev)
    if want_dx or want_dw:
        need = qlora_head_loss_bwd_workspace_bytes(M, V, K, copy, dx_dtype if want_dx else None,
                                                   grad_dtype if want_dw else None)
        workspace = _bytes(workspace, need, dev)
    st = _lib.load().qlora_head_loss_bwd(
        *head, scale, _at(stats), _at(dloss), _at(dX), lddx, _FLOATS[dx_dtype], _at(dW),
        _FLOATS[grad_dtype], int(accumulate), _at(workspace),
        0 if workspace is None else workspace.numel(), _here(dev))
    if st:
        _lib.check(st, "qlora_head_loss_bwd")
    return dX, dW


class TensorList:
    """Tensors as qlora_grad_norm and qlora_grad_scale take them: contiguous,
    fp32 or bf16, on one device. A program whose gradients stay where they are
    makes the list once (qlora_tensor_list), outside of a graph's capture. It is a
    list of the memory in which they lie then: it holds that memory, and a table
    of its pieces on the device, with which a call is one launch for all of
    them. A tensor that is given other memory later (set_, or a new .grad) is not in
    the list with it; memory that is moved under its tensors (a storage that is
    resized) is refused by every later call. A captured graph has no such check."""

    def __init__(self, tensors, table=True):
        self.tensors = tuple(tensors)
        self.device = self.tensors[0].device if self.tensors else None
        self.array = (_lib.Tensor * max(1, len(self.tensors)))()
        for d, t in zip(self.array, self.tensors):
            if t.dtype not in _FLOATS:
                raise ValueError(f"tensors: dtype {t.dtype}, expected fp32 or bf16")
            if not t.is_contiguous():
                raise ValueError("tensors: must be contiguous")
            if t.device != self.device:
                raise ValueError(f"tensors: on {t.device} and on {self.device}")
            d.data, d.n, d.dtype, d.reserved = t.data_ptr(), t.numel(), _FLOATS[t.dtype], 0
        self.address = ctypes.addressof(self.array)
        # Each storage once: the views of one buffer are checked at once (448 storages
        # of their own take some 60 us a call).
        held = {}
        for t in self.tensors if table else ():
            s = t.untyped_storage()
            held.setdefault(s.data_ptr(), s)
        self.storages = [(s, p) for p, s in held.items()]
        lib, count = _lib.load(), len(self.tensors)
        self.workspace_bytes = int(lib.qlora_grad_norm_workspace_bytes(self.address, count))
        self.table = None
        need = int(lib.qlora_tensor_table_bytes(self.address, count)) if table else 0
        if need:
            rows = torch.empty(need, dtype=torch.uint8)
            _lib.check(lib.qlora_tensor_table(self.address, count, rows.data_ptr(), need),
                       "qlora_tensor_table")
            self.table = rows.to(self.device)

    def __len__(self):
        return len(self.tensors)

    def in_place(self) -> "TensorList":
        """The list itself, if its memory is still where it was."""
        for s, p in self.storages:
            if s.data_ptr() != p:
                raise ValueError("tensors: a storage of the list was moved since the list was made")
        return self


def qlora_tensor_list(tensors) -> TensorList:
    """The tensors as a list that a program keeps (see TensorList)."""
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


def _tensors(tensors) -> TensorList:
    """A list that the program keeps, or one for this call alone."""
    return tensors.in_place() if isinstance(tensors, TensorList) else TensorList(tensors, table=False)


def qlora_grad_norm_workspace_bytes(grads) -> int:
    return _tensors(grads).workspace_bytes


def qlora_grad_norm(grads, max_norm: float = float("inf"), result: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 [2] on the device: the global norm of all gradients (a TensorList or
    tensors), and the factor that clips it to max_norm (1 where the norm is not
    above it)."""
    grads = _tensors(grads)
    dev = grads.device
    if dev is None:
        if result is None:
            raise ValueError("qlora_grad_norm: no tensors, and no result to say on which device")
        dev = result.device
    if result is not None:
        _vector(result, "result", (2,), _F32, dev)
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return qlora_grad_norm(grads, max_norm, result, workspace)
    if result is None:
        result = torch.empty(2, dtype=torch.float32, device=dev)
    if grads.workspace_bytes or workspace is not None:
        workspace = _bytes(workspace, grads.workspace_bytes, dev)
    st = _lib.load().qlora_grad_norm(grads.address, len(grads), _at(grads.table), max_norm,
                                     _at(result), _at(workspace),
                                     0 if workspace is None else workspace.numel(), _here(dev))
    if st:
        _lib.check(st, "qlora_grad_norm")
    return result


def qlora_grad_scale(grads, factor: torch.Tensor, out=None, stream=None) -> None:
    """Every gradient times factor (one fp32 value on the device, such as
    qlora_grad_norm's result[1:]), in place or into out (a TensorList or tensors
    of the same sizes and dtypes)."""
    grads = _tensors(grads)
    dev = grads.device
    _one_factor(factor, "factor")
    if dev is None:
        return
    if factor.device != dev:
        raise ValueError(f"factor: on {factor.device}, expected {dev}")
    if out is not None:
        out = _tensors(out)
        if len(out) != len(grads) or out.device != dev:
            raise ValueError("qlora_grad_scale: out needs as many tensors, on the same device")
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return qlora_grad_scale(grads, factor, out)
    st = _lib.load().qlora_grad_scale(grads.address, None if out is None else out.address,
                                      len(grads), _at(grads.table),
                                      None if out is None else _at(out.table), _at(factor),
                                      _here(dev))
    if st:
        _lib.check(st, "qlora_grad_scale")
