"""ConvRot W8A8 / W4A8 INT8 linear layers for NVIDIA B200 (sm_100a).

A thin Python binding over libconvrot.so (include/convrot.h).  Each function
has the name of the C entry point it calls and only marshals arguments:
PyTorch supplies device memory and the current CUDA stream; every step of the
method runs in the library's CUDA kernels.  There is no CPU fallback: calls
raise if the library or a CUDA device is missing.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _capi

__all__ = [
    "ConvRotError", "lib", "convrot_version", "convrot_device_status",
    "convrot_quantize_weight", "convrot_quantize_weight_w4", "convrot_smoothquant_calibrate",
    "convrot_rotate_quant_act", "convrot_linear_workspace_bytes", "convrot_int8_linear",
    "convrot_w4a8_linear", "convrot_int8_linear_noalloc", "convrot_int8_gemm_s32", "convrot_w4a8_gemm_s32",
    "convrot_swiglu_workspace_bytes", "convrot_int8_linear_swiglu", "convrot_w4a8_linear_swiglu",
    "convrot_interleave_gate_up", "convrot_fold_row_scales",
    "convrot_rotate_act_bf16", "convrot_weight_only_workspace_bytes", "convrot_weight_only_linear",
    "convrot_weight_only_gemm_f32",
    "convrot_rope_append", "convrot_attention_prompt",
    "convrot_attention_decode_workspace_bytes", "convrot_attention_decode",
    "Workspace", "ConvRotLinear", "ConvRotFusedLinear", "ConvRotMLP",
    "rope_table", "PagedKVCache", "ConvRotAttention",
]


class ConvRotError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {_capi.STATUS.get(status, status)}")


def lib():
    return _capi.load()


def _check(fn: str, status: int):
    if status != 0:
        raise ConvRotError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t: torch.Tensor, dtype, name: str, dim: Optional[int] = None, shape=None):
    """dtype, contiguity and shape of one operand.  The device is checked
    afterwards, for all operands of a call together (_on_device)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _on_device(**operands) -> torch.device:
    """Every operand is a CUDA tensor on one device, and that device is the
    current one: the library launches on the current device, on that device's
    current stream.  None entries (optional operands) are skipped."""
    dev = None
    for name, t in operands.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (no CPU fallback)")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}; the other operands are on {dev}")
    cur = torch.cuda.current_device()
    if dev.index != cur:
        raise ValueError(f"the operands are on {dev} but the current device is cuda:{cur}")
    return dev


def convrot_version() -> int:
    return lib().convrot_version()


# Device timeouts reported so far.  A kernel that gave up on a bounded wait may
# leave partial sums and tile counters in its split-tile workspace; every
# Workspace zero-fills itself again before its next use once this has moved.
_timeouts_reported = 0


def _note_status(st: int) -> None:
    global _timeouts_reported
    if st == 6:  # CONVROT_ERR_DEVICE_TIMEOUT
        _timeouts_reported += 1


def convrot_device_status(device=None) -> int:
    """Synchronises the current stream and returns/clears the device error word.

    Bit 0: a kernel gave up on a bounded wait; every Workspace is then
    zero-filled again before its next use.  Bit 1: an attention kernel met a
    position, slot, page or length outside its tensor and left that access out."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
    detail = ctypes.c_uint32(0)
    st = lib().convrot_device_status(_stream(dev), ctypes.byref(detail))
    if st not in (0, 2, 6):
        _check("convrot_device_status", st)
    _note_status(st)
    return int(detail.value)


# ---------------------------------------------------------------- weights
def convrot_quantize_weight(W: torch.Tensor, group: int = 256,
                            col_scale: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    _need(W, torch.bfloat16, "W", 2)
    N, K = W.shape
    if col_scale is not None:
        _need(col_scale, torch.float32, "col_scale", shape=(K,))
    _on_device(W=W, col_scale=col_scale)
    Wq = torch.empty(N, K, dtype=torch.int8, device=W.device)
    s_row = torch.empty(N, dtype=torch.float32, device=W.device)
    _check("convrot_quantize_weight", lib().convrot_quantize_weight(
        _ptr(W), N, K, group, _ptr(col_scale), _ptr(Wq), _ptr(s_row), _stream(W.device)))
    return Wq, s_row


def convrot_quantize_weight_w4(W: torch.Tensor, group: int = 256,
                               col_scale: Optional[torch.Tensor] = None, clip_lo: float = 0.80,
                               clip_hi: float = 1.00, clip_steps: int = 21):
    _need(W, torch.bfloat16, "W", 2)
    N, K = W.shape
    if col_scale is not None:
        _need(col_scale, torch.float32, "col_scale", shape=(K,))
    _on_device(W=W, col_scale=col_scale)
    Wq4 = torch.empty(N, K // 2, dtype=torch.uint8, device=W.device)
    s_row = torch.empty(N, dtype=torch.float32, device=W.device)
    _check("convrot_quantize_weight_w4", lib().convrot_quantize_weight_w4(
        _ptr(W), N, K, group, _ptr(col_scale), clip_lo, clip_hi, clip_steps, _ptr(Wq4),
        _ptr(s_row), _stream(W.device)))
    return Wq4, s_row


def convrot_smoothquant_calibrate(x: torch.Tensor, norm_w: Optional[torch.Tensor], W: torch.Tensor,
                                  eps: float = 1e-6, alpha: float = 0.5):
    """SmoothQuant scales of the linear W fed by x (norm_w None: x reaches W as
    it is, and the second result is scratch)."""
    _need(x, torch.bfloat16, "x", 2)
    M, K = x.shape
    _need(W, torch.bfloat16, "W", 2)
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("x and W disagree on K")
    if norm_w is not None:
        _need(norm_w, torch.float32, "norm_w", shape=(K,))
    _on_device(x=x, W=W, norm_w=norm_w)
    smooth = torch.empty(K, dtype=torch.float32, device=x.device)
    folded = torch.empty(K, dtype=torch.float32, device=x.device)
    _check("convrot_smoothquant_calibrate", lib().convrot_smoothquant_calibrate(
        _ptr(x), M, K, _ptr(norm_w), eps, _ptr(W), N, alpha, _ptr(smooth), _ptr(folded),
        _stream(x.device)))
    return smooth, folded


# ---------------------------------------------------------------- activations
def convrot_rotate_quant_act(x: torch.Tensor, group: int = 256,
                             norm_w: Optional[torch.Tensor] = None, eps: float = 1e-6,
                             out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    _need(x, torch.bfloat16, "x", 2)
    M, K = x.shape
    if norm_w is not None:
        _need(norm_w, torch.float32, "norm_w", shape=(K,))
    if out is None:
        Xq = s_tok = None
    else:
        Xq, s_tok = out
        _need(Xq, torch.int8, "Xq", shape=(M, K))
        _need(s_tok, torch.float32, "s_tok", shape=(M,))
    _on_device(x=x, norm_w=norm_w, Xq=Xq, s_tok=s_tok)
    if out is None:
        Xq = torch.empty(M, K, dtype=torch.int8, device=x.device)
        s_tok = torch.empty(M, dtype=torch.float32, device=x.device)
    _check("convrot_rotate_quant_act", lib().convrot_rotate_quant_act(
        _ptr(x), M, K, group, _ptr(norm_w), eps, _ptr(Xq), _ptr(s_tok), _stream(x.device)))
    return Xq, s_tok


# ---------------------------------------------------------------- GEMM
def convrot_linear_workspace_bytes(M: int, N: int, K: int, weight_bits: int = 8) -> int:
    return int(lib().convrot_linear_workspace_bytes(M, N, K, weight_bits))


def _capturing(device: torch.device) -> bool:
    return device.type == "cuda" and torch.cuda.is_current_stream_capturing()


class Workspace:
    """Device workspace for the GEMM's split tiles, grown on demand.

    It starts zero-filled; the library leaves it zero after every call whose
    kernels complete, so it is reused without clearing.  After
    convrot_device_status has reported a device timeout (an aborted call may
    leave partial sums behind) it is zero-filled again before its next use;
    graphs captured with it before are to be captured again.
    One Workspace must not be used by calls that run concurrently on
    different streams, replays of captured graphs among them.

    A call captured into a graph takes the buffer if it is there, large enough
    and clear by then.  Otherwise (no call has run before the capture) it takes
    one of the graph's own, which every replay clears.  When the Workspace grows,
    at least to twice its size, the buffers before stay: captured graphs may go
    on using them.
    """

    kept = ()       # the buffers before self.buf
    own = None      # the graph's own buffer that was handed out last

    def __init__(self, device=None):
        self.device = torch.device("cuda", torch.cuda.current_device() if device is None else device)
        self.buf: Optional[torch.Tensor] = None
        self.epoch = _timeouts_reported

    def get(self, nbytes: int) -> Tuple[Optional[int], int]:
        if nbytes == 0:
            return None, 0
        short = self.buf is None or self.buf.numel() < nbytes
        if short or self.epoch != _timeouts_reported:
            if _capturing(self.device):  # (a fill recorded here runs at the replays, not now)
                self.own = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
                return self.own.data_ptr(), nbytes
            if short:
                if self.buf is not None:
                    self.kept = (*self.kept, self.buf)
                    nbytes = max(nbytes, 2 * self.buf.numel())
                self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
            else:
                self.buf.zero_()
            self.epoch = _timeouts_reported
        return self.buf.data_ptr(), self.buf.numel()


_default_ws = {}


def _workspace_on(index: int, ws: Workspace) -> Workspace:
    if ws.device.index != index:
        raise ValueError(f"the workspace is on {ws.device}, the operands are on cuda:{index}")
    return ws


def _workspace(dev: torch.device, nbytes: int, ws: Optional[Workspace]):
    if ws is None:
        key = (dev.index, torch.cuda.current_stream(dev).cuda_stream)
        ws = _default_ws.get(key)
        if ws is None:
            ws = _default_ws[key] = Workspace(dev.index)
    p, n = _workspace_on(dev.index, ws).get(nbytes)
    return (ctypes.c_void_p(p) if p else None), n


def _gemm_check(Xq, Wq, w4: bool):
    _need(Xq, torch.int8, "Xq", 2)
    _need(Wq, torch.uint8 if w4 else torch.int8, "Wq4" if w4 else "Wq", 2)
    M, K = Xq.shape
    N = Wq.shape[0]
    if Wq.shape[1] * (2 if w4 else 1) != K:
        raise ValueError("weight and activation disagree on K")
    return M, N, K


def _linear_operands(Xq, s_tok, Wq, s_row, out, w4: bool, out_cols=None):
    """Checks the operands of a W8A8 / W4A8 linear; returns (M, N, K, Y) with
    Y the caller's `out` or a new bf16 [M, out_cols] tensor."""
    M, N, K = _gemm_check(Xq, Wq, w4)
    cols = N if out_cols is None else out_cols
    _need(s_tok, torch.float32, "s_tok", shape=(M,))
    _need(s_row, torch.float32, "s_row", shape=(N,))
    if out is not None:
        _need(out, torch.bfloat16, "out", shape=(M, cols))
    dev = _on_device(Xq=Xq, s_tok=s_tok, Wq=Wq, s_row=s_row, out=out)
    Y = torch.empty(M, cols, dtype=torch.bfloat16, device=dev) if out is None else out
    return M, N, K, Y


def convrot_int8_linear(Xq, s_tok, Wq, s_row, out=None, workspace: Optional[Workspace] = None):
    M, N, K, Y = _linear_operands(Xq, s_tok, Wq, s_row, out, False)
    ws, wn = _workspace(Xq.device, convrot_linear_workspace_bytes(M, N, K, 8), workspace)
    _check("convrot_int8_linear", lib().convrot_int8_linear(
        _ptr(Xq), _ptr(s_tok), _ptr(Wq), _ptr(s_row), M, N, K, _ptr(Y), ws, wn,
        _stream(Xq.device)))
    return Y


def convrot_int8_linear_noalloc(Xq, s_tok, Wq, s_row, out=None):
    """convrot_int8_linear without a caller workspace: the library's fixed
    24 MiB per-device array serves as the split-tile workspace (for callers
    that cannot allocate device memory where they run the layer).  Calls that
    overlap on the GPU race on that array."""
    M, N, K, Y = _linear_operands(Xq, s_tok, Wq, s_row, out, False)
    _check("convrot_int8_linear_noalloc", lib().convrot_int8_linear_noalloc(
        _ptr(Xq), _ptr(s_tok), _ptr(Wq), _ptr(s_row), M, N, K, _ptr(Y), _stream(Xq.device)))
    return Y


def convrot_w4a8_linear(Xq, s_tok, Wq4, s_row, out=None, workspace: Optional[Workspace] = None):
    M, N, K, Y = _linear_operands(Xq, s_tok, Wq4, s_row, out, True)
    ws, wn = _workspace(Xq.device, convrot_linear_workspace_bytes(M, N, K, 4), workspace)
    _check("convrot_w4a8_linear", lib().convrot_w4a8_linear(
        _ptr(Xq), _ptr(s_tok), _ptr(Wq4), _ptr(s_row), M, N, K, _ptr(Y), ws, wn,
        _stream(Xq.device)))
    return Y


def convrot_int8_gemm_s32(Xq, Wq, workspace: Optional[Workspace] = None):
    M, N, K = _gemm_check(Xq, Wq, False)
    _on_device(Xq=Xq, Wq=Wq)
    acc = torch.empty(M, N, dtype=torch.int32, device=Xq.device)
    ws, wn = _workspace(Xq.device, convrot_linear_workspace_bytes(M, N, K, 8), workspace)
    _check("convrot_int8_gemm_s32", lib().convrot_int8_gemm_s32(
        _ptr(Xq), _ptr(Wq), M, N, K, _ptr(acc), ws, wn, _stream(Xq.device)))
    return acc


def convrot_w4a8_gemm_s32(Xq, Wq4, workspace: Optional[Workspace] = None):
    M, N, K = _gemm_check(Xq, Wq4, True)
    _on_device(Xq=Xq, Wq4=Wq4)
    acc = torch.empty(M, N, dtype=torch.int32, device=Xq.device)
    ws, wn = _workspace(Xq.device, convrot_linear_workspace_bytes(M, N, K, 4), workspace)
    _check("convrot_w4a8_gemm_s32", lib().convrot_w4a8_gemm_s32(
        _ptr(Xq), _ptr(Wq4), M, N, K, _ptr(acc), ws, wn, _stream(Xq.device)))
    return acc


# ---------------------------------------------------------------- weight-only path
def convrot_rotate_act_bf16(x: torch.Tensor, group: int = 256, norm_w: Optional[torch.Tensor] = None,
                            eps: float = 1e-6, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Xr = bf16([RMSNorm] x rotated by the group Hadamard), not quantised."""
    _need(x, torch.bfloat16, "x", 2)
    M, K = x.shape
    if norm_w is not None:
        _need(norm_w, torch.float32, "norm_w", shape=(K,))
    if out is not None:
        _need(out, torch.bfloat16, "out", shape=(M, K))
    _on_device(x=x, norm_w=norm_w, out=out)
    Xr = torch.empty(M, K, dtype=torch.bfloat16, device=x.device) if out is None else out
    _check("convrot_rotate_act_bf16", lib().convrot_rotate_act_bf16(
        _ptr(x), M, K, group, _ptr(norm_w), eps, _ptr(Xr), _stream(x.device)))
    return Xr


def _wo_check(Xr, Wq):
    _need(Xr, torch.bfloat16, "Xr", 2)
    _need(Wq, torch.int8, "Wq", 2)
    if Xr.shape[1] != Wq.shape[1]:
        raise ValueError("weight and activation disagree on K")
    return Xr.shape[0], Wq.shape[0], Xr.shape[1]


def convrot_weight_only_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().convrot_weight_only_workspace_bytes(M, N, K))


def convrot_weight_only_linear(Xr, Wq, s_row, out=None, workspace: Optional[Workspace] = None):
    """Y = bf16(s_row * (Xr @ Wq^T)) on rotated bf16 activations, int8 weights."""
    M, N, K = _wo_check(Xr, Wq)
    _need(s_row, torch.float32, "s_row", shape=(N,))
    if out is not None:
        _need(out, torch.bfloat16, "out", shape=(M, N))
    _on_device(Xr=Xr, Wq=Wq, s_row=s_row, out=out)
    Y = torch.empty(M, N, dtype=torch.bfloat16, device=Xr.device) if out is None else out
    ws, wn = _workspace(Xr.device, convrot_weight_only_workspace_bytes(M, N, K), workspace)
    _check("convrot_weight_only_linear", lib().convrot_weight_only_linear(
        _ptr(Xr), _ptr(Wq), _ptr(s_row), M, N, K, _ptr(Y), ws, wn, _stream(Xr.device)))
    return Y


def convrot_weight_only_gemm_f32(Xr, Wq, workspace: Optional[Workspace] = None):
    M, N, K = _wo_check(Xr, Wq)
    _on_device(Xr=Xr, Wq=Wq)
    acc = torch.empty(M, N, dtype=torch.float32, device=Xr.device)
    ws, wn = _workspace(Xr.device, convrot_weight_only_workspace_bytes(M, N, K), workspace)
    _check("convrot_weight_only_gemm_f32", lib().convrot_weight_only_gemm_f32(
        _ptr(Xr), _ptr(Wq), M, N, K, _ptr(acc), ws, wn, _stream(Xr.device)))
    return acc


# ---------------------------------------------------------------- MLP boundary
def convrot_swiglu_workspace_bytes(M: int, I: int, K: int, weight_bits: int = 8) -> int:
    return int(lib().convrot_swiglu_workspace_bytes(M, I, K, weight_bits))


def _swiglu(fn, Xq, s_tok, Wq_gu, s_row_gu, w4, out, workspace):
    M, N2, K = _gemm_check(Xq, Wq_gu, w4)
    if N2 % 2:
        raise ValueError("the gate/up weight must have an even number of rows")
    I = N2 // 2
    M, N2, K, H = _linear_operands(Xq, s_tok, Wq_gu, s_row_gu, out, w4, out_cols=I)
    ws, wn = _workspace(Xq.device, convrot_swiglu_workspace_bytes(M, I, K, 4 if w4 else 8), workspace)
    _check(fn, getattr(lib(), fn)(
        _ptr(Xq), _ptr(s_tok), _ptr(Wq_gu), _ptr(s_row_gu), M, I, K, _ptr(H), ws, wn,
        _stream(Xq.device)))
    return H


def convrot_int8_linear_swiglu(Xq, s_tok, Wq_gu, s_row_gu, out=None,
                               workspace: Optional[Workspace] = None):
    """H = bf16(SiLU(gate) * up) from interleaved gate/up rows (I = rows / 2)."""
    return _swiglu("convrot_int8_linear_swiglu", Xq, s_tok, Wq_gu, s_row_gu, False, out, workspace)


def convrot_w4a8_linear_swiglu(Xq, s_tok, Wq4_gu, s_row_gu, out=None,
                               workspace: Optional[Workspace] = None):
    return _swiglu("convrot_w4a8_linear_swiglu", Xq, s_tok, Wq4_gu, s_row_gu, True, out, workspace)


def convrot_interleave_gate_up(Wg: torch.Tensor, Wu: torch.Tensor) -> torch.Tensor:
    """Rows of gate and up in alternating blocks of 16 (any dtype, 1-D or 2-D)."""
    if Wg.shape != Wu.shape or Wg.dtype != Wu.dtype or Wg.device != Wu.device:
        raise ValueError("gate and up must match in shape, dtype and device")
    if not (Wg.is_contiguous() and Wu.is_contiguous()):
        raise ValueError("gate and up must be contiguous")
    _on_device(Wg=Wg, Wu=Wu)
    I = Wg.shape[0]
    row_bytes = Wg.numel() // max(I, 1) * Wg.element_size()
    out = torch.empty((2 * I,) + tuple(Wg.shape[1:]), dtype=Wg.dtype, device=Wg.device)
    _check("convrot_interleave_gate_up", lib().convrot_interleave_gate_up(
        _ptr(Wg), _ptr(Wu), I, row_bytes, _ptr(out), _stream(Wg.device)))
    return out


def convrot_fold_row_scales(s_row: torch.Tensor, smooth: torch.Tensor) -> torch.Tensor:
    """s_row /= smooth in place (a SmoothQuant scale folded into weight rows)."""
    _need(s_row, torch.float32, "s_row", 1)
    _need(smooth, torch.float32, "smooth", shape=tuple(s_row.shape))
    _on_device(s_row=s_row, smooth=smooth)
    _check("convrot_fold_row_scales", lib().convrot_fold_row_scales(
        _ptr(s_row), _ptr(smooth), s_row.numel(), _stream(s_row.device)))
    return s_row


# ---------------------------------------------------------------- attention
# These calls are short on the GPU (a decode step's append takes 2 us), so their
# checks first ask whether all is well in as few steps as there are, and look
# for what is wrong only if it is not.
def _heads(t: torch.Tensor, name: str, rows: Optional[int] = None, heads: Optional[int] = None,
           dim: Optional[int] = None):
    """A bf16 [rows, heads, D] operand whose heads lie next to one another; rows
    may be further apart (a column view of a fused projection's output).
    Returns (rows, heads, D, row stride)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dimensions [rows, heads, D]")
    r, h, d = t.shape
    if (rows is not None and r != rows) or (heads is not None and h != heads) or (dim is not None and d != dim):
        for got, want, what in ((r, rows, "rows"), (h, heads, "heads"), (d, dim, "elements per head")):
            if want is not None and got != want:
                raise ValueError(f"{name} must have {want} {what}, got {got}")
    sr, sh, sd = t.stride()
    if (sd != 1 or (sh != d and h > 1) or (r > 1 and (sr < h * d or sr % 8))) and t.numel():
        raise ValueError(f"{name} must have contiguous heads and rows a multiple of 8 elements apart, got strides {t.stride()}")
    return r, h, d, sr if r > 1 else h * d


def _vector(t: torch.Tensor, dtype, name: str, n: int):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == (n,) and t.is_contiguous()):
        _need(t, dtype, name, shape=(n,))


def _cache(k_cache, v_cache, k_scale, v_scale):
    """Checks a paged cache; returns (pages, kv_heads, page_size, D)."""
    i8 = k_scale is not None or v_scale is not None
    dtype = torch.int8 if i8 else torch.bfloat16
    _need(k_cache, dtype, "k_cache", 4)
    shape = k_cache.shape
    if not (isinstance(v_cache, torch.Tensor) and v_cache.dtype is dtype and v_cache.shape == shape
            and v_cache.is_contiguous()):
        _need(v_cache, dtype, "v_cache", shape=shape)
    if i8:
        _need(k_scale, torch.float32, "k_scale", shape=shape[:3])
        _need(v_scale, torch.float32, "v_scale", shape=shape[:3])
    return shape


def _current_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# the same handle without building a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _one_device(names, *operands):
    """_on_device for operands given in the order of `names`; returns the index
    of the device and its current stream's handle."""
    at = operands[0].get_device()
    if at >= 0 and at == torch.cuda.current_device():
        for t in operands:
            if t is not None and t.get_device() != at:
                break
        else:
            return at, _raw_stream(at)
    dev = _on_device(**dict(zip(names.split(), operands)))
    return dev.index, _raw_stream(dev.index)


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def convrot_rope_append(q, k, v, rope, positions, slots, k_cache, v_cache, *, k_scale=None, v_scale=None,
                        q_norm=None, k_norm=None, eps: float = 1e-6, q_out=None, k_out=None):
    """Rotates q and k (after an optional per-head RMSNorm) by their positions'
    rows of the table `rope` and writes k and v into a paged cache at `slots`
    (page * page_size + offset; negative: nowhere).  Returns (q_out, k_out);
    the rotated k is written only where the caller gives a k_out.  q_out and
    k_out may be q and k themselves."""
    T, Hq, D, sq = _heads(q, "q")
    _, Hkv, _, sk = _heads(k, "k", T, None, D)
    sv = _heads(v, "v", T, Hkv, D)[3]
    pages, heads, page_size, dim = _cache(k_cache, v_cache, k_scale, v_scale)
    if heads != Hkv or dim != D:
        raise ValueError(f"k_cache must hold {Hkv} heads of {D} elements, got shape {tuple(k_cache.shape)}")
    _need(rope, torch.float32, "rope", 2)
    _vector(positions, torch.int32, "positions", T)
    _vector(slots, torch.int64, "slots", T)
    if q_norm is not None:
        _vector(q_norm, torch.float32, "q_norm", D)
    if k_norm is not None:
        _vector(k_norm, torch.float32, "k_norm", D)
    sqo = sq if q_out is q else _heads(q_out, "q_out", T, Hq, D)[3] if q_out is not None else Hq * D
    sko = _heads(k_out, "k_out", T, Hkv, D)[3] if k_out is not None else 0
    dev, stream = _one_device("q k v rope positions slots k_cache v_cache k_scale v_scale q_norm k_norm q_out k_out", q, k, v,
                              rope, positions, slots, k_cache, v_cache, k_scale, v_scale, q_norm, k_norm, q_out, k_out)
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    R, turned = rope.shape
    _check("convrot_rope_append", lib().convrot_rope_append(
        q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, T, Hq, Hkv, D, rope.data_ptr(), R, turned, positions.data_ptr(),
        slots.data_ptr(), _at(q_norm), _at(k_norm), eps, q_out.data_ptr(), sqo, _at(k_out), sko, k_cache.data_ptr(),
        v_cache.data_ptr(), _at(k_scale), _at(v_scale), pages, page_size, stream))
    return q_out, k_out


def convrot_attention_prompt(q, k, v, cu_seqlens, cu_seqlens_k=None, *, scale: Optional[float] = None,
                             causal: bool = True, out=None):
    """Attention over whole prompts packed one after another: sequence i is rows
    cu_seqlens[i] .. cu_seqlens[i + 1] of q, and of k and v unless they have
    offsets of their own.  scale None: D ** -0.5.  A new `out` is not
    initialised: rows of no sequence hold what the memory held."""
    T, Hq, D, sq = _heads(q, "q")
    Tk, Hkv, _, sk = _heads(k, "k", None, None, D)
    sv = _heads(v, "v", Tk, Hkv, D)[3]
    _need(cu_seqlens, torch.int32, "cu_seqlens", 1)
    n = cu_seqlens.shape[0] - 1
    if cu_seqlens_k is None:
        if Tk != T:
            raise ValueError("k and q have different lengths: cu_seqlens_k is needed")
        cu_seqlens_k = cu_seqlens
    else:
        _vector(cu_seqlens_k, torch.int32, "cu_seqlens_k", n + 1)
    if n < 0:
        raise ValueError("cu_seqlens must hold one offset more than there are sequences")
    so = _heads(out, "out", T, Hq, D)[3] if out is not None else Hq * D
    dev, stream = _one_device("q k v cu_seqlens cu_seqlens_k out", q, k, v, cu_seqlens, cu_seqlens_k, out)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    _check("convrot_attention_prompt", lib().convrot_attention_prompt(
        q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, T, Tk, Hq, Hkv, D, cu_seqlens.data_ptr(),
        cu_seqlens_k.data_ptr(), n, D ** -0.5 if scale is None else scale, int(causal), out.data_ptr(), so, stream))
    return out


def convrot_attention_decode_workspace_bytes(seqs: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().convrot_attention_decode_workspace_bytes(seqs, q_heads, kv_heads, head_dim))


# workspace sizes by device and heads: they do not depend on the batch
_decode_ws_bytes = {}


def convrot_attention_decode(q, k_cache, v_cache, block_table, seq_lens, *, k_scale=None, v_scale=None,
                             scale: Optional[float] = None, out=None, workspace: Optional[Workspace] = None):
    """Attention of one new token per sequence over a paged cache (bf16, or
    int8 with scales).  seq_lens counts the new token, whose key and value the
    cache already holds.  scale None: D ** -0.5."""
    B, Hq, D, sq = _heads(q, "q")
    pages, Hkv, page_size, Dc = _cache(k_cache, v_cache, k_scale, v_scale)
    if Dc != D:
        raise ValueError(f"q has {D} elements per head, the cache {Dc}")
    if not isinstance(block_table, torch.Tensor) or block_table.dtype is not torch.int32:
        raise TypeError("block_table must be a torch.int32 tensor")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must have shape ({B}, pages per sequence), got {tuple(block_table.shape)}")
    cols = block_table.shape[1]
    st, sc = block_table.stride()
    if ((cols > 1 and sc != 1) or (B > 1 and st < cols)) and block_table.numel():
        raise ValueError("block_table must have contiguous rows")
    _vector(seq_lens, torch.int32, "seq_lens", B)
    so = _heads(out, "out", B, Hq, D)[3] if out is not None else Hq * D
    dev, stream = _one_device("q k_cache v_cache block_table seq_lens k_scale v_scale out", q, k_cache, v_cache, block_table,
                              seq_lens, k_scale, v_scale, out)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if workspace is None:
        workspace = _default_ws.get((dev, stream)) or _default_ws.setdefault((dev, stream), Workspace(dev))
        capturing = torch.cuda.is_current_stream_capturing()
    else:
        _workspace_on(dev, workspace)
        capturing = False
    need = _decode_ws_bytes.get((dev, Hq, Hkv, D))
    if need is None and B:
        need = _decode_ws_bytes[dev, Hq, Hkv, D] = convrot_attention_decode_workspace_bytes(B, Hq, Hkv, D)
    if capturing and B:
        # a captured graph gets its own: graphs may be replayed at the same time
        own = torch.empty(need, dtype=torch.uint8, device=q.device)
        own[:4096].zero_()
        ws, wn = own.data_ptr(), need
    else:
        ws, wn = workspace.get(need or 0)
    _check("convrot_attention_decode", lib().convrot_attention_decode(
        q.data_ptr(), sq, B, Hq, Hkv, D, k_cache.data_ptr(), v_cache.data_ptr(), _at(k_scale), _at(v_scale), pages, page_size,
        block_table.data_ptr(), st if B > 1 else cols, cols, seq_lens.data_ptr(), D ** -0.5 if scale is None else scale,
        out.data_ptr(), so, ws, wn, stream))
    return out


class ConvRotLinear:
    """A quantised linear layer: prepared weights plus the per-token forward.

    forward(x) = convrot_rotate_quant_act (optionally with the fused RMSNorm)
    followed by convrot_int8_linear / convrot_w4a8_linear.
    """

    def __init__(self, W: torch.Tensor, *, weight_bits: int = 8, group: int = 256,
                 norm_w: Optional[torch.Tensor] = None, col_scale: Optional[torch.Tensor] = None,
                 eps: float = 1e-6):
        self.group = group
        self.weight_bits = weight_bits
        self.eps = eps
        self.norm_w = norm_w
        self.N, self.K = W.shape
        if weight_bits == 8:
            self.Wq, self.s_row = convrot_quantize_weight(W, group, col_scale)
        elif weight_bits == 4:
            self.Wq, self.s_row = convrot_quantize_weight_w4(W, group, col_scale)
        else:
            raise ValueError("weight_bits must be 8 or 4")
        self.workspace = Workspace(W.device.index)

    @classmethod
    def from_checkpoint(cls, layer: dict, *, device=None, norm_w: Optional[torch.Tensor] = None,
                        eps: float = 1e-6):
        """A linear from an entry of checkpoint.load_quantized_layers (the stored
        codes and row scales are used as they are; nothing is re-quantised)."""
        self = cls.__new__(cls)
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
        self.group, self.weight_bits, self.eps, self.norm_w = int(layer["group"]), int(layer["bits"]), eps, norm_w
        self.Wq = torch.from_numpy(layer["Wq"]).to(dev)
        self.s_row = torch.from_numpy(layer["s_row"]).to(dev)
        self.N = self.Wq.shape[0]
        self.K = self.Wq.shape[1] * (2 if self.weight_bits == 4 else 1)
        self.workspace = Workspace(dev.index)
        return self

    def to_checkpoint(self) -> dict:
        """The layer's stored form for checkpoint.save_quantized_layers."""
        return {"Wq": self.Wq.cpu().numpy(), "s_row": self.s_row.cpu().numpy(),
                "group": self.group, "bits": self.weight_bits}

    @classmethod
    def with_smoothquant(cls, W, x_calib, norm_w, *, weight_bits=8, group=256, eps=1e-6, alpha=0.5):
        smooth, folded = convrot_smoothquant_calibrate(x_calib, norm_w, W, eps, alpha)
        return cls(W, weight_bits=weight_bits, group=group, norm_w=folded, col_scale=smooth, eps=eps)

    def forward_weight_only(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The same layer with bf16 activations: rotate (no quantisation), then the
        bf16 tensor-core GEMM over the int8 weight codes (int8 weights only)."""
        if self.weight_bits != 8:
            raise ValueError("the weight-only path takes int8 weights")
        Xr = convrot_rotate_act_bf16(x, self.group, self.norm_w, self.eps)
        return convrot_weight_only_linear(Xr, self.Wq, self.s_row, out, self.workspace)

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        Xq, s_tok = convrot_rotate_quant_act(x, self.group, self.norm_w, self.eps)
        if self.weight_bits == 8:
            return convrot_int8_linear(Xq, s_tok, self.Wq, self.s_row, out, self.workspace)
        return convrot_w4a8_linear(Xq, s_tok, self.Wq, self.s_row, out, self.workspace)

    __call__ = forward


class ConvRotFusedLinear:
    """Several linears that read the same input, run as ONE GEMM over their
    concatenated output rows: a fused projection set such as q/k/v of an
    attention block, or a gated-DeltaNet input projection together with its
    small-N companion (the MOSS-Image card quantises attention, gated-DeltaNet
    projections and MLP linears).  Every row is quantised on its own, so the
    fused layer's codes, scales and outputs are those of the separate layers;
    one launch replaces several, and small-N members no longer under-fill the
    GPU.  A shared SmoothQuant scale (with a norm) is calibrated over all
    members' columns, since they share the input.
    """

    def __init__(self, weights, *, weight_bits: int = 8, group: int = 256,
                 norm_w: Optional[torch.Tensor] = None, x_calib: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, alpha: float = 0.5):
        W = torch.cat(list(weights))
        self.sizes = [int(w.shape[0]) for w in weights]
        col = None
        if x_calib is not None and norm_w is not None:
            col, norm_w = convrot_smoothquant_calibrate(x_calib, norm_w, W, eps, alpha)
        self.col_scale = col
        self.linear = ConvRotLinear(W, weight_bits=weight_bits, group=group, norm_w=norm_w,
                                    col_scale=col, eps=eps)

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None):
        """One output per member, as column views of the fused [M, sum N] result."""
        return torch.split(self.linear(x, out), self.sizes, dim=1)

    __call__ = forward


class ConvRotMLP:
    """The MLP block down(SiLU(gate(x)) * up(x)) of the quantised decoder layer.

    forward(x) = rotate-quantise (with the fused RMSNorm) -> one gate/up GEMM
    whose epilogue writes H = SiLU(g) * u -> rotate-quantise H -> down_proj.
    With calibration input, SmoothQuant scales are folded into the norm
    weight (gate/up input) and into up_proj's row scales (down_proj input),
    as the MOSS-Image card's "How it was made" describes.
    """

    def __init__(self, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor, *,
                 norm_w: Optional[torch.Tensor] = None, x_calib: Optional[torch.Tensor] = None,
                 group: int = 256, eps: float = 1e-6, alpha: float = 0.5):
        self.group, self.eps = group, eps
        self.I, self.H = Wg.shape
        self.workspace = Workspace(Wg.device.index)
        col = None
        self.norm_w = norm_w
        if x_calib is not None and norm_w is not None:
            col, self.norm_w = convrot_smoothquant_calibrate(x_calib, norm_w, torch.cat([Wg, Wu]), eps, alpha)
        Wq_g, s_g = convrot_quantize_weight(Wg, group, col)
        Wq_u, s_u = convrot_quantize_weight(Wu, group, col)
        self.Wq_gu = convrot_interleave_gate_up(Wq_g, Wq_u)
        s_gu = convrot_interleave_gate_up(s_g, s_u)
        smooth_d = None
        if x_calib is not None:
            Xq, s_tok = convrot_rotate_quant_act(x_calib, group, self.norm_w, eps)
            h = convrot_int8_linear_swiglu(Xq, s_tok, self.Wq_gu, s_gu, workspace=self.workspace)
            smooth_d, _ = convrot_smoothquant_calibrate(h, None, Wd, eps, alpha)
            convrot_fold_row_scales(s_u, smooth_d)
            s_gu = convrot_interleave_gate_up(s_g, s_u)
        self.s_gu = s_gu
        self.Wq_d, self.s_d = convrot_quantize_weight(Wd, group, smooth_d)

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        Xq, s_tok = convrot_rotate_quant_act(x, self.group, self.norm_w, self.eps)
        h = convrot_int8_linear_swiglu(Xq, s_tok, self.Wq_gu, self.s_gu, workspace=self.workspace)
        Hq, s_h = convrot_rotate_quant_act(h, self.group, None, self.eps)
        return convrot_int8_linear(Hq, s_h, self.Wq_d, self.s_d, out, self.workspace)

    __call__ = forward


def rope_table(rows: int, dim: int, theta: float = 1e6, device=None) -> torch.Tensor:
    """fp32 [rows, dim]: cosines, then sines, of position * theta^(-2 i / dim),
    the angles taken in fp64 (an fp32 angle is off by 2^-24 of itself, which at
    position 10^6 is 0.06 of a radian)."""
    freq = theta ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=device) / dim)
    angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


# A slot past every cache.
NO_PLACE = 1 << 62


class PagedKVCache:
    """One layer's keys and values in pages of page_size tokens: bf16, or int8
    with one fp32 scale per token and head.  Which sequence owns which page is
    the caller's block table (int32 [sequences, pages per sequence])."""

    def __init__(self, pages: int, kv_heads: int, head_dim: int, *, page_size: int = 64, int8: bool = False,
                 device=None):
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
        shape = (pages, kv_heads, page_size, head_dim)
        self.page_size = page_size
        self.k, self.v = (torch.zeros(shape, dtype=torch.int8 if int8 else torch.bfloat16, device=dev) for _ in range(2))
        self.k_scale, self.v_scale = ((torch.zeros(shape[:3], device=dev) for _ in range(2)) if int8 else (None, None))

    def slots(self, block_table: torch.Tensor, sequence: torch.Tensor, position: torch.Tensor) -> torch.Tensor:
        """Slots (int64) of tokens at `position` of rows `sequence` of the block
        table.  A token that is not to be stored has a negative slot: its page is
        not there (negative), or its sequence or position is negative (padding).
        One that the table has no place for has a slot past every cache, which
        convrot_rope_append leaves out and reports."""
        rows, cols = block_table.shape
        sequence, position = sequence.long(), position.long()
        column = position // self.page_size
        slot = torch.full_like(position, NO_PLACE)
        if rows and cols:
            page = block_table[sequence.clamp(0, rows - 1), column.clamp(0, cols - 1)].long()
            slot = torch.where((sequence < rows) & (column < cols), page * self.page_size + position % self.page_size, slot)
        return torch.where((sequence < 0) | (position < 0), -1, slot)


class ConvRotAttention:
    """The attention block of the quantised decoder layer: one fused q/k/v
    projection (behind the fused RMSNorm), position rotation and append to a
    paged cache, attention, o projection.  Beside ConvRotMLP it completes the
    layer; the four projections are the ones the model cards quantise.

    rope is a rope_table (or any table of that form); q_norm and k_norm are the
    per-head RMSNorm weights (applied as 1 + w) of models that have them.
    """

    def __init__(self, Wq: torch.Tensor, Wk: torch.Tensor, Wv: torch.Tensor, Wo: torch.Tensor, *, q_heads: int,
                 kv_heads: int, rope: torch.Tensor, weight_bits: int = 8, group: int = 256,
                 norm_w: Optional[torch.Tensor] = None, q_norm: Optional[torch.Tensor] = None,
                 k_norm: Optional[torch.Tensor] = None, x_calib: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 scale: Optional[float] = None):
        if Wq.shape[0] % q_heads or q_heads % kv_heads:
            raise ValueError("q_heads must divide the rows of Wq and be a multiple of kv_heads")
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, Wq.shape[0] // q_heads
        if Wk.shape[0] != kv_heads * self.head_dim or Wv.shape[0] != kv_heads * self.head_dim:
            raise ValueError(f"Wk and Wv must have {kv_heads} x {self.head_dim} rows")
        if Wo.shape[1] != Wq.shape[0]:
            raise ValueError("Wo must have as many columns as Wq has rows")
        self.rope, self.q_norm, self.k_norm, self.eps, self.scale = rope, q_norm, k_norm, eps, scale
        self.qkv = ConvRotFusedLinear([Wq, Wk, Wv], weight_bits=weight_bits, group=group, norm_w=norm_w,
                                      x_calib=x_calib, eps=eps)
        self.o = ConvRotLinear(Wo, weight_bits=weight_bits, group=group, eps=eps)

    def _append(self, x, positions, slots, cache: PagedKVCache, rotated_k: bool):
        q, k, v = (t.unflatten(1, (-1, self.head_dim)) for t in self.qkv(x))
        convrot_rope_append(q, k, v, self.rope, positions, slots, cache.k, cache.v, k_scale=cache.k_scale,
                            v_scale=cache.v_scale, q_norm=self.q_norm, k_norm=self.k_norm, eps=self.eps, q_out=q,
                            k_out=k if rotated_k else None)
        return q, k, v

    def prompt(self, x: torch.Tensor, cu_seqlens: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
               cache: PagedKVCache) -> torch.Tensor:
        """Whole prompts, packed one after another: x bf16 [tokens, hidden].  A token
        sees the tokens of its prompt in this call, not what the cache held
        before.  Rows behind the last prompt (padding) hold nothing of use."""
        q, k, v = self._append(x, positions, slots, cache, True)
        return self.o(convrot_attention_prompt(q, k, v, cu_seqlens, scale=self.scale).flatten(1))

    def decode(self, x: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor, cache: PagedKVCache,
               block_table: torch.Tensor, seq_lens: torch.Tensor) -> torch.Tensor:
        """One new token per sequence: x bf16 [sequences, hidden]; seq_lens counts it."""
        q, _, _ = self._append(x, positions, slots, cache, False)
        o = convrot_attention_decode(q, cache.k, cache.v, block_table, seq_lens, k_scale=cache.k_scale,
                                     v_scale=cache.v_scale, scale=self.scale)
        return self.o(o.flatten(1))
