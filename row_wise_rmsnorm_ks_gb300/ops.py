"""Tensor-level API over the C ABI, with Kernscope's signatures ("API contract"):

    rms_norm(x, weight, eps=1e-6) -> y
    fused_add_rms_norm(x, residual, weight, eps=1e-6) -> None   (x and residual updated in place)
    gated_add_rms_norm(x, residual, weight, *, post_weight, gate, ...) -> None   (the same, with a norm
                                                         of x before it, a gate and scales)

    rms_norm_host(x, weight, eps=1e-6, *, out=None, workspace=None) -> out
    fused_add_rms_norm_host(x, residual, weight, eps=1e-6, *, workspace=None) -> None
(the last two take rows in host memory: without a workspace the kernels read and write pinned
host rows directly over the host link; with a device workspace the library copies them through
it in overlapping chunks).

Checks follow Kernscope "API contract / Inputs": x is (..., hidden) with a non-empty last
dimension, weight is (hidden,), tensors are contiguous CUDA tensors of one dtype (fp16, bf16 or
fp32) on one device, eps is finite and positive, the fused op's residual has x's shape and the
storage of x, residual and weight does not overlap; tensors that require grad are rejected
(inference only). The leading dimensions are flattened into rows. Every launch goes through
libks on the tensor's device and the current torch stream; nothing is computed here.
"""
from __future__ import annotations

import math

import torch

from . import _abi

_DTYPES = {torch.float32: _abi.KS_DTYPE_F32, torch.float16: _abi.KS_DTYPE_F16,
           torch.bfloat16: _abi.KS_DTYPE_BF16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # torch without CUDA has none, nor CUDA tensors
_current_device = torch.cuda.current_device
_grad = torch.is_grad_enabled
_BIG = 2.0 ** 127  # what a scale may be: finite in 32 bits, times log2(e) too


def _launch(call, args: bytes, device: torch.device) -> None:
    index = device.index
    if _current_device() == index:
        status = call(args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = call(args, _raw_stream(index))
    if status:
        _abi.check(status)


def _check(x: torch.Tensor, weight: torch.Tensor, eps: float, names=("x", "weight")):
    if not isinstance(x, torch.Tensor) or not isinstance(weight, torch.Tensor):
        raise TypeError("x and weight must be torch tensors")
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}; use float16, bfloat16 or float32")
    if weight.dtype != x.dtype:
        raise TypeError(f"{names[1]} dtype {weight.dtype} differs from {names[0]} dtype {x.dtype}")
    if x.device.type != "cuda" or weight.device != x.device:
        raise ValueError("tensors must be CUDA tensors on one device (there is no CPU path)")
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("the last dimension of x must be non-empty")
    if weight.dim() != 1 or weight.shape[0] != x.shape[-1]:
        raise ValueError(f"weight must have shape ({x.shape[-1]},), got {tuple(weight.shape)}")
    if not x.is_contiguous() or not weight.is_contiguous():
        raise ValueError("tensors must be contiguous")
    if torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad):
        raise RuntimeError("these kernels are inference-only: inputs must not require grad")
    if not (isinstance(eps, (int, float)) and math.isfinite(eps) and eps > 0):
        raise ValueError("eps must be finite and positive")


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, *,
             out: torch.Tensor | None = None) -> torch.Tensor:
    """y = cast(fp32(x) * rsqrt(mean(fp32(x)^2) + eps) * fp32(weight)) per row. `out` may be x
    itself (in place) or a new contiguous tensor of x's shape and dtype."""
    _check(x, weight, eps)
    if out is None:
        out = torch.empty_like(x)
    elif (out.shape != x.shape or out.dtype != x.dtype or out.device != x.device
          or not out.is_contiguous()):
        raise ValueError("out must be a contiguous tensor with x's shape, dtype and device")
    hidden = x.shape[-1]
    rows = x.numel() // hidden
    with torch.cuda.device(x.device):
        _abi.check(_abi.ks_rms_norm(out.data_ptr(), x.data_ptr(), weight.data_ptr(), rows, hidden,
                                    float(eps), _DTYPES[x.dtype], _stream(x.device)))
    return out


def fused_add_rms_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor,
                       eps: float = 1e-6) -> None:
    """In place: residual <- cast(fp32(x) + fp32(residual)); x <- RMSNorm of the FP32 sum
    times fp32(weight). Returns None."""
    _check(x, weight, eps)
    if not isinstance(residual, torch.Tensor) or residual.shape != x.shape:
        raise ValueError("residual must have the same shape as x")
    if residual.dtype != x.dtype or residual.device != x.device or not residual.is_contiguous():
        raise ValueError("residual must be contiguous, with x's dtype and device")
    if torch.is_grad_enabled() and residual.requires_grad:
        raise RuntimeError("these kernels are inference-only: inputs must not require grad")
    hidden = x.shape[-1]
    rows = x.numel() // hidden
    with torch.cuda.device(x.device):
        _abi.check(_abi.ks_fused_add_rms_norm(x.data_ptr(), residual.data_ptr(),
                                              weight.data_ptr(), rows, hidden, float(eps),
                                              _DTYPES[x.dtype], _stream(x.device)))
    return None


def _gate_rows(gate: torch.Tensor, x: torch.Tensor):
    """(rows that share a row of the gate, its row stride, its column stride)."""
    if gate.__class__ is torch.Tensor and gate.shape == x.shape[-1:] and gate.dtype is x.dtype \
            and gate.device == x.device and gate.is_contiguous() and not gate.requires_grad:
        return x.numel() // x.shape[-1], 0, 1  # one for all rows
    if not isinstance(gate, torch.Tensor) or gate.dtype != x.dtype:
        raise TypeError(f"gate must be a tensor of {x.dtype}")
    if gate.device != x.device or not gate.is_contiguous():
        raise ValueError("gate must be contiguous, on x's device")
    if torch.is_grad_enabled() and gate.requires_grad:
        raise RuntimeError("these kernels are inference-only: inputs must not require grad")
    hidden, lead = x.shape[-1], x.shape[:-1]
    shape = (1,) * (x.dim() - gate.dim()) + tuple(gate.shape)
    own = len(lead)  # leading dimensions that the gate has of its own: those up to its last that is not 1
    while own > 0 and shape[own - 1] == 1:
        own -= 1
    if len(shape) != x.dim() or shape[-1] not in (1, hidden) or shape[:own] != tuple(lead[:own]):
        raise ValueError(f"gate must have x's leading dimensions up to some point and ones behind it, and a last "
                         f"dimension of {hidden} or 1; got {tuple(gate.shape)} for {tuple(x.shape)}")
    return math.prod(lead[own:]), shape[-1], 1 if shape[-1] == hidden else 0


def gated_add_rms_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor, *,
                       post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                       residual_scale: float = 1.0, block_scale: float = 1.0, eps: float = 1e-6) -> None:
    """What lies between two blocks that norm their outputs too, in place, per row and in FP32:

        n = x * rsqrt(mean(x^2) + eps) * post_weight       (x itself without post_weight)
        s = residual_scale * residual + block_scale * gate * n
        residual <- cast(s);  x <- cast(s * rsqrt(mean(s^2) + eps) * weight)

    x is the block's output and becomes the next block's input. gate: (hidden,) for one vector, x's leading
    dimensions up to some point and ones behind it for one per sequence or token ((B, 1, hidden) for an x of
    (B, S, hidden)); a last dimension of 1 is one value for a row. weight and post_weight are (hidden,); all
    tensors have x's dtype. Returns None."""
    try:  # what a call mostly is, in one go; anything else is looked at point by point
        dt, dev, shape, code = x.dtype, x.device, x.shape, _DTYPES[x.dtype]
        row = shape[-1:]
        fine = (x.is_cuda and row[0] > 0 and residual.shape == shape and weight.shape == row and residual.dtype is dt
                and weight.dtype is dt and residual.device == dev and weight.device == dev and x.is_contiguous()
                and residual.is_contiguous() and weight.is_contiguous() and 0.0 < eps < math.inf
                and (post_weight is None or (post_weight.shape == row and post_weight.dtype is dt
                                             and post_weight.device == dev and post_weight.is_contiguous()
                                             and not post_weight.requires_grad))
                and eps.__class__ is residual_scale.__class__ is block_scale.__class__ is float
                and -_BIG < residual_scale < _BIG and -_BIG < block_scale < _BIG
                and not (x.requires_grad or residual.requires_grad or weight.requires_grad))
    except (AttributeError, KeyError, ValueError, TypeError, IndexError):
        fine = False
    if not fine:
        _check_gated(x, residual, weight, post_weight, residual_scale, block_scale, eps)
        dt, dev, shape, code = x.dtype, x.device, x.shape, _DTYPES[x.dtype]
    gate_p, per_gate, row_stride, column_stride = 0, 1, 0, 0
    if gate is not None:
        per_gate, row_stride, column_stride = _gate_rows(gate, x)
        gate_p = gate.data_ptr()
    hidden = shape[-1]
    rows = x.numel() // hidden
    if rows == 0:
        return None
    _launch(_abi.ks_gated_add_rms_norm, _abi.GATED_NORM_ARGS.pack(
        x.data_ptr(), residual.data_ptr(), weight.data_ptr(), post_weight.data_ptr() if post_weight is not None else 0,
        gate_p, rows, hidden, per_gate, row_stride, column_stride, eps, residual_scale, block_scale, code), dev)
    return None


def _check_gated(x, residual, weight, post_weight, residual_scale, block_scale, eps):
    _check(x, weight, eps)
    if not isinstance(residual, torch.Tensor) or residual.shape != x.shape:
        raise ValueError("residual must have the same shape as x")
    if residual.dtype != x.dtype or residual.device != x.device or not residual.is_contiguous():
        raise ValueError("residual must be contiguous, with x's dtype and device")
    if post_weight is not None:
        _check(x, post_weight, eps, names=("x", "post_weight"))
    if torch.is_grad_enabled() and residual.requires_grad:
        raise RuntimeError("these kernels are inference-only: inputs must not require grad")
    for v, n in ((residual_scale, "residual_scale"), (block_scale, "block_scale")):
        if not (isinstance(v, (int, float)) and abs(v) < _BIG):
            raise ValueError(f"{n} must be finite (below 2^127)")


def _check_host(x: torch.Tensor, weight: torch.Tensor, workspace: torch.Tensor, eps: float):
    if not isinstance(x, torch.Tensor) or x.device.type != "cpu":
        raise ValueError("x must be a CPU tensor (pin it for the copies to overlap)")
    if x.dtype not in _DTYPES or weight.dtype != x.dtype:
        raise TypeError("x and weight must share a dtype: float16, bfloat16 or float32")
    if weight.device.type != "cuda" or weight.dim() != 1 or weight.shape[0] != x.shape[-1]:
        raise ValueError("weight must be a CUDA tensor of shape (hidden,)")
    if workspace is not None and (not isinstance(workspace, torch.Tensor)
                                  or workspace.device != weight.device
                                  or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor on weight's device")
    if workspace is None and not x.is_pinned():
        raise ValueError("without a workspace the host rows must be pinned")
    if not (x.is_contiguous() and weight.is_contiguous()):
        raise ValueError("tensors must be contiguous")
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("the last dimension of x must be non-empty")
    if not (isinstance(eps, (int, float)) and math.isfinite(eps) and eps > 0):
        raise ValueError("eps must be finite and positive")


def _ws(workspace):
    if workspace is None:
        return None, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def rms_norm_host(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, *,
                  workspace: torch.Tensor | None = None,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """RMSNorm of host rows through the device: returns `out` (a host tensor, x's shape; may be
    x). Ordered on the current stream of weight's device; synchronise it before reading `out`."""
    _check_host(x, weight, workspace, eps)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, pin_memory=x.is_pinned())
    elif out.shape != x.shape or out.dtype != x.dtype or out.device.type != "cpu":
        raise ValueError("out must be a CPU tensor with x's shape and dtype")
    hidden = x.shape[-1]
    rows = x.numel() // hidden
    with torch.cuda.device(weight.device):
        _abi.check(_abi.ks_rms_norm_host(out.data_ptr(), x.data_ptr(), weight.data_ptr(), rows,
                                         hidden, float(eps), _DTYPES[x.dtype], *_ws(workspace),
                                         _stream(weight.device)))
    return out


def fused_add_rms_norm_host(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor,
                            eps: float = 1e-6, *, workspace: torch.Tensor | None = None) -> None:
    """Fused residual-add RMSNorm of host rows through the device, in place on both host
    tensors. Ordered on the current stream of weight's device; synchronise before reading."""
    _check_host(x, weight, workspace, eps)
    if (not isinstance(residual, torch.Tensor) or residual.shape != x.shape
            or residual.dtype != x.dtype or residual.device.type != "cpu"
            or not residual.is_contiguous()):
        raise ValueError("residual must be a contiguous CPU tensor with x's shape and dtype")
    hidden = x.shape[-1]
    rows = x.numel() // hidden
    with torch.cuda.device(weight.device):
        _abi.check(_abi.ks_fused_add_rms_norm_host(x.data_ptr(), residual.data_ptr(),
                                                   weight.data_ptr(), rows, hidden, float(eps),
                                                   _DTYPES[x.dtype], *_ws(workspace),
                                                   _stream(weight.device)))
    return None


# ------------------------------------------------------------------ the next operators

def _check_plain(x: torch.Tensor, name="x"):
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
        raise TypeError(f"{name} must be a float16, bfloat16 or float32 tensor")
    if x.device.type != "cuda":
        raise ValueError("tensors must be CUDA tensors (there is no CPU path)")
    if not x.is_contiguous():
        raise ValueError("tensors must be contiguous")
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("the last dimension must be non-empty")
    if torch.is_grad_enabled() and x.requires_grad:
        raise RuntimeError("these kernels are inference-only: inputs must not require grad")


def silu_and_mul(x: torch.Tensor) -> torch.Tensor:
    """SwiGLU (Kernscope, "Numerical contract / SwiGLU activation"): x of shape (..., 2D) gives
    cast(gate * sigmoid(gate) * up) of shape (..., D), gate = x[..., :D], up = x[..., D:], FP32
    throughout. x is read-only; D may be odd; leading dimensions may be empty."""
    _check_plain(x)
    if x.shape[-1] % 2:
        raise ValueError("the last dimension of x must be even")
    d = x.shape[-1] // 2
    out = torch.empty(tuple(x.shape[:-1]) + (d,), dtype=x.dtype, device=x.device)
    rows = x.numel() // x.shape[-1]
    with torch.cuda.device(x.device):
        _abi.check(_abi.ks_silu_and_mul(out.data_ptr(), x.data_ptr(), rows, d, _DTYPES[x.dtype],
                                        _stream(x.device)))
    return out


def softmax(x: torch.Tensor, *, out: torch.Tensor | None = None) -> torch.Tensor:
    """Softmax over the last dimension (Kernscope, "Numerical contract / Softmax"), FP32
    max/exp/sum/divide, cast back; rows with NaN or +inf, or all -inf, come out NaN."""
    _check_plain(x)
    if out is None:
        out = torch.empty_like(x)
    elif out.shape != x.shape or out.dtype != x.dtype or out.device != x.device:
        raise ValueError("out must match x in shape, dtype and device")
    hidden = x.shape[-1]
    with torch.cuda.device(x.device):
        _abi.check(_abi.ks_softmax(out.data_ptr(), x.data_ptr(), x.numel() // hidden, hidden,
                                   _DTYPES[x.dtype], _stream(x.device)))
    return out


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, eps: float = 1e-5, *,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """LayerNorm over the last dimension with FP32 steps:
    cast((((x - mean) * rsqrt(var + eps)) * weight) + bias); weight and bias optional."""
    _check_plain(x)
    hidden = x.shape[-1]
    for t, n in ((weight, "weight"), (bias, "bias")):
        if t is not None and (t.dtype != x.dtype or t.device != x.device or t.dim() != 1
                              or t.shape[0] != hidden or not t.is_contiguous()):
            raise ValueError(f"{n} must be a contiguous ({hidden},) tensor of x's dtype and device")
    if not (isinstance(eps, (int, float)) and math.isfinite(eps) and eps > 0):
        raise ValueError("eps must be finite and positive")
    if out is None:
        out = torch.empty_like(x)
    with torch.cuda.device(x.device):
        _abi.check(_abi.ks_layer_norm(out.data_ptr(), x.data_ptr(),
                                      weight.data_ptr() if weight is not None else None,
                                      bias.data_ptr() if bias is not None else None,
                                      x.numel() // hidden, hidden, float(eps), _DTYPES[x.dtype],
                                      _stream(x.device)))
    return out
