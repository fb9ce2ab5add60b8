"""The operators around the expert forward (include/moe.h): the norms before and after a
block with its gate and scaled residual, and their gradients; a whole mixture-of-experts layer
for a few tokens; the linear layer on microscaled 4-bit weights.

Argument marshalling only, as in _abi.py, but in a compiled module (_moe_torch): at decoding
sizes a call is its time on the host.  Tensors that a call makes for its caller are allocated on
the stream it runs on, on the inputs' device; every tensor of a call has to be on that one device.
"""

from __future__ import annotations

import contextlib
import ctypes

import torch

from ._abi import MOE_BF16, MOE_E2M1X2, MOE_F32, MOE_I32, MOE_I64, MoeW13, _TENSOR, _check, load

GATE_ACTS = {"none": 0, "sigmoid": 1, "tanh": 2}
SCALE_E8M0_32, SCALE_E4M3_16 = 0, 1

_DT = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32, torch.int32: MOE_I32, torch.int64: MOE_I64}


# For calls of the C entry points through load(), such as the tests of their status codes; the functions
# below go through the compiled module, which fills its own.

def _desc(t: torch.Tensor | None):
    """The bytes of a moe_tensor_t (None stays NULL); unknown dtypes are rejected by the library."""
    if t is None:
        return None
    n, z, s = t.dim(), t.shape, t.stride()
    dt = _DT.get(t.dtype, 99)
    if n == 2:
        return _TENSOR(t.data_ptr(), dt, 2, z[0], z[1], 0, 0, s[0], s[1], 0, 0, 0, 0, 0, 0, 0)
    if n == 1:
        return _TENSOR(t.data_ptr(), dt, 1, z[0], 0, 0, 0, s[0], 0, 0, 0, 0, 0, 0, 0, 0)
    if n > 4:
        raise ValueError(f"a tensor of {n} dimensions")
    pad = (0, 0, 0, 0)[n:]
    return _TENSOR(t.data_ptr(), dt, n, *z, *pad, *s, *pad, 0, 0, 0, 0, 0)


def _codes_desc(codes: torch.Tensor, scale: torch.Tensor):
    """The bytes of a MOE_E2M1X2 matrix: two codes a byte, scales of one byte."""
    z, s, q = codes.shape, codes.stride(), scale.stride()
    return _TENSOR(codes.data_ptr(), MOE_E2M1X2, 2, z[0], 2 * z[1], 0, 0, s[0], s[1], 0, 0, scale.data_ptr(),
                   q[0], q[1], 0, 0)


_module = None


def _ops():
    """The compiled module; the library behind it is loaded (or reported missing) first."""
    global _module
    if _module is None:
        load()
        try:
            from . import _moe_torch
        except ImportError as e:
            raise RuntimeError(f"the binding was not built: run python -m {__package__}.build") from e
        _moe_torch.set_check(_check)
        _module = _moe_torch
    return _module


@contextlib.contextmanager
def _on(stream, tensor):
    """Makes `stream` (a torch stream, or a raw handle on the tensor's device) the current one."""
    device = tensor.device
    if device.type != "cuda":
        raise ValueError(f"a tensor on {device}: the operators run on a CUDA device only")
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"a stream of {stream.device} for tensors on {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _act(name: str) -> int:
    if name not in GATE_ACTS:
        raise ValueError(f"gate_act {name!r}: one of {', '.join(GATE_ACTS)}")
    return GATE_ACTS[name]


def norm_before(x, weight=None, *, eps=1e-6, out=None, out_dtype=None, rstd=None, stream=None):
    """(out, rstd): out[t] = x[t] * rstd[t] * weight, rstd[t] = 1 / sqrt(mean(x[t]^2) + eps).

    x [T, H] bf16 or f32, any strides; out in out_dtype (x's by default)."""
    f = (_module or _ops()).norm_before
    if stream is None:
        return f(x, weight, eps, out, out_dtype, rstd)
    with _on(stream, x):
        return f(x, weight, eps, out, out_dtype, rstd)


def norm_after(y, residual=None, weight=None, gate=None, *, gate_act="none", normalize=True, residual_scale=1.0,
               eps=1e-6, out=None, out_dtype=None, rstd=None, next_norm=None, next_weight=None, next_out=None,
               next_dtype=None, next_rstd=None, stream=None):
    """out = residual_scale * residual + a(gate) * y * rstd * weight, and with a next norm
    (next_norm=True, or next_weight, next_out or next_rstd given) that sum's own norm in the same pass.

    Returns (out, rstd), or (out, rstd, next_out, next_rstd) with a next norm.  gate is
    [T or 1, H or 1]; out takes the residual's dtype (y's without one) and next_out out's,
    unless out_dtype / next_dtype say otherwise.  With normalize=False the norm of y is left
    out and rstd is ones."""
    f = (_module or _ops()).norm_after
    args = (y, residual, weight, gate, _act(gate_act), 1 if normalize else 0, residual_scale, eps, out, out_dtype,
            rstd, next_norm, next_weight, next_out, next_dtype, next_rstd)
    if stream is None:
        return f(*args)
    with _on(stream, y):
        return f(*args)


def norm_backward_workspace_bytes(T: int, H: int) -> int:
    return int(load().moe_norm_backward_workspace_bytes(T, H))


def norm_before_backward(dout, x, rstd, weight=None, *, residual_grad=None, residual_scale=1.0, dx=None,
                         dweight=None, weight_grad=True, grad_dtype=torch.float32, workspace=None, stream=None):
    """(dx, dweight): the gradient of norm_before given dout, plus residual_scale *
    residual_grad, the gradient that reaches x past the block.  dweight (in grad_dtype) is None
    without a weight or with weight_grad=False."""
    f = (_module or _ops()).norm_before_backward
    args = (dout, x, rstd, weight, residual_grad, residual_scale, dx, dweight, weight_grad, grad_dtype, workspace)
    if stream is None:
        return f(*args)
    with _on(stream, dout):
        return f(*args)


def norm_after_backward(dout, y, rstd, weight=None, gate=None, *, gate_act="none", normalize=True, dy=None,
                        dweight=None, dgate=None, weight_grad=True, gate_grad=True, grad_dtype=torch.float32,
                        workspace=None, stream=None):
    """(dy, dweight, dgate): the gradient of norm_after given dout, rstd as the forward wrote it.
    dweight and dgate (in grad_dtype; dgate of the gate's shape, summed over its axes of size
    1) are None without a weight or a gate, or with weight_grad / gate_grad False.  The gradient
    with respect to the residual is residual_scale * dout (norm_before_backward adds it)."""
    f = (_module or _ops()).norm_after_backward
    args = (dout, y, rstd, weight, gate, _act(gate_act), 1 if normalize else 0, dy, dweight, dgate, weight_grad,
            gate_grad, grad_dtype, workspace)
    if stream is None:
        return f(*args)
    with _on(stream, dout):
        return f(*args)


def layer_decode_workspace_bytes(T: int, H: int, I: int, E: int, k: int, mxfp4: bool = False) -> int:
    """E and k with the shared expert counted in."""
    return int(load().moe_layer_decode_workspace_bytes(T, H, I, E, k, MOE_E2M1X2 if mxfp4 else MOE_BF16))


def layer_decode(x, router, w13: MoeW13, w2, k: int, *, w2_scale=None, pre_weight=None, eps=1e-6, renormalize=True,
                 shared_expert=False, post_norm=False, post_weight=None, gate=None, gate_act="none",
                 residual_scale=1.0, out=None, topk_ids=None, topk_weights=None, workspace=None, stream=None):
    """(out, topk_ids, topk_weights) of a whole mixture-of-experts layer on x [T, H] bf16, T <= 32:
    norm, router [E, H], the k experts of largest softmax (and the shared expert E with weight 1),
    their SwiGLU sum, and residual_scale * x + a(gate) * that sum (normed with post_norm).

    w13 from w13_from_packed / w13_from_views, on x's device."""
    f = (_module or _ops()).layer_decode
    args = (x, router, ctypes.addressof(w13), w2, w2_scale, k, pre_weight, eps, 1 if renormalize else 0,
            1 if shared_expert else 0, 1 if post_norm else 0, post_weight, gate, _act(gate_act), residual_scale, out,
            topk_ids, topk_weights, workspace)
    if stream is None:
        return f(*args)
    with _on(stream, x):
        return f(*args)


def quantize_nvfp4(src, global_scale=None, *, stream=None):
    """(codes uint8 [R, K/2], scales float8_e4m3fn [R, K/16], global_scale f32 [1]) of src [R, K]
    (bf16 or f32, K a multiple of 32): e2m1 codes, an e4m3 scale per 16, one float scale for the
    tensor.  Without a given global_scale it is amax / 2688, by torch: |src| written out and read back,
    which costs more than the quantisation itself; keep the scale where src's range is known."""
    with contextlib.nullcontext() if stream is None else _on(stream, src):
        if global_scale is None:
            top = src.abs().amax().float() if src.numel() else torch.zeros((), device=src.device)
            global_scale = (top / 2688.0).reshape(1)
        codes, scales = (_module or _ops()).quantize_nvfp4(src, global_scale)
    return codes, scales, global_scale


def linear_fp4_workspace_bytes(T: int, N: int, K: int, scale_format: int) -> int:
    return int(load().moe_linear_fp4_workspace_bytes(T, N, K, scale_format))


def linear_fp4(x, weight, weight_scale, *, x_global=None, w_global=None, out=None, workspace=None, stream=None):
    """out [T, N] bf16 = x [T, K] (bf16 or f32, quantised on the way in) times the transposed 4-bit
    weight [N, K]: codes uint8 [N, K/2] and, either e4m3 scales [N, K/16] (quantize_nvfp4; x_global
    the float scale of x, w_global the weight's) or e8m0 scales [N, K/32] (quantize_mxfp4)."""
    f = (_module or _ops()).linear_fp4
    if stream is None:
        return f(x, weight, weight_scale, x_global, w_global, out, workspace)
    with _on(stream, x):
        return f(x, weight, weight_scale, x_global, w_global, out, workspace)
