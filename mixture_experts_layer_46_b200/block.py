"""The operators around the expert forward (include/moe.h): the norms before and after a
block with its gate and scaled residual, and their gradients; a whole mixture-of-experts layer
for a few tokens; the linear layer on microscaled 4-bit weights.

Argument marshalling only, as in _abi.py.  Tensors that a call makes for its caller are
allocated on the stream it runs on, on the inputs' device; every tensor of a call has to be on
that one device.
"""

from __future__ import annotations

import contextlib
import ctypes
import struct

import torch

from ._abi import MOE_BF16, MOE_E2M1X2, MOE_F32, MOE_I32, MOE_I64, MoeW13, _check, load

GATE_ACTS = {"none": 0, "sigmoid": 1, "tanh": 2}

_DT = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32, torch.int32: MOE_I32, torch.int64: MOE_I64}
# moe_tensor_t: data, dtype, ndim, sizes[4], strides[4], scale, scale_strides[4]
_TENSOR = struct.Struct("=Qii4q4qQ4q").pack


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


def _experts_desc(codes: torch.Tensor, scale: torch.Tensor):
    """The bytes of a MOE_E2M1X2 weight of all experts [E, rows, 2 * bytes]."""
    z, s, q = codes.shape, codes.stride(), scale.stride()
    return _TENSOR(codes.data_ptr(), MOE_E2M1X2, 3, z[0], z[1], 2 * z[2], 0, s[0], s[1], s[2], 0, scale.data_ptr(),
                   q[0], q[1], q[2], 0)


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


class _Call:
    """The device and stream of a call: checks that the tensors share one CUDA device, makes it
    current and, with a stream of its own, makes that the stream new tensors belong to."""

    __slots__ = ("device", "stream", "_stack")

    def __init__(self, stream, first, *others):
        index = first.get_device()  # -1: host memory
        for t in others:
            if t is not None and t.get_device() != index:
                raise ValueError(f"tensors on {first.device} and on {t.device}")
        if index < 0:
            raise ValueError(f"a tensor on {first.device}: the operators run on a CUDA device only")
        self.device, self._stack = first.device, None
        if stream is None and index == torch.cuda.current_device():
            self.stream = _raw_stream(index)
            return
        if isinstance(stream, int):
            stream = (torch.cuda.ExternalStream(stream, device=self.device) if stream
                      else torch.cuda.default_stream(self.device))
        if stream is not None and stream.device != self.device:
            raise ValueError(f"a stream of {stream.device} for tensors on {self.device}")
        self._stack = contextlib.ExitStack()
        self._stack.enter_context(torch.cuda.device(self.device))
        if stream is not None:
            self._stack.enter_context(torch.cuda.stream(stream))
        self.stream = _raw_stream(index)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        if self._stack is not None:
            self._stack.close()
        return False

    def empty(self, *shape, dtype):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def workspace(self, given, need):
        if given is None:
            return torch.empty(max(need, 1), dtype=torch.uint8, device=self.device)
        return given


def _act(name: str) -> int:
    if name not in GATE_ACTS:
        raise ValueError(f"gate_act {name!r}: one of {', '.join(GATE_ACTS)}")
    return GATE_ACTS[name]


def _rows(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} has {t.dim()} dimensions, not 2")
    return t.shape


def norm_before(x, weight=None, *, eps=1e-6, out=None, out_dtype=None, rstd=None, stream=None):
    """(out, rstd): out[t] = x[t] * rstd[t] * weight, rstd[t] = 1 / sqrt(mean(x[t]^2) + eps).

    x [T, H] bf16 or f32, any strides; out in out_dtype (x's by default)."""
    T, H = _rows(x, "x")
    with _Call(stream, x, weight, out, rstd) as c:
        if out is None:
            out = c.empty(T, H, dtype=out_dtype or x.dtype)
        if rstd is None:
            rstd = c.empty(T, dtype=torch.float32)
        _check(load().moe_norm_before(_desc(x), _desc(weight), eps, _desc(out), _desc(rstd), c.stream),
               "moe_norm_before")
    return out, rstd


def norm_after(y, residual=None, weight=None, gate=None, *, gate_act="none", normalize=True, residual_scale=1.0,
               eps=1e-6, out=None, out_dtype=None, rstd=None, next_norm=None, next_weight=None, next_out=None,
               next_dtype=None, next_rstd=None, stream=None):
    """out = residual_scale * residual + a(gate) * y * rstd * weight, and with a next norm
    (next_norm=True, or next_weight or next_out given) that sum's own norm in the same pass.

    Returns (out, rstd), or (out, rstd, next_out, next_rstd) with a next norm.  gate is
    [T or 1, H or 1]; out takes the residual's dtype (y's without one) and next_out out's,
    unless out_dtype / next_dtype say otherwise.  With normalize=False the norm of y is left
    out and rstd is ones."""
    T, H = _rows(y, "y")
    act = _act(gate_act)
    if next_norm is None:
        next_norm = next_weight is not None or next_out is not None or next_rstd is not None
    with _Call(stream, y, residual, weight, gate, out, rstd, next_weight, next_out, next_rstd) as c:
        if out is None:
            out = c.empty(T, H, dtype=out_dtype or (y if residual is None else residual).dtype)
        if rstd is None:
            rstd = c.empty(T, dtype=torch.float32)
        if next_norm and next_out is None:
            next_out = c.empty(T, H, dtype=next_dtype or out.dtype)
        if next_norm and next_rstd is None:
            next_rstd = c.empty(T, dtype=torch.float32)
        _check(load().moe_norm_after(_desc(y), _desc(residual), _desc(weight), _desc(gate), act,
                                     1 if normalize else 0, residual_scale, eps, _desc(out), _desc(rstd),
                                     _desc(next_weight), _desc(next_out), _desc(next_rstd), c.stream),
               "moe_norm_after")
    return (out, rstd, next_out, next_rstd) if next_norm else (out, rstd)


def norm_backward_workspace_bytes(T: int, H: int) -> int:
    return int(load().moe_norm_backward_workspace_bytes(T, H))


def norm_before_backward(dout, x, rstd, weight=None, *, residual_grad=None, residual_scale=1.0, dx=None,
                         dweight=None, weight_grad=True, grad_dtype=torch.float32, workspace=None, stream=None):
    """(dx, dweight): the gradient of norm_before given dout, plus residual_scale *
    residual_grad, the gradient that reaches x past the block.  dweight (in grad_dtype) is None
    without a weight or with weight_grad=False."""
    T, H = _rows(dout, "dout")
    want = dweight is not None or (weight is not None and weight_grad)
    with _Call(stream, dout, x, rstd, weight, residual_grad, dx, dweight, workspace) as c:
        if dx is None:
            dx = c.empty(T, H, dtype=x.dtype)
        if want and dweight is None:
            dweight = c.empty(H, dtype=grad_dtype)
        ws = c.workspace(workspace, norm_backward_workspace_bytes(T, H)) if want else None
        _check(load().moe_norm_before_backward(
            _desc(dout), _desc(x), _desc(rstd), _desc(weight), _desc(residual_grad), residual_scale, _desc(dx),
            _desc(dweight), ws.data_ptr() if want else None, ws.numel() * ws.element_size() if want else 0, c.stream),
            "moe_norm_before_backward")
    return dx, dweight


def norm_after_backward(dout, y, rstd, weight=None, gate=None, *, gate_act="none", normalize=True, dy=None,
                        dweight=None, dgate=None, weight_grad=True, gate_grad=True, grad_dtype=torch.float32,
                        workspace=None, stream=None):
    """(dy, dweight, dgate): the gradient of norm_after given dout, rstd as the forward wrote it.
    dweight and dgate (in grad_dtype; dgate of the gate's shape, summed over its axes of size
    1) are None without a weight or a gate, or with weight_grad / gate_grad False.  The gradient
    with respect to the residual is residual_scale * dout (norm_before_backward adds it)."""
    T, H = _rows(dout, "dout")
    act = _act(gate_act)
    want_w = dweight is not None or (weight is not None and weight_grad)
    want_g = dgate is not None or (gate is not None and gate_grad)
    with _Call(stream, dout, y, rstd, weight, gate, dy, dweight, dgate, workspace) as c:
        if dy is None:
            dy = c.empty(T, H, dtype=y.dtype)
        if want_w and dweight is None:
            dweight = c.empty(H, dtype=grad_dtype)
        if want_g and dgate is None:
            dgate = c.empty(*gate.shape, dtype=grad_dtype)
        want = want_w or want_g
        ws = c.workspace(workspace, norm_backward_workspace_bytes(T, H)) if want else None
        _check(load().moe_norm_after_backward(
            _desc(dout), _desc(y), _desc(rstd), _desc(weight), _desc(gate), act, 1 if normalize else 0, _desc(dy),
            _desc(dweight), _desc(dgate), ws.data_ptr() if want else None,
            ws.numel() * ws.element_size() if want else 0, c.stream),
            "moe_norm_after_backward")
    return dy, dweight, dgate


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
    T, H = _rows(x, "x")
    E, _ = _rows(router, "router")
    act = _act(gate_act)
    n = 1 if shared_expert else 0
    with _Call(stream, x, router, w2, w2_scale, pre_weight, post_weight, gate, out, topk_ids, topk_weights,
               workspace) as c:
        if out is None:
            out = c.empty(T, H, dtype=torch.bfloat16)
        if topk_ids is None:
            topk_ids = c.empty(T, k + n, dtype=torch.int32)
        if topk_weights is None:
            topk_weights = c.empty(T, k + n, dtype=torch.float32)
        if w2_scale is None:
            d2, mx = _desc(w2), False
        else:
            d2, mx = _experts_desc(w2, w2_scale), True
        ws = c.workspace(workspace, layer_decode_workspace_bytes(T, H, w13.gate.sizes[1], E + n, k + n, mx))
        _check(load().moe_layer_decode(
            _desc(x), _desc(pre_weight), eps, _desc(router), k, 1 if renormalize else 0, n, ctypes.byref(w13), d2,
            1 if post_norm else 0, _desc(post_weight), _desc(gate), act, residual_scale, _desc(topk_ids),
            _desc(topk_weights), _desc(out), ws.data_ptr(), ws.numel() * ws.element_size(), c.stream),
            "moe_layer_decode")
    return out, topk_ids, topk_weights


SCALE_E8M0_32, SCALE_E4M3_16 = 0, 1


def _code_form(codes, scale):
    """The scale format of a code matrix, from its scales' type; checks both tensors' sizes."""
    if codes.dtype not in (torch.uint8, getattr(torch, "float4_e2m1fn_x2", torch.uint8)):
        raise ValueError(f"codes of type {codes.dtype}, not uint8 or float4_e2m1fn_x2")
    if codes.dim() != 2 or scale.dim() != 2:
        raise ValueError(f"codes of {codes.dim()} and scales of {scale.dim()} dimensions, not 2")
    if scale.dtype == torch.float8_e4m3fn:
        form, per = SCALE_E4M3_16, 16
    elif scale.dtype in (torch.uint8, getattr(torch, "float8_e8m0fnu", torch.uint8)):
        form, per = SCALE_E8M0_32, 32
    else:
        raise ValueError(f"scales of type {scale.dtype}: float8_e4m3fn per 16, or uint8 / float8_e8m0fnu per 32")
    N, K = codes.shape[0], 2 * codes.shape[1]
    if K % 32 != 0 or tuple(scale.shape) != (N, K // per):
        raise ValueError(f"scales of shape {tuple(scale.shape)} for codes of {N} rows of {K} elements")
    return form


def quantize_nvfp4(src, global_scale=None, *, stream=None):
    """(codes uint8 [R, K/2], scales float8_e4m3fn [R, K/16], global_scale f32 [1]) of src [R, K]
    (bf16 or f32, K a multiple of 32): e2m1 codes, an e4m3 scale per 16, one float scale for the
    tensor.  Without a given global_scale it is amax / 2688, which costs a pass over src."""
    R, K = _rows(src, "src")
    with _Call(stream, src, global_scale) as c:
        if global_scale is None:
            global_scale = ((src.abs().amax().float() if src.numel() else torch.zeros((), device=src.device))
                            / 2688.0).reshape(1)
        codes = c.empty(R, K // 2, dtype=torch.uint8)
        scales = c.empty(R, K // 16, dtype=torch.float8_e4m3fn)
        _check(load().moe_quantize_nvfp4(_desc(src), _desc(global_scale), _codes_desc(codes, scales), c.stream),
               "moe_quantize_nvfp4")
    return codes, scales, global_scale


def linear_fp4_workspace_bytes(T: int, N: int, K: int, scale_format: int) -> int:
    return int(load().moe_linear_fp4_workspace_bytes(T, N, K, scale_format))


def linear_fp4(x, weight, weight_scale, *, x_global=None, w_global=None, out=None, workspace=None, stream=None):
    """out [T, N] bf16 = x [T, K] (bf16 or f32, quantised on the way in) times the transposed 4-bit
    weight [N, K]: codes uint8 [N, K/2] and, either e4m3 scales [N, K/16] (quantize_nvfp4; x_global
    the float scale of x, w_global the weight's) or e8m0 scales [N, K/32] (quantize_mxfp4)."""
    T, K = _rows(x, "x")
    form = _code_form(weight, weight_scale)
    with _Call(stream, x, weight, weight_scale, x_global, w_global, out, workspace) as c:
        N = weight.shape[0]
        if out is None:
            out = c.empty(T, N, dtype=torch.bfloat16)
        ws = c.workspace(workspace, linear_fp4_workspace_bytes(T, N, K, form))
        _check(load().moe_linear_fp4(_desc(x), _codes_desc(weight, weight_scale), form, _desc(x_global),
                                     _desc(w_global), _desc(out), ws.data_ptr(), ws.numel() * ws.element_size(),
                                     c.stream), "moe_linear_fp4")
    return out
