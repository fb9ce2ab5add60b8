"""Argument checks of the operators around the expert forward: refused before any device work
(these run without a GPU: the tensors are host memory that no kernel ever sees)."""

import pytest
import torch

import mixture_experts_layer_46_b200 as moe
from mixture_experts_layer_46_b200.block import _desc

BF, F32 = torch.bfloat16, torch.float32
INVALID, SHAPE, DTYPE, LAYOUT, SMALL = 1, 2, 3, 4, 5


def rows(T=4, H=64, dt=BF):
    return torch.zeros(T, H, dtype=dt)


def before(x=None, w=None, eps=1e-6, out=None, rstd=None):
    x = rows() if x is None else x
    out = rows() if out is None else out
    return moe.load().moe_norm_before(_desc(x), _desc(w), eps, _desc(out), _desc(rstd), None)


def after(y=None, x=None, w=None, gate=None, act=0, norm=1, alpha=1.0, eps=1e-6, out=None, rstd=None, wn=None,
          nxt=None, nrstd=None):
    y = rows() if y is None else y
    out = rows() if out is None else out
    return moe.load().moe_norm_after(_desc(y), _desc(x), _desc(w), _desc(gate), act, norm, alpha, eps, _desc(out),
                                     _desc(rstd), _desc(wn), _desc(nxt), _desc(nrstd), None)


def before_bwd(dout=None, x=None, rstd=None, w=None, dres=None, dx=None, dw=None, ws=None, n=None):
    dout, x = rows() if dout is None else dout, rows() if x is None else x
    rstd, dx = torch.zeros(4) if rstd is None else rstd, rows() if dx is None else dx
    return moe.load().moe_norm_before_backward(
        _desc(dout), _desc(x), _desc(rstd), _desc(w), _desc(dres), 1.0, _desc(dx), _desc(dw),
        ws.data_ptr() if ws is not None else None, (ws.numel() if n is None else n) if ws is not None else 0, None)


def after_bwd(dout=None, y=None, rstd=None, w=None, gate=None, act=0, norm=1, dy=None, dw=None, dg=None, ws=None):
    dout, y = rows() if dout is None else dout, rows() if y is None else y
    dy = rows() if dy is None else dy
    return moe.load().moe_norm_after_backward(
        _desc(dout), _desc(y), _desc(rstd), _desc(w), _desc(gate), act, norm, _desc(dy), _desc(dw), _desc(dg),
        ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0, None)


@pytest.mark.parametrize("call,want", [
    (lambda: before(x=torch.zeros(4)), INVALID),
    (lambda: before(x=rows(4, 16392), out=rows(4, 16392)), INVALID),
    (lambda: before(eps=-1.0), INVALID),
    (lambda: before(eps=float("nan")), INVALID),
    (lambda: before(eps=float("inf")), INVALID),
    (lambda: before(x=rows().half()), DTYPE),
    (lambda: before(out=rows().half()), DTYPE),
    (lambda: before(out=rows(4, 65)), SHAPE),
    (lambda: before(out=rows(5, 64)), SHAPE),
    (lambda: before(w=torch.zeros(63)), SHAPE),
    (lambda: before(w=torch.zeros(64, 1)), INVALID),
    (lambda: before(w=torch.zeros(64, dtype=torch.int32)), DTYPE),
    (lambda: before(out=torch.zeros(1, 64, dtype=BF).expand(4, 64)), LAYOUT),
    (lambda: before(out=torch.zeros(4, 1, dtype=BF).expand(4, 64)), LAYOUT),
    (lambda: before(rstd=torch.zeros(3)), SHAPE),
    (lambda: before(rstd=torch.zeros(4, dtype=BF)), DTYPE),
    (lambda: before(rstd=torch.zeros(1).expand(4)), LAYOUT),
    (lambda: after(x=rows(3)), SHAPE),
    (lambda: after(act=3), INVALID),
    (lambda: after(norm=2), INVALID),
    (lambda: after(gate=torch.zeros(2, 64)), SHAPE),
    (lambda: after(gate=torch.zeros(4, 32)), SHAPE),
    (lambda: after(gate=torch.zeros(64)), INVALID),
    (lambda: after(gate=torch.zeros(4, 64, dtype=torch.float64)), DTYPE),
    (lambda: after(nxt=rows(4, 32)), SHAPE),
    (lambda: after(wn=torch.zeros(32)), SHAPE),
    (lambda: after(nrstd=torch.zeros(5)), SHAPE),
    (lambda: before_bwd(x=rows(4, 32)), SHAPE),
    (lambda: before_bwd(rstd=torch.zeros(4, 1)), INVALID),
    (lambda: before_bwd(dres=rows(1)), SHAPE),
    (lambda: before_bwd(dw=torch.zeros(64)), INVALID),
    (lambda: before_bwd(dw=torch.zeros(32)), SHAPE),
    (lambda: after_bwd(), INVALID),                                          # normalised, no rstd
    (lambda: after_bwd(rstd=torch.zeros(4), dg=torch.zeros(4, 64)), INVALID),  # a gate's gradient without a gate
    (lambda: after_bwd(rstd=torch.zeros(4), gate=torch.zeros(1, 64), dg=torch.zeros(4, 64)), SHAPE),
    (lambda: after_bwd(rstd=torch.zeros(4), gate=torch.zeros(4, 64), dg=torch.zeros(4, 1).expand(4, 64)), LAYOUT),
    (lambda: after_bwd(rstd=torch.zeros(4), gate=torch.zeros(1, 64), dg=torch.zeros(1, 64)), INVALID),  # no workspace
])
def test_norms_refuse(call, want):
    assert call() == want


def test_norm_workspace():
    n = moe.norm_backward_workspace_bytes(4, 64)
    assert n >= 4 * 64 * 4
    raw = torch.zeros(n + 512, dtype=torch.uint8)
    ws = raw[(-raw.data_ptr()) % 256:][:n]
    assert before_bwd(dw=torch.zeros(64), ws=ws, n=n - 1) == SMALL
    assert before_bwd(dw=torch.zeros(64), ws=raw[(-raw.data_ptr()) % 256 + 1:][:n]) == INVALID  # not 256-byte aligned
    assert moe.norm_backward_workspace_bytes(-1, 64) == 0
    assert moe.norm_backward_workspace_bytes(4, 16385) == 0
    # grows with T only up to the number of blocks
    assert moe.norm_backward_workspace_bytes(1 << 20, 4096) == moe.norm_backward_workspace_bytes(1 << 30, 4096)


def test_wrappers_refuse_host_tensors_and_bad_names():
    x = rows()
    with pytest.raises(ValueError, match="CUDA"):
        moe.norm_before(x)
    with pytest.raises(ValueError, match="CUDA"):
        moe.norm_after(x, x)
    with pytest.raises(ValueError, match="gate_act"):
        moe.norm_after(x, x, gate_act="relu")
    with pytest.raises(ValueError, match="dimensions"):
        moe.norm_before(torch.zeros(4))
