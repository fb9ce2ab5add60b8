"""Argument checks of the operators around the expert forward: refused before any device work
(these run without a GPU: the tensors are host memory that no kernel ever sees)."""

import pytest
import torch

import mixture_experts_layer_46_b200 as moe
from mixture_experts_layer_46_b200.block import _codes_desc, _desc

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


# ---------------------------------------------------------------- the 4-bit linear layer

U8 = torch.uint8


def linear(x=None, w=None, sf=None, form=1, xg=0, wg=None, out=None, ws=None, n=None):
    x = rows(8) if x is None else x
    w = torch.zeros(48, 32, dtype=U8) if w is None else w
    sf = torch.zeros(48, 4, dtype=U8) if sf is None else sf
    xg = torch.zeros(1) if isinstance(xg, int) else xg
    out = torch.zeros(8, 48, dtype=BF) if out is None else out
    return moe.load().moe_linear_fp4(_desc(x), _codes_desc(w, sf) if w.dtype == U8 else _desc(w), form, _desc(xg),
                                     _desc(wg), _desc(out), ws.data_ptr() if ws is not None else None,
                                     (ws.numel() if n is None else n) if ws is not None else 0, None)


@pytest.mark.parametrize("call,want", [
    (lambda: linear(form=2), INVALID),
    (lambda: linear(xg=None), INVALID),                       # e4m3 scales need x's float scale
    (lambda: linear(form=0), INVALID),                        # e8m0 scales have none
    (lambda: linear(form=0, xg=None, wg=torch.zeros(1)), INVALID),
    (lambda: linear(xg=torch.zeros(2)), SHAPE),
    (lambda: linear(xg=torch.zeros(1, dtype=BF)), DTYPE),
    (lambda: linear(wg=torch.zeros(1, 1)), INVALID),
    (lambda: linear(x=torch.zeros(64)), INVALID),
    (lambda: linear(x=rows(8).half()), DTYPE),
    (lambda: linear(w=rows(48, 64)), DTYPE),
    (lambda: linear(out=torch.zeros(8, 48)), DTYPE),
    (lambda: linear(out=torch.zeros(7, 48, dtype=BF)), SHAPE),
    (lambda: linear(out=torch.zeros(8, 47, dtype=BF)), SHAPE),
    (lambda: linear(x=rows(8, 96)), SHAPE),
    (lambda: linear(x=rows(8, 48), w=torch.zeros(48, 24, dtype=U8)), SHAPE),  # K not a multiple of 32
    (lambda: linear(out=torch.zeros(1, 48, dtype=BF).expand(8, 48)), LAYOUT),
    (lambda: linear(w=torch.zeros(48, 40, dtype=U8)[:, :32]), LAYOUT),        # rows 40 bytes apart
    (lambda: linear(w=torch.zeros(32, 48, dtype=U8).t()), LAYOUT),
    (lambda: linear(w=torch.zeros(1, 32, dtype=U8).expand(48, 32)), LAYOUT),
    (lambda: linear(), INVALID),                              # no workspace
])
def test_linear_refuses(call, want):
    assert call() == want


def test_linear_workspace():
    n = moe.linear_fp4_workspace_bytes(8, 48, 64, moe.SCALE_E4M3_16)
    raw = torch.zeros(n + 512, dtype=U8)
    ws = raw[(-raw.data_ptr()) % 256:][:n]
    assert linear(ws=ws, n=n - 1) == SMALL
    assert linear(ws=raw[(-raw.data_ptr()) % 256 + 16:][:n]) == INVALID
    assert moe.linear_fp4_workspace_bytes(8, 48, 48, 0) == 0
    assert moe.linear_fp4_workspace_bytes(-1, 48, 64, 0) == 0
    assert moe.linear_fp4_workspace_bytes(8, 48, 64, 7) == 0
    # codes of x, its scales in whole blocks of 256 rows, the weight's scales
    assert moe.linear_fp4_workspace_bytes(8192, 8192, 4096, 1) < 8192 * 2048 + 2 * 8960 * 256 + 4096


def test_linear_wrapper_refuses():
    x, w = rows(8), torch.zeros(48, 32, dtype=U8)
    with pytest.raises(ValueError, match="shape"):
        moe.linear_fp4(x, w, torch.zeros(48, 3, dtype=U8))
    with pytest.raises(ValueError, match="shape"):
        moe.linear_fp4(x, w, torch.zeros(48, 2, dtype=U8).view(torch.float8_e4m3fn))
    with pytest.raises(ValueError, match="type"):
        moe.linear_fp4(x, w, torch.zeros(48, 2))
    with pytest.raises(ValueError, match="type"):
        moe.linear_fp4(x, torch.zeros(48, 32), torch.zeros(48, 2, dtype=U8))
    with pytest.raises(ValueError, match="CUDA"):
        moe.linear_fp4(x, w, torch.zeros(48, 2, dtype=U8))
    with pytest.raises(ValueError, match="CUDA"):
        moe.quantize_nvfp4(x)


@pytest.mark.parametrize("src,G,dst,want", [
    (rows(4, 48), torch.zeros(1), (4, 48), SHAPE),
    (rows(4, 64), torch.zeros(2), (4, 64), SHAPE),
    (rows(4, 64), torch.zeros(1), (5, 64), SHAPE),
    (rows(4, 64).half(), torch.zeros(1), (4, 64), DTYPE),
    (rows(4, 64), torch.zeros(1, dtype=BF), (4, 64), DTYPE),
    (torch.zeros(64), torch.zeros(1), (4, 64), INVALID),
])
def test_quantize_refuses(src, G, dst, want):
    codes, sf = torch.zeros(dst[0], dst[1] // 2, dtype=U8), torch.zeros(dst[0], dst[1] // 16, dtype=U8)
    assert moe.load().moe_quantize_nvfp4(_desc(src), _desc(G), _codes_desc(codes, sf), None) == want


# ---------------------------------------------------------------- a whole layer for a few tokens

def layer(T=2, H=64, I=32, E=4, k=2, x=None, pre=None, eps=1e-6, router=None, renorm=1, shared=0, post=0, pw=None,
          gate=None, act=0, ids=None, wts=None, out=None, w13=None, w2=None, ws=None, n=None):
    import ctypes

    x = rows(T, H) if x is None else x
    router = rows(E, H) if router is None else router
    w13 = torch.zeros(E + shared, 2 * I, H, dtype=BF) if w13 is None else w13
    w2 = torch.zeros(E + shared, H, I, dtype=BF) if w2 is None else w2
    ids = torch.zeros(T, k + shared, dtype=torch.int32) if ids is None else ids
    wts = torch.zeros(T, k + shared) if wts is None else wts
    out = rows(T, H) if out is None else out
    return moe.load().moe_layer_decode(
        _desc(x), _desc(pre), eps, _desc(router), k, renorm, shared, ctypes.byref(moe.w13_from_packed(w13)), _desc(w2),
        post, _desc(pw), _desc(gate), act, 1.0, _desc(ids), _desc(wts), _desc(out),
        ws.data_ptr() if ws is not None else None, (ws.numel() if n is None else n) if ws is not None else 0, None)


@pytest.mark.parametrize("call,want", [
    (lambda: layer(T=33), INVALID),
    (lambda: layer(k=5), INVALID),
    (lambda: layer(k=0, ids=torch.zeros(2, 1, dtype=torch.int32), wts=torch.zeros(2, 1)), INVALID),
    (lambda: layer(E=40, k=32, shared=1), INVALID),
    (lambda: layer(E=1025), INVALID),
    (lambda: layer(eps=float("nan")), INVALID),
    (lambda: layer(renorm=2), INVALID),
    (lambda: layer(act=5), INVALID),
    (lambda: layer(pw=torch.zeros(64)), INVALID),                       # a post weight without the post norm
    (lambda: layer(x=torch.zeros(2, 64)), DTYPE),
    (lambda: layer(router=torch.zeros(4, 64, dtype=torch.float16)), DTYPE),
    (lambda: layer(ids=torch.zeros(2, 2)), DTYPE),
    (lambda: layer(wts=torch.zeros(2, 2, dtype=BF)), DTYPE),
    (lambda: layer(router=rows(4, 32)), SHAPE),
    (lambda: layer(pre=torch.zeros(63)), SHAPE),
    (lambda: layer(ids=torch.zeros(2, 3, dtype=torch.int32)), SHAPE),
    (lambda: layer(w13=torch.zeros(5, 64, 64, dtype=BF)), SHAPE),
    (lambda: layer(w2=torch.zeros(4, 64, 64, dtype=BF)), SHAPE),
    (lambda: layer(gate=torch.zeros(3, 64)), SHAPE),
    (lambda: layer(out=rows(2, 32)), SHAPE),
    (lambda: layer(ids=torch.zeros(1, 2, dtype=torch.int32).expand(2, 2)), LAYOUT),
    (lambda: layer(out=torch.zeros(1, 64, dtype=BF).expand(2, 64)), LAYOUT),
    (lambda: layer(), INVALID),                                         # no workspace
])
def test_layer_refuses(call, want):
    assert call() == want


def test_layer_workspace():
    n = moe.layer_decode_workspace_bytes(2, 64, 32, 4, 2)
    raw = torch.zeros(n + 512, dtype=U8)
    ws = raw[(-raw.data_ptr()) % 256:][:n]
    assert layer(ws=ws, n=n - 1) == SMALL
    assert layer(ws=raw[(-raw.data_ptr()) % 256 + 16:][:n]) == INVALID
    assert moe.layer_decode_workspace_bytes(33, 64, 32, 4, 2) == 0
    assert moe.layer_decode_workspace_bytes(2, 16416, 32, 4, 2) == 0
    with pytest.raises(ValueError, match="CUDA"):
        moe.layer_decode(rows(2), rows(4), moe.w13_from_packed(torch.zeros(4, 64, 64, dtype=BF)), torch.zeros(4, 64, 32, dtype=BF), 2)


def test_layer_wrapper_checks_the_scales():
    """w2's codes and scales by type and shape: e4m3 scales per 16, or too few, are not read as e8m0 per 32."""
    w13 = moe.w13_from_packed(torch.zeros(4, 512, 128, dtype=U8), torch.zeros(4, 512, 8, dtype=U8))
    codes = torch.zeros(4, 256, 128, dtype=U8)
    call = lambda w2, s: moe.layer_decode(rows(2, 256), rows(4, 256), w13, w2, 2, w2_scale=s)
    for s in (torch.zeros(4, 256, 16, dtype=U8).view(torch.float8_e4m3fn), torch.zeros(4, 256, 8),
              torch.zeros(4, 256, 8, dtype=U8).view(torch.float8_e4m3fn)):
        with pytest.raises(ValueError, match="type"):
            call(codes, s)
    for s in (torch.zeros(4, 256, 7, dtype=U8), torch.zeros(4, 255, 8, dtype=U8), torch.zeros(256, 8, dtype=U8),
              torch.zeros(4, 256, 16, dtype=U8), torch.zeros(3, 256, 8, dtype=U8)):
        with pytest.raises(ValueError, match="shape"):
            call(codes, s)
    with pytest.raises(ValueError, match="codes of type"):
        call(torch.zeros(4, 256, 128, dtype=BF), torch.zeros(4, 256, 8, dtype=U8))
    with pytest.raises(ValueError, match="CUDA"):
        call(codes, torch.zeros(4, 256, 8, dtype=U8))


@pytest.mark.parametrize("ws", [torch.zeros(1, dtype=U8).expand(1 << 24), torch.zeros(1 << 22, dtype=U8)[::2]])
def test_wrappers_refuse_workspaces_that_are_not_one_block_of_memory(ws):
    """Their element count says nothing of the bytes behind their address."""
    x, r, w = rows(), torch.zeros(4), torch.zeros(64)
    w13 = moe.w13_from_packed(torch.zeros(4, 64, 64, dtype=BF))
    for call in (lambda: moe.norm_before_backward(x, x, r, w, workspace=ws),
                 lambda: moe.norm_after_backward(x, x, r, w, workspace=ws),
                 lambda: moe.layer_decode(x, rows(4), w13, torch.zeros(4, 64, 32, dtype=BF), 2, workspace=ws),
                 lambda: moe.linear_fp4(x, torch.zeros(48, 32, dtype=U8), torch.zeros(48, 2, dtype=U8), workspace=ws)):
        with pytest.raises(ValueError, match="contiguous"):
            call()


def test_wrappers_pass_on_what_a_truth_value_raises():
    """A flag whose truth value raises is that error, not a false flag."""
    x, r, w, many = rows(), torch.zeros(4), torch.zeros(64), torch.zeros(2)
    for call in (lambda: moe.norm_after(x, next_norm=many), lambda: moe.norm_before_backward(x, x, r, w, weight_grad=many),
                 lambda: moe.norm_after_backward(x, x, r, w, weight_grad=many),
                 lambda: moe.norm_after_backward(x, x, r, w, torch.zeros(1, 64), gate_grad=many)):
        with pytest.raises(RuntimeError, match="[Bb]oolean value"):
            call()


def test_the_binding_is_compiled_again_for_another_torch(monkeypatch, tmp_path):
    """Newer than its sources is not enough: its binary interface is that of the torch it was compiled with."""
    from mixture_experts_layer_46_b200 import build

    runs = []
    monkeypatch.setattr(build, "BINDING_FOR", str(tmp_path / "built_for"))
    monkeypatch.setattr(build, "_stale", lambda target, deps: False)
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, check: runs.append(cmd))
    build.build_binding()
    assert len(runs) == 1 and build.BINDING in runs[0]
    build.build_binding()
    assert len(runs) == 1
    (tmp_path / "built_for").write_text("torch 0.0, another Python")
    build.build_binding()
    assert len(runs) == 2
    build.build_binding(force=True)
    assert len(runs) == 3
