"""The norms around a block and their gradients against plain 64-bit formulas.

Tolerances, with u = 2^-24 (fp32) and h = half a step of the output's type (bf16 2^-8, fp32 u):
  * r = 1 / sqrt(mean): a sum of non-negative squares, at most 16 sequential additions a thread and
    10 in the trees, each relative u; halved by the root, plus root, division and mean: below
    2^-19 relative.  Products, the activation (a few ulp) and the sum with the residual add less
    than 2^-20.  So |out - ref| <= 2^-18 (|alpha x| + |z|) + h |ref|.
  * the next norm sees out's unrounded error, scaled by r' w': 2^-17 (|alpha x| + |z|) r' |w'| + h |ref|.
  * dy, dx: r (|p| + |yh| mean|p yh|) in place of the magnitudes above, same factors.
  * column sums over T rows: at most T + 64 additions of terms with a relative error below
    2^-18: (2^-18 + (T + 64) u) sum|term| + h |ref|.
"""

import os
import subprocess
import sys

import pytest
import torch

import mixture_experts_layer_46_b200 as moe

pytestmark = pytest.mark.gpu

BF, F32, D = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
H_OF = {BF: 2.0 ** -8, F32: U}


def rnd(g, *shape, dt=BF, scale=1.0, pad=0):
    v = torch.randn(*shape[:-1], shape[-1] + pad, generator=g) * scale
    return v.to(dt).cuda()[..., : shape[-1]]


def gate_of(g, kind, T, H, dt):
    shape = {"none": None, "full": (T, H), "channel": (1, H), "token": (T, 1), "one": (1, 1)}[kind]
    return None if shape is None else rnd(g, *shape, dt=dt)


def act64(v, act):
    v = v.to(D)
    return torch.sigmoid(v) if act == "sigmoid" else torch.tanh(v) if act == "tanh" else v


def slope64(v, act):
    a = act64(v, act)
    return a * (1 - a) if act == "sigmoid" else 1 - a * a if act == "tanh" else torch.ones_like(a)


def within(got, ref, room):
    assert got.shape == ref.shape
    room = room + H_OF[got.dtype] * ref.abs()
    bad = (got.to(D) - ref).abs() > room
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {((got.to(D) - ref).abs() / room).max():.3g} x the room"


def rstd64(v, eps=1e-6):
    return 1 / (v.to(D).pow(2).mean(-1) + eps).sqrt()


SHAPES = [(1, 1), (1, 4096), (2, 7), (3, 64), (5, 1407), (33, 2048), (700, 512), (9, 4104), (3, 16384), (257, 1000),
          (320, 16384), (310, 9000), (400, 6000)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("xdt,odt,wdt", [(BF, BF, BF), (F32, BF, F32), (BF, F32, None)])
def test_before(T, H, xdt, odt, wdt):
    g = torch.Generator().manual_seed(T * 7 + H)
    x = rnd(g, T, H, dt=xdt, scale=3.0)
    w = None if wdt is None else rnd(g, H, dt=wdt)
    out, r = moe.norm_before(x, w, out_dtype=odt)
    ref_r = rstd64(x)
    ref = x.to(D) * ref_r[:, None] * (1.0 if w is None else w.to(D))
    within(r, ref_r, 2.0 ** -19 * ref_r)
    within(out, ref, 2.0 ** -18 * ref.abs())
    assert out.dtype == odt and r.dtype == F32


def after_ref(y, x, w, gate, act, norm, alpha, wn):
    ry = rstd64(y) if norm else torch.ones(y.shape[0], dtype=D, device="cuda")
    z = y.to(D) * ry[:, None] * (1.0 if w is None else w.to(D)) * (1.0 if gate is None else act64(gate, act))
    a = alpha * x.to(D) if x is not None else torch.zeros_like(z)
    out = a + z
    rn = rstd64(out)
    return ry, out, out * rn[:, None] * (1.0 if wn is None else wn.to(D)), rn, a.abs() + z.abs()


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gate,act", [("none", "none"), ("full", "tanh"), ("channel", "none"), ("token", "sigmoid"),
                                      ("one", "tanh")])
@pytest.mark.parametrize("xdt,ydt,norm,alpha", [(BF, BF, True, 1.0), (F32, BF, True, 0.5), (BF, F32, False, -0.25)])
def test_after(T, H, gate, act, xdt, ydt, norm, alpha):
    g = torch.Generator().manual_seed(T + H)
    y, x = rnd(g, T, H, dt=ydt, scale=0.3), rnd(g, T, H, dt=xdt, scale=2.0)
    w, wn = rnd(g, H, dt=BF), rnd(g, H, dt=F32)
    gt = gate_of(g, gate, T, H, BF if act == "none" else F32)
    out, r, nxt, rn = moe.norm_after(y, x, w, gt, gate_act=act, normalize=norm, residual_scale=alpha, next_weight=wn,
                                     next_dtype=BF)
    ry, ref, refn, refr, mag = after_ref(y, x, w, gt, act, norm, alpha, wn)
    within(r, ry, 2.0 ** -19 * ry)
    within(out, ref, 2.0 ** -18 * mag)
    # r' has out's error averaged over the row on top of its own
    rel = 2.0 ** -17 * mag.pow(2).mean(-1).sqrt() * refr + 2.0 ** -18
    within(rn, refr, rel * refr)
    within(nxt, refn, 2.0 ** -17 * mag * refr[:, None] * wn.abs().to(D) + rel[:, None] * refn.abs())
    # the short form gives the same stream, and a call without a residual or a weight works
    o2, r2 = moe.norm_after(y, x, w, gt, gate_act=act, normalize=norm, residual_scale=alpha)
    assert torch.equal(o2, out) and torch.equal(r2, r)
    o3, _ = moe.norm_after(y, normalize=norm)
    within(o3, y.to(D) * ry[:, None], 2.0 ** -18 * (y.to(D) * ry[:, None]).abs())


def grads_ref(do, y, r, w, gate, act, norm):
    yh = y.to(D) * r.to(D)[:, None] if norm else y.to(D)
    a = act64(gate, act) if gate is not None else torch.ones(1, 1, dtype=D, device="cuda")
    wd = w.to(D) if w is not None else torch.ones(y.shape[1], dtype=D, device="cuda")
    d = do.to(D) * a
    p = d * wd
    rr = r.to(D)[:, None] if norm else 1.0
    dy = rr * (p - yh * (p * yh).mean(-1, keepdim=True)) if norm else p
    mdy = rr * (p.abs() + yh.abs() * (p * yh).abs().mean(-1, keepdim=True)) if norm else p.abs()
    dw, mdw = (d * yh).sum(0), (d * yh).abs().sum(0)
    dg = mdg = None
    if gate is not None:
        e = do.to(D) * yh * wd * slope64(gate, act)
        dims = [i for i in (0, 1) if gate.shape[i] == 1]
        dg, mdg = (e.sum(dims, keepdim=True), e.abs().sum(dims, keepdim=True)) if dims else (e, e.abs())
    return dy, mdy, dw, mdw, dg, mdg


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gate,act", [("none", "none"), ("full", "tanh"), ("channel", "sigmoid"), ("token", "none"),
                                      ("one", "tanh")])
@pytest.mark.parametrize("dt,ydt,norm,gdt", [(BF, BF, True, F32), (F32, BF, True, BF), (BF, F32, False, F32)])
def test_after_backward(T, H, gate, act, dt, ydt, norm, gdt):
    g = torch.Generator().manual_seed(3 * T + H)
    do, y = rnd(g, T, H, dt=dt), rnd(g, T, H, dt=ydt, scale=0.5)
    w, gt = rnd(g, H, dt=BF), gate_of(g, gate, T, H, BF)
    r = rstd64(y).float()
    dy, dw, dg = moe.norm_after_backward(do, y, r, w, gt, gate_act=act, normalize=norm, grad_dtype=gdt)
    rdy, mdy, rdw, mdw, rdg, mdg = grads_ref(do, y, r, w, gt, act, norm)
    within(dy, rdy, 2.0 ** -18 * mdy)
    within(dw, rdw, (2.0 ** -18 + (T + 64) * U) * mdw)
    if gt is None:
        assert dg is None
    else:
        assert dg.shape == gt.shape
        within(dg, rdg, (2.0 ** -18 + (T + 64) * U) * mdg)
    # the same call again gives the same bits
    again = moe.norm_after_backward(do, y, r, w, gt, gate_act=act, normalize=norm, grad_dtype=gdt)
    for a, b in zip((dy, dw, dg), again):
        assert a is b is None or torch.equal(a, b)


@pytest.mark.parametrize("T,H", SHAPES + [(5000, 96)])
@pytest.mark.parametrize("dt,xdt,alpha", [(BF, BF, 1.0), (BF, F32, 0.7), (F32, BF, 0.0)])
def test_before_backward(T, H, dt, xdt, alpha):
    g = torch.Generator().manual_seed(5 * T + H)
    do, x, dres = rnd(g, T, H, dt=dt), rnd(g, T, H, dt=xdt, scale=2.0), rnd(g, T, H, dt=xdt)
    w = rnd(g, H, dt=BF)
    r = rstd64(x).float()
    dx, dw = moe.norm_before_backward(do, x, r, w, residual_grad=dres, residual_scale=alpha)
    rdx, mdx, rdw, mdw, _, _ = grads_ref(do, x, r, w, None, "none", True)
    within(dx, rdx + alpha * dres.to(D), 2.0 ** -18 * (mdx + abs(alpha) * dres.to(D).abs()))
    within(dw, rdw, (2.0 ** -18 + (T + 64) * U) * mdw)
    dx2, none = moe.norm_before_backward(do, x, r)
    rdx2 = grads_ref(do, x, r, None, None, "none", True)
    assert none is None
    within(dx2, rdx2[0], 2.0 ** -18 * rdx2[1])


def test_gradients_against_differences():
    # L = sum(c * out) of the whole chain in fp32; central differences of step 2^-6 relative
    # to values near 1: truncation ~ 2^-12 of the third derivative (order 1), rounding
    # ~ sqrt(T H) u / 2^-6; 2^-8 of the largest entry covers both with room
    g = torch.Generator().manual_seed(0)
    T, H, s = 3, 24, 2.0 ** -6
    x, y, c = (rnd(g, T, H, dt=F32) for _ in range(3))
    w, gt = rnd(g, H, dt=F32), rnd(g, 1, H, dt=F32)

    def loss(x, y, w, gt):
        o, _, n, _ = moe.norm_after(y, x, w, gt, gate_act="tanh", residual_scale=0.5, next_weight=w)
        return (o.to(D) * c.to(D)).sum() + (n.to(D) * c.to(D)).sum()

    out, r, _, rn = moe.norm_after(y, x, w, gt, gate_act="tanh", residual_scale=0.5, next_weight=w)
    dout, dwn = moe.norm_before_backward(c, out, rn, w, residual_grad=c)
    dy, dw, dg = moe.norm_after_backward(dout, y, r, w, gt, gate_act="tanh")
    for name, at, grad in (("x", 0, 0.5 * dout), ("y", 1, dy), ("w", 2, dw + dwn), ("gate", 3, dg)):
        args = [x, y, w, gt]
        num = torch.zeros_like(args[at], dtype=D)
        for i in range(args[at].numel()):
            hi, lo = args[at].clone(), args[at].clone()
            hi.view(-1)[i] += s
            lo.view(-1)[i] -= s
            num.view(-1)[i] = (loss(*args[:at], hi, *args[at + 1:]) - loss(*args[:at], lo, *args[at + 1:])) / (2 * s)
        assert (num - grad.to(D)).abs().max() <= 2.0 ** -8 * num.abs().max(), name


def test_strides_and_alignment_give_the_wide_path_bits_or_the_reference():
    g = torch.Generator().manual_seed(9)
    T, H = 37, 256
    x, y = rnd(g, T, H, scale=2.0), rnd(g, T, H)
    w, wn, gt = rnd(g, H), rnd(g, H), rnd(g, T, H)
    want = moe.norm_after(y, x, w, gt, next_weight=wn)

    def spread(t):  # every second column of a wider, oddly offset buffer
        big = torch.zeros(t.shape[0], 2 * t.shape[1] + 3, dtype=t.dtype, device="cuda")
        v = big[:, 1: 1 + 2 * t.shape[1]: 2]
        v.copy_(t)
        return v

    out, nxt = spread(torch.zeros_like(x)), torch.zeros(H, T, dtype=BF, device="cuda").t()
    w2 = torch.zeros(H, 3, dtype=BF, device="cuda")[:, 1].copy_(w)
    got = moe.norm_after(spread(y), spread(x), w2, gt.t().contiguous().t(), out=out, next_weight=wn, next_out=nxt)
    ry, ref, refn, refr, mag = after_ref(y, x, w, gt, "none", True, 1.0, wn)
    within(got[0], ref, 2.0 ** -18 * mag)
    within(got[2], refn, 2.0 ** -16 * mag * refr[:, None] * wn.abs().to(D))
    within(want[0], ref, 2.0 ** -18 * mag)
    # an expanded (stride 0) input row is one row for every token
    one = x[:1].expand(T, H)
    o, _ = moe.norm_before(one, w)
    assert torch.equal(o, o[:1].expand(T, H))
    # in place on the residual, and rows behind the tensor's last stay as they were
    buf = torch.full((T + 3, H), 7.0, dtype=BF, device="cuda")
    buf[:T] = x
    moe.norm_after(y, buf[:T], w, gt, out=buf[:T], next_weight=wn)
    assert torch.equal(buf[:T], want[0]) and bool((buf[T:] == 7.0).all())


def test_empty_batch_zero_rows_and_non_finite_values():
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    out, r = moe.norm_before(e, w)
    assert out.shape == (0, 64) and r.shape == (0,)
    dw = torch.full((64,), 5.0, device="cuda")
    dg = torch.full((1, 64), 5.0, device="cuda")
    moe.norm_before_backward(e, e, r, w, dweight=dw)
    assert bool((dw == 0).all())
    moe.norm_after_backward(e, e, r, w, torch.ones(1, 64, device="cuda"), dweight=dw.fill_(5.0), dgate=dg)
    assert bool((dw == 0).all()) and bool((dg == 0).all())
    # a row of zeros stays zero; a NaN or an infinity stays in its row
    x = torch.ones(4, 64, dtype=BF, device="cuda")
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 5] = float("inf")
    out, _ = moe.norm_before(x, w)
    assert bool((out[0] == 1).all()) and bool((out[1] == 0).all()) and bool(out[2].isnan().all())
    assert bool(out[3, 5].isnan()) and bool((out[3, :5] == 0).all())
    # residual_scale 0 leaves the residual's infinities out
    o, _ = moe.norm_after(torch.ones(4, 64, dtype=BF, device="cuda"), x, w, residual_scale=0.0)
    assert bool((o == 1).all())


def test_streams_graphs_and_workspaces():
    g = torch.Generator().manual_seed(1)
    T, H = 300, 1024
    do, y, x = (rnd(g, T, H) for _ in range(3))
    w, gt = rnd(g, H), rnd(g, 1, H)
    out, r, nxt, rn = moe.norm_after(y, x, w, gt, next_weight=w)
    want = moe.norm_after_backward(do, y, r, w, gt)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.norm_after_backward(do, y, r, w, gt, stream=s)
    junk = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(8)]  # must not land in the call's workspace
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del junk
    # captured with a workspace of its own, replayed on other inputs
    ws = torch.empty(moe.norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    dy, dw, dg = torch.empty_like(y), torch.empty(H, device="cuda"), torch.empty(1, H, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.norm_after(y, x, w, gt, out=out, rstd=r, next_weight=w, next_out=nxt, next_rstd=rn)
        moe.norm_after_backward(do, y, r, w, gt, dy=dy, dweight=dw, dgate=dg, workspace=ws)
    y.copy_(rnd(g, T, H))
    do.copy_(rnd(g, T, H))
    graph.replay()
    o2, r2 = moe.norm_after(y, x, w, gt)
    want = moe.norm_after_backward(do, y, r2, w, gt)
    torch.cuda.synchronize()
    assert torch.equal(o2, out)
    for a, b in zip((dy, dw, dg), want):
        assert torch.equal(a, b)


def test_far_offsets():
    """Rows past 2^31 elements: the last ones are those that a small call gives, both ways."""
    T, H = 600_000, 4096
    g = torch.Generator().manual_seed(3)
    tail, w = rnd(g, 64, H), rnd(g, H)
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    x[-64:] = tail
    out, r = moe.norm_before(x, w)
    want, rw = moe.norm_before(tail, w)
    assert torch.equal(out[-64:], want) and torch.equal(r[-64:], rw)
    dx, dw = moe.norm_before_backward(x, x, r, w, dx=out)
    wdx, wdw = moe.norm_before_backward(tail, tail, rw, w)
    assert torch.equal(dx[-64:], wdx)
    assert bool(((dw - wdw).abs() <= 2.0 ** -12 * wdw.abs().max()).all())


def test_two_streams_share_nothing():
    """Gradients at once on two streams, workspaces of their own."""
    g = torch.Generator().manual_seed(4)
    xs = [rnd(g, 64 + i, 512) for i in range(10)]
    w = rnd(g, 512)
    r = [moe.norm_before(x, w)[1] for x in xs]
    want = [moe.norm_before_backward(x, x, q, w) for x, q in zip(xs, r)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [moe.norm_before_backward(x, x, q, w, stream=st[i % 2]) for i, (x, q) in enumerate(zip(xs, r))]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T,H", [(1, 4096), (900, 4096), (2000, 1024), (70, 1407)])
def test_in_place(T, H):
    """An output on top of an input of its shape, or one tensor given twice: the bits of separate ones."""
    g = torch.Generator().manual_seed(T + H)
    y, x, w = rnd(g, T, H), rnd(g, T, H), rnd(g, H)
    gate = rnd(g, T, H)
    clone = lambda *ts: [t.clone() for t in ts]
    want = moe.norm_before(x, w)
    a, = clone(x)
    assert torch.equal(moe.norm_before(a, w, out=a)[0], want[0]) and torch.equal(a, want[0])
    want = moe.norm_after(y, x, w, gate, gate_act="tanh", next_weight=w)
    for into in ("y", "x"):
        a, b = clone(y, x)
        got = moe.norm_after(a, b, w, gate, gate_act="tanh", next_weight=w, out=a if into == "y" else b)
        for u, v in zip(got, want):
            assert torch.equal(u, v)
    twice = moe.norm_after(x, x, w)
    assert torch.equal(twice[0], moe.norm_after(x.clone(), x, w)[0])
    r, d = want[1], rnd(g, T, H)
    want = moe.norm_before_backward(d, x, r, w, residual_grad=y, residual_scale=0.5)
    for into in range(3):
        ins = clone(d, x, y)
        got = moe.norm_before_backward(ins[0], ins[1], r, w, residual_grad=ins[2], residual_scale=0.5, dx=ins[into])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    want = moe.norm_after_backward(d, y, r, w, gate)
    for into in range(2):
        ins = clone(d, y)
        got = moe.norm_after_backward(ins[0], ins[1], r, w, gate, dy=ins[into])
        for u, v in zip(got, want):
            assert torch.equal(u, v)


def test_a_block_as_it_trains():
    """The norms around a block, run together: the gradient of a loss through norm, a linear block,
    gate, scaled residual and the next norm, against differentiation in 64 bits."""
    T, H, alpha = 40, 96, 0.7
    g = torch.Generator().manual_seed(8)
    x, wb, w0, w1, w2, gate, c = (rnd(g, T, H, dt=F32), rnd(g, H, H, dt=F32, scale=H ** -0.5), rnd(g, H, dt=F32),
                                  rnd(g, H, dt=F32), rnd(g, H, dt=F32), rnd(g, 1, H, dt=F32), rnd(g, T, H, dt=F32))
    xn, rx = moe.norm_before(x, w0)
    y = xn @ wb
    out, ry, nxt, rn = moe.norm_after(y, x, w1, gate, gate_act="sigmoid", residual_scale=alpha, next_weight=w2)
    dout, dw2 = moe.norm_before_backward(c, out, rn, w2)
    dy, dw1, dgate = moe.norm_after_backward(dout, y, ry, w1, gate, gate_act="sigmoid")
    dx, dw0 = moe.norm_before_backward(dy @ wb.T, x, rx, w0, residual_grad=dout, residual_scale=alpha)
    L = [t.to(D).requires_grad_() for t in (x, w0, w1, gate, w2)]
    norm = lambda v, w: v / (v.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w
    o = alpha * L[0] + torch.sigmoid(L[3]) * norm(norm(L[0], L[1]) @ wb.to(D), L[2])
    (norm(o, L[4]) * c.to(D)).sum().backward()
    for got, leaf in zip((dx, dw0, dw1, dgate, dw2), L):
        # (chained fp32 steps with matrix products of 96 terms in between: each within 2^-16)
        assert float((got.to(D) - leaf.grad).norm() / leaf.grad.norm()) <= 2.0 ** -14


def test_rings_between_the_default_and_the_raised_limit():
    """Rows whose ring just fills the 48 KB that a launch may have without asking (the kernel's own
    shared memory is part of them), in a process that has not asked for more yet."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = """
import test_gpu_norms as t
for T, H in [(700, 4880), (4096, 3056), (4096, 4080)]:
    t.test_before(T, H, t.BF, t.BF, t.BF)
for T, H in [(700, 4080), (700, 4072), (4096, 3056)]:
    t.test_after(T, H, "none", "none", t.BF, t.BF, True, 1.0)
    t.test_after_backward(T, H, "channel", "sigmoid", t.BF, t.BF, True, t.F32)
for T, H in [(700, 2712), (700, 4080)]:
    t.test_before_backward(T, H, t.BF, t.BF, 1.0)
"""
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("T,H", [(4, 64), (5, 33), (900, 512), (400, 16384)])
@pytest.mark.parametrize("gate,act", [("none", "none"), ("full", "tanh"), ("channel", "sigmoid"), ("token", "sigmoid"),
                                      ("one", "none")])
def test_without_the_norm_the_gradient_of_y_does_not_read_y(T, H, gate, act):
    """normalize=False: dy is dout times gate and weight, whatever y holds."""
    g = torch.Generator().manual_seed(T + 3 * H)
    do, y, w, gt = rnd(g, T, H), rnd(g, T, H), rnd(g, H), gate_of(g, gate, T, H, BF)
    y[1, 5], y[2, 7], y[3, 0] = float("inf"), float("nan"), -float("inf")
    dy, _, _ = moe.norm_after_backward(do, y, None, w, gt, gate_act=act, normalize=False)
    ref = do.to(D) * w.to(D) * (1.0 if gt is None else act64(gt, act))
    assert bool(dy.isfinite().all())
    within(dy, ref, 2.0 ** -18 * ref.abs())


def test_an_empty_call_launches_nothing_and_says_so():
    w, e, x = torch.ones(64, device="cuda"), torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(2, 64, device="cuda")
    r = torch.empty(0, device="cuda")
    codes, sf, G = moe.quantize_nvfp4(x)
    w13, w2 = moe.w13_from_packed(torch.zeros(4, 64, 64, dtype=BF, device="cuda")), torch.zeros(4, 64, 32, dtype=BF, device="cuda")
    for call in (lambda: moe.norm_before(e, w), lambda: moe.norm_after(e, e, w, next_norm=True),
                 lambda: moe.norm_before_backward(e, e, r), lambda: moe.norm_after_backward(e, e, r),
                 lambda: moe.quantize_nvfp4(e, G), lambda: moe.linear_fp4(e, codes, sf, x_global=G),
                 lambda: moe.layer_decode(e, torch.zeros(4, 64, device="cuda"), w13, w2, 2)):
        moe.norm_before(x, w)
        assert moe.last_launch_count() == 1
        call()
        assert moe.last_launch_count() == 0
