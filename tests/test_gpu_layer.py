"""A whole mixture-of-experts layer for a few tokens against plain 64-bit formulas.

The choice of experts has to be the exact one; the weights are off by less than 2^-20.  The
output, with h = 2^-8 (half a step of bf16): xn is rounded (h), so the gate and up products are
off by h A with A = |W| |xn|; silu's slope stays below 1.1, so the activation is off by
h (1.1 A_g (|u| + h A_u) + |silu(g)| A_u + |a|) with its own rounding, the slot's row by |W2|
times that and h |y| of its own, fp32 sums and exponentials by less than a hundredth of all this
(2 % more room).  The norm after it passes an error d on as r |w| (d + |y| r rms(d)); the output
rounds once.  Those are worst cases; roundings of random sign add up to far less, so the root
mean square error has to stay below 2^-6 of the block's part and 2^-8 of the output besides."""

import pytest
import torch

import mixture_experts_layer_46_b200 as moe

pytestmark = pytest.mark.gpu

BF, F32, D = torch.bfloat16, torch.float32, torch.float64
HB = 2.0 ** -8


def make(seed, T, H, I, E, shared=False, rdt=BF, wdt=BF):
    g = torch.Generator().manual_seed(seed)
    n = E + (1 if shared else 0)
    rn = lambda *s: torch.randn(*s, generator=g)
    return dict(x=(rn(T, H) * 2).to(BF).cuda(), router=(rn(E, H) / H ** 0.5).to(rdt).cuda(),
                pre=(1 + 0.2 * rn(H)).to(wdt).cuda(), post=(1 + 0.2 * rn(H)).to(wdt).cuda(),
                w13=(rn(n, 2 * I, H) / H ** 0.5).to(BF).cuda(), w2=(rn(n, H, I) / I ** 0.5).to(BF).cuda())


def route64(x, pre, router, k, renorm, shared, eps=1e-6):
    xd = x.to(D)
    xn = xd / (xd.pow(2).mean(-1, keepdim=True) + eps).sqrt() * (1.0 if pre is None else pre.to(D))
    logits = xn @ router.to(D).T
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    p = torch.softmax(logits, -1).gather(1, ids[:, :k])
    if renorm:
        p = p / p.sum(-1, keepdim=True)
    ids = ids[:, :k]
    if shared:
        ids = torch.cat([ids, torch.full_like(ids[:, :1], router.shape[0])], 1)
        p = torch.cat([p, torch.ones_like(p[:, :1])], 1)
    return xn, ids, p


def act64(v, act):
    v = v.to(D)
    return torch.sigmoid(v) if act == "sigmoid" else torch.tanh(v) if act == "tanh" else v


def layer64(s, k, renorm=True, shared=False, post=False, gate=None, act="none", alpha=1.0, eps=1e-6, pre=None):
    xn, ids, p = route64(s["x"], pre, s["router"], k, renorm, shared, eps)
    T, H = s["x"].shape
    I = s["w2"].shape[2]
    y, d = torch.zeros(T, H, dtype=D, device="cuda"), torch.zeros(T, H, dtype=D, device="cuda")
    for t in range(T):
        for j, e in enumerate(ids[t].tolist()):
            W, W2 = s["w13"][e].to(D), s["w2"][e].to(D)
            gu, A = W @ xn[t], W.abs() @ xn[t].abs()
            g, u = gu[:I], gu[I:]
            si = g * torch.sigmoid(g)
            a = si * u
            da = HB * (1.1 * A[:I] * (u.abs() + HB * A[I:]) + si.abs() * A[I:] + a.abs())
            ys = W2 @ a
            y[t] += p[t, j] * ys
            d[t] += p[t, j] * (W2.abs() @ da + HB * ys.abs())
    if post is not False:
        r = 1 / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        w = post.to(D).abs() if post is not None else 1.0
        d = r * w * (d + y.abs() * r * d.pow(2).mean(-1, keepdim=True).sqrt())
        y = y * r * (post.to(D) if post is not None else 1.0)
    if gate is not None:
        a = act64(gate, act)
        y, d = y * a, d * a.abs()
    return alpha * s["x"].to(D) + y, ids, p, 1.02 * d, y


def check(got, ref):
    out, ids, p = got
    want, wi, wp, room, z = ref
    assert torch.equal(ids.long(), wi)
    assert bool(((p.to(D) - wp).abs() <= 2.0 ** -20 * wp).all())
    err = (out.to(D) - want).abs()
    room = room + HB * want.abs()
    assert bool((err <= room).all()), f"{int((err > room).sum())} of {err.numel()} off, worst {(err / room).max():.3g} x the room"
    rms = lambda v: float(v.pow(2).mean().sqrt())
    assert rms(err) <= 2.0 ** -6 * rms(z) + HB * rms(want)


CASES = [  # T, H, I, E, k, shared, renorm, post, gate, act, alpha
    (1, 128, 64, 4, 1, False, True, False, None, "none", 1.0),
    (1, 4096, 1536, 16, 8, False, True, False, None, "none", 1.0),
    (4, 256, 96, 8, 2, False, False, False, "token", "sigmoid", 0.5),
    (5, 1024, 416, 40, 3, True, False, True, "token", "sigmoid", 0.5),
    (32, 512, 128, 128, 8, False, True, True, "channel", "none", 1.0),
    (32, 256, 64, 16, 1, False, True, False, "full", "tanh", 0.0),
    (3, 160, 32, 1, 1, True, True, True, "one", "none", 1.0),
    (11, 288, 160, 24, 5, True, True, False, "channel", "tanh", 1.0),
    (7, 2048, 64, 1000, 8, False, True, False, None, "none", 1.0),
    (2, 64, 32, 31, 31, True, True, True, None, "none", 2.0),
    # rows of up to four tokens in columns of 512: two warps a row, a row and a half, many rows a block
    (4, 800, 544, 12, 8, False, True, False, None, "none", 1.0),
    (3, 8192, 96, 6, 2, False, True, False, "channel", "sigmoid", 1.0),
    (2, 8224, 64, 6, 2, False, True, False, None, "none", 1.0),
    (4, 32, 8192, 6, 3, False, True, True, None, "none", 1.0),
    (1, 512, 4096, 40, 31, True, True, False, None, "none", 1.0),
    (4, 1024, 1536, 5, 4, False, True, False, None, "none", 1.0),
]


@pytest.mark.parametrize("T,H,I,E,k,shared,renorm,post,gate,act,alpha", CASES)
def test_layer(T, H, I, E, k, shared, renorm, post, gate, act, alpha):
    s = make(T * 31 + H, T, H, I, E, shared)
    g = torch.Generator().manual_seed(5)
    shape = {None: None, "channel": (1, H), "token": (T, 1), "full": (T, H), "one": (1, 1)}[gate]
    gt = None if shape is None else torch.randn(*shape, generator=g).to(BF).cuda()
    call = lambda: moe.layer_decode(s["x"], s["router"], moe.w13_from_packed(s["w13"]), s["w2"], k, pre_weight=s["pre"],
                                    renormalize=renorm, shared_expert=shared, post_norm=post,
                                    post_weight=s["post"] if post else None, gate=gt, gate_act=act, residual_scale=alpha)
    got = call()
    check(got, layer64(s, k, renorm, shared, s["post"] if post else False, gt, act, alpha, pre=s["pre"]))
    if T * (k + shared) <= 32:
        assert moe.last_launch_count() in (2 + post, 3 + post)
    for a, b in zip(got, call()):
        assert torch.equal(a, b)
    assert moe.device_errors() == (0, 0)


@pytest.mark.parametrize("rdt,wdt", [(F32, BF), (BF, F32), (F32, None)])
def test_types_and_strides(rdt, wdt):
    """f32 router or weights, x and out through their strides, int64 ids inside a wider tensor."""
    T, H, I, E, k = 6, 192, 64, 12, 2
    s = make(3, T, H, I, E, rdt=rdt, wdt=wdt or BF)
    s["x"] = s["x"].t().contiguous().t()
    pre = s["pre"] if wdt is not None else None
    ref = layer64(s, k, pre=pre)
    wide_r = torch.zeros(E, H + 3, dtype=rdt, device="cuda")
    wide_r[:, :H] = s["router"]
    ids = torch.full((T, 3, k), -7, dtype=torch.int64, device="cuda")
    wts = torch.full((T, 3, k), 9.0, device="cuda")
    out = torch.full((T, 2 * H), 5.0, dtype=BF, device="cuda")
    moe.layer_decode(s["x"], wide_r[:, :H], moe.w13_from_packed(s["w13"]), s["w2"], k, pre_weight=pre, out=out[:, ::2],
                     topk_ids=ids[:, 1], topk_weights=wts[:, 1])
    check((out[:, ::2], ids[:, 1], wts[:, 1]), ref)
    assert bool((out[:, 1::2] == 5.0).all()) and bool((ids[:, ::2] == -7).all()) and bool((wts[:, ::2] == 9.0).all())


def test_ties_go_to_the_lower_expert():
    s = make(9, 4, 256, 64, 16)
    s["router"][9] = s["router"][2]
    s["router"][12] = s["router"][2]
    s["router"][5] = s["router"][4]
    out, ids, p = moe.layer_decode(s["x"], s["router"], moe.w13_from_packed(s["w13"]), s["w2"], 16)
    check((out, ids, p), layer64(s, 16))
    for row in ids.tolist():
        assert row.index(2) < row.index(9) < row.index(12) and row.index(4) < row.index(5)


def test_in_place_none_and_empty():
    s = make(4, 3, 256, 64, 8)
    ref = layer64(s, 2, pre=s["pre"])
    w13 = moe.w13_from_packed(s["w13"])
    out, ids, p = moe.layer_decode(s["x"][:0], s["router"], w13, s["w2"], 2)
    assert out.shape == (0, 256) and ids.shape == (0, 2)
    x = s["x"].clone()
    check(moe.layer_decode(x, s["router"], w13, s["w2"], 2, pre_weight=s["pre"], out=x), ref)


def test_graph_and_stream():
    T, H, I, E, k = 3, 512, 128, 16, 4
    s = make(11, T, H, I, E)
    w13 = moe.w13_from_packed(s["w13"])
    ws = torch.empty(moe.layer_decode_workspace_bytes(T, H, I, E, k), dtype=torch.uint8, device="cuda")
    bufs = dict(out=torch.empty(T, H, dtype=BF, device="cuda"), topk_ids=torch.empty(T, k, dtype=torch.int32, device="cuda"),
                topk_weights=torch.empty(T, k, device="cuda"), workspace=ws)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    first = moe.layer_decode(s["x"], s["router"], w13, s["w2"], k, stream=st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = moe.layer_decode(s["x"], s["router"], w13, s["w2"], k, **bufs)
    keep = s["x"].clone()
    for seed in (1, 2):
        s["x"].copy_(make(seed, T, H, I, E)["x"])
        ws.fill_(255)
        graph.replay()
        check(got, layer64(s, k))
    s["x"].copy_(keep)
    graph.replay()
    for a, b in zip(got, first):
        assert torch.equal(a, b)


def test_mxfp4_experts():
    """The MXFP4 forward between the same two ends."""
    T, H, I, E, k = 4, 512, 256, 8, 2
    s = make(21, T, H, I, E)
    c13, s13 = moe.quantize_mxfp4(s["w13"])
    c2, s2 = moe.quantize_mxfp4(s["w2"])
    w13 = moe.w13_from_packed(c13, s13)
    out, ids, p = moe.layer_decode(s["x"], s["router"], w13, c2, k, w2_scale=s2, pre_weight=s["pre"], post_norm=True,
                                   post_weight=s["post"], residual_scale=0.5)
    _, wi, wp = route64(s["x"], s["pre"], s["router"], k, True, False)
    assert torch.equal(ids.long(), wi) and bool(((p.to(D) - wp).abs() <= 2.0 ** -20 * wp).all())
    xn, _ = moe.norm_before(s["x"], s["pre"])
    y = moe.forward(xn, w13, c2, ids, p, w2_scale=s2)
    want, _ = moe.norm_after(y, s["x"], s["post"], residual_scale=0.5)
    # (the norm's row may round the other way in a few places, which moves a 4-bit code by a step)
    e = (out.to(D) - want.to(D)).pow(2).mean().sqrt() / want.to(D).pow(2).mean().sqrt()
    assert float(e) <= 2.0 ** -6


def test_decode_steps_through_two_layers():
    """Two layers one after the other for some steps, the second's input the first's output, as a
    decoding loop runs them: the same as each layer's formula on what it got."""
    a, b = make(1, 2, 256, 64, 8), make(2, 2, 256, 64, 8)
    x = a["x"]
    for _ in range(3):
        la = moe.layer_decode(x, a["router"], moe.w13_from_packed(a["w13"]), a["w2"], 2, pre_weight=a["pre"])
        lb = moe.layer_decode(la[0], b["router"], moe.w13_from_packed(b["w13"]), b["w2"], 2, pre_weight=b["pre"],
                              post_norm=True, post_weight=b["post"])
        check(la, layer64(dict(a, x=x), 2, pre=a["pre"]))
        check(lb, layer64(dict(b, x=la[0]), 2, pre=b["pre"], post=b["post"]))
        x = lb[0]


@pytest.mark.parametrize("T,post", [(1, False), (3, True), (6, False)])
def test_steps_in_flight(T, post):
    """Many steps of changing routing in flight, the second kernel's early reads among them: the
    bits of the same steps taken one at a time."""
    H, I, E, k = 256, 512, 32, 2
    s = make(31, T, H, I, E)
    w13 = moe.w13_from_packed(s["w13"])
    ws = torch.empty(moe.layer_decode_workspace_bytes(T, H, I, E, k), dtype=torch.uint8, device="cuda")
    ids, wts = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    xs = [make(100 + i, T, H, 32, 1)["x"] for i in range(40)]
    call = lambda x, out: moe.layer_decode(x, s["router"], w13, s["w2"], k, pre_weight=s["pre"], post_norm=post, out=out,
                                           topk_ids=ids, topk_weights=wts, workspace=ws)
    one = []
    for x in xs:
        one.append((call(x, None)[0], ids.clone()))
        torch.cuda.synchronize()
    outs = [torch.empty(T, H, dtype=BF, device="cuda") for _ in xs]
    for x, o in zip(xs, outs):
        call(x, o)
    torch.cuda.synchronize()
    assert len({tuple(i.flatten().tolist()) for _, i in one}) > 10
    for (o, _), got in zip(one, outs):
        assert torch.equal(o, got)


def test_two_streams():
    """Two calls at once, a workspace each."""
    T, H, I, E, k = 2, 1024, 512, 16, 4
    s = make(41, T, H, I, E)
    w13 = moe.w13_from_packed(s["w13"])
    xs = [make(200 + i, T, H, 32, 1)["x"] for i in range(20)]
    want = [moe.layer_decode(x, s["router"], w13, s["w2"], k) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [moe.layer_decode(x, s["router"], w13, s["w2"], k, stream=streams[i % 2]) for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


def test_an_infinite_router_row_ranks_last():
    s = make(51, 2, 256, 64, 8)
    s["router"][3, 7] = float("inf")
    out, ids, p = moe.layer_decode(s["x"], s["router"], moe.w13_from_packed(s["w13"]), s["w2"], 7)
    xd = s["x"].double()
    logits = (xd / (xd.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()) @ s["router"].double().T
    logits[:, 3] = -float("inf")  # inf * x carries its rounding along as NaN, which ranks below every number
    want = torch.sort(logits, dim=-1, descending=True, stable=True)[1][:, :7]
    assert torch.equal(ids.long(), want)


@pytest.mark.parametrize("layout", ["bf16", "bf16_unaligned", "f32"])
@pytest.mark.parametrize("T", [2, 7, 12])
def test_logits_that_are_not_finite_rank_last_in_every_layout(T, layout):
    """A router row with an infinity or a NaN ranks below every number, whichever way the router is read."""
    H, E = 256, 12
    s = make(53, T, H, 64, E)
    s["router"][3, 7], s["router"][5, 8], s["router"][9, 9] = float("inf"), float("nan"), -float("inf")
    router = s["router"]
    if layout == "f32":
        router = router.float()
    elif layout == "bf16_unaligned":
        router = torch.zeros(E, H + 3, dtype=BF, device="cuda")[:, :H].copy_(router)
    out, ids, p = moe.layer_decode(s["x"], router, moe.w13_from_packed(s["w13"]), s["w2"], 8)
    finite = [e for e in range(E) if e not in (3, 5, 9)]
    _, wi, wp = route64(s["x"], None, s["router"][finite], 8, True, False)
    assert torch.equal(ids.long(), torch.tensor(finite, device="cuda")[wi])
    assert bool(((p.to(D) - wp).abs() <= 2.0 ** -20 * wp).all())
    assert bool(out.isfinite().all())
    # with more experts wanted than are finite, the others follow in the order of their indices
    _, ids, _ = moe.layer_decode(s["x"], router, moe.w13_from_packed(s["w13"]), s["w2"], E)
    assert bool((ids[:, 9:] == torch.tensor([3, 5, 9], dtype=torch.int32, device="cuda")).all())


@pytest.mark.parametrize("T,k,shared,post,gate,act", [(1, 2, False, True, None, "none"), (4, 8, False, False, "token", "sigmoid"),
                                                      (4, 3, True, True, "channel", "none"), (12, 2, False, True, "full", "tanh"),
                                                      (32, 4, True, False, None, "none")])
def test_mxfp4_experts_against_64_bit_formulas(T, k, shared, post, gate, act):
    """The experts in 4 bits between the two ends, all in 64 bits but for the roundings that the form has
    by definition (xn to bf16, xn and h to 4 bits).  Where those fall the other way a code moves by a
    step: at most the forward's own bound, 6e-2 of its largest value (twice that after a norm), and
    in root mean square 2^-6, with 2^-8 of the output besides."""
    import oracle

    H, I, E = 512, 256, 16
    s = make(61 + T, T, H, I, E, shared)
    c13, s13 = moe.quantize_mxfp4(s["w13"])
    c2, s2 = moe.quantize_mxfp4(s["w2"])
    g = torch.Generator().manual_seed(5)
    shape = {None: None, "channel": (1, H), "token": (T, 1), "full": (T, H)}[gate]
    gt = None if shape is None else torch.randn(*shape, generator=g).to(BF).cuda()
    out, ids, p = moe.layer_decode(s["x"], s["router"], moe.w13_from_packed(c13, s13), c2, k, w2_scale=s2, pre_weight=s["pre"],
                                   shared_expert=shared, post_norm=post, post_weight=s["post"] if post else None, gate=gt,
                                   gate_act=act, residual_scale=0.5)
    xn, wi, wp = route64(s["x"], s["pre"], s["router"], k, True, shared)
    assert torch.equal(ids.long(), wi) and bool(((p.to(D) - wp).abs() <= 2.0 ** -20 * wp).all())
    c, sc = c13.cpu(), s13.cpu()
    z = oracle.moe_forward(xn.to(BF).cpu(), c[:, :I], c[:, I:], c2.cpu(), wi.int().cpu(), wp.float().cpu(),
                           scales=(sc[:, :I], sc[:, I:], s2.cpu()))[0].to(D).cuda()
    if post:
        z = z / (z.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * s["post"].to(D)
    if gt is not None:
        z = z * act64(gt, act)
    want = 0.5 * s["x"].to(D) + z
    err, rms = (out.to(D) - want).abs(), lambda v: float(v.pow(2).mean().sqrt())
    assert bool((err <= (2 if post else 1) * 6e-2 * z.abs().max() + HB * want.abs()).all())
    assert rms(err) <= 2.0 ** -6 * rms(z) + HB * rms(want)
