"""The 4-bit linear layer and its quantiser against plain 64-bit formulas.

The quantiser's codes and scales have to be the exact ones.  The product's tolerance: with the
exact codes every term is exact up to the scales' product (2^-23 relative); the fp32 sum of at
most K/16 + 40 partial sums loses below one step (2^-23) of S = sum |terms| at each addition
(the tensor core may cut where a fused multiply-add rounds), the float scales 2^-22 |out|, and
the output rounds once: |out - ref| <= (K/16 + 48) 2^-23 S + 2^-8 |ref|."""

import pytest
import torch

import mixture_experts_layer_46_b200 as moe

pytestmark = pytest.mark.gpu

BF, F32, D = torch.bfloat16, torch.float32, torch.float64
GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=D)
E4M3 = torch.tensor([(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127],
                    dtype=D)


def nearest(v, table):
    """Index of the table's number nearest to v >= 0, the even index on a tie."""
    table = table.to(v.device)
    i = torch.bucketize(v, (table[1:] + table[:-1]) / 2)  # a border goes down
    up = (i + 1).clamp(max=len(table) - 1)
    tie = (i % 2 == 1) & (v == (table[i] + table[up]) / 2)
    return torch.where(tie, up, i)


def nv64(x, G):
    """codes [R, K] (0 .. 15), scale codes [R, K/16], values: of the definition in 64 bits."""
    R, K = x.shape
    b, G = x.to(D).reshape(R, K // 16, 16), G.to(D)
    s = nearest(b.abs().amax(-1) / (6.0 * G), E4M3)
    unit = E4M3.to(x.device)[s] * G
    q = torch.where(unit[..., None] > 0, b.abs() / unit[..., None].clamp(min=1e-300), torch.zeros_like(b))
    c = nearest(q.clamp(max=6.0), GRID)
    v = GRID.to(x.device)[c] * torch.sign(b) * unit[..., None]
    code = c + 8 * ((b < 0) & (unit[..., None] > 0))
    return code.reshape(R, K), s, v.reshape(R, K)


def mx64(x):
    R, K = x.shape
    b = x.to(D).reshape(R, K // 32, 32)
    e = torch.frexp(b.abs().amax(-1))[1].to(D) - 3
    unit = torch.exp2(e.clamp(-127, 127))
    v = GRID.to(x.device)[nearest((b.abs() / unit[..., None]).clamp(max=6.0), GRID)] * torch.sign(b) * unit[..., None]
    return v.reshape(R, K)


def unpack(codes):
    return torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1).long()


def rows(seed, T, K, dt=BF, pad=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K + pad, generator=g) * torch.exp(torch.randn(T, 1, generator=g)) * scale
    x[:, :: max(1, K // 5)] *= 8.0
    return x.to(dt).cuda()[:, :K]


def check(out, xv, wv):
    ref, S = xv @ wv.T, xv.abs() @ wv.abs().T
    K = xv.shape[1]
    room = (K / 16 + 48) * 2.0 ** -23 * S + 2.0 ** -8 * ref.abs()
    err = (out.to(D) - ref).abs()
    assert out.dtype == BF and out.shape == ref.shape
    assert bool((err <= room).all()), f"{int((err > room).sum())} of {err.numel()} off, worst {(err / room.clamp(min=1e-300)).max():.3g} x the room"


def weight(seed, N, K, form):
    w = rows(seed, N, K, F32, scale=K ** -0.5)
    if form == "nv":
        codes, sf, G = moe.quantize_nvfp4(w)
        return codes, sf, G, nv64(w, G)[2]
    codes, sf = moe.quantize_mxfp4(w)
    return codes, sf, None, mx64(w)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("R,K,pad", [(1, 32, 0), (7, 96, 0), (33, 4096, 0), (128, 160, 8), (5, 64, 3)])
def test_quantize(R, K, pad, dt):
    x = rows(R + K, R, K, dt, pad)
    codes, sf, G = moe.quantize_nvfp4(x)
    want_c, want_s, _ = nv64(x, G)
    assert torch.equal(sf.view(torch.uint8).long(), want_s)
    assert torch.equal(unpack(codes), want_c)


@pytest.mark.parametrize("G", [2.0 ** -9, 2.0 ** -9 * 1.1, 1.0, 1e-3, 1e-20, 3e-5])
def test_quantize_borders(G):
    """Values on and next to every border of codes and scales, blocks of zeros, tiny and huge ones."""
    step = torch.tensor([G], dtype=F32)
    blocks = []
    for s in (1.0, 1.125, 0.015625, 240.0, 448.0, 2.0 ** -9):
        unit = s * step.to(D)
        for m in (1.0, 1 - 2.0 ** -23, 1 + 2.0 ** -23):
            b = [6.0] + [float(v) for v in (GRID[1:] + GRID[:-1]) / 2] + [-float(v) for v in GRID]
            blocks.append((torch.tensor(b, dtype=D) * unit * m).float())
    for i in (3, 17, 60, 100, 125):  # block maxima half way between two scales
        mid = (E4M3[i] + E4M3[i + 1]) / 2 * 6.0
        for m in (1.0, 1 - 2.0 ** -22, 1 + 2.0 ** -22):
            blocks.append(torch.linspace(-1, 1, 16) * (mid * step.to(D) * m).float())
    blocks += [torch.zeros(16), torch.full((16,), 1e-38), torch.full((16,), 3e38), torch.full((16,), -1e4)]
    if len(blocks) % 2:
        blocks.append(torch.zeros(16))
    x = torch.stack(blocks).reshape(-1, 32).cuda()
    codes, sf, _ = moe.quantize_nvfp4(x, step.cuda())
    want_c, want_s, _ = nv64(x, step.cuda())
    assert torch.equal(sf.view(torch.uint8).long(), want_s)
    assert torch.equal(unpack(codes), want_c)


def test_quantize_zero_scale_gives_zeros():
    x = rows(3, 4, 64)
    for G in (0.0, -1.0):
        codes, sf, _ = moe.quantize_nvfp4(x, torch.tensor([G], device="cuda"))
        assert int(codes.count_nonzero()) == 0 and int(sf.view(torch.uint8).count_nonzero()) == 0


SHAPES = [(1, 1, 32), (1, 64, 128), (1, 4096, 4096), (2, 77, 640), (3, 1000, 4096), (4, 33, 2976),      # by rows
          (5, 64, 128), (5, 1, 32), (16, 333, 4096), (14, 999, 992), (7, 2048, 2048),
          (17, 64, 128), (40, 1, 32), (31, 333, 96), (128, 224, 256), (129, 450, 288), (256, 2048, 512),  # on pairs
          (257, 97, 1184), (1023, 1024, 4096), (700, 8192, 1024), (2500, 1111, 384), (16, 1024, 4096),
          (2049, 8000, 2048), (300, 8111, 1536), (515, 8190, 2080)]


@pytest.mark.parametrize("form", ["nv", "mx"])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_linear(T, N, K, form):
    x = rows(T + N, T, K)
    codes, sf, wg, wv = weight(K + N, N, K, form)
    xg = (x.float().abs().max() / 2688.0).reshape(1) if form == "nv" else None
    out = moe.linear_fp4(x, codes, sf, x_global=xg, w_global=wg)
    check(out, nv64(x, xg)[2] if form == "nv" else mx64(x), wv)
    assert torch.equal(out, moe.linear_fp4(x, codes, sf, x_global=xg, w_global=wg))
    assert moe.last_launch_count() == (1 if T <= 16 and (T - 1) * N * K <= (1 << 23) + 5120 * K else 2)


@pytest.mark.parametrize("form", ["nv", "mx"])
@pytest.mark.parametrize("T", [3, 140])
def test_linear_strides(T, form):
    """f32 x through its strides, an output inside a wider one, weights and scales inside wider rows."""
    N, K = 130, 416
    x = rows(1, K, T + 3, F32).t()[:T]
    wide = rows(2, N, K, F32, scale=0.05)
    if form == "nv":
        codes, sf, wg = moe.quantize_nvfp4(wide)
        wv, xg = nv64(wide, wg)[2], (x.abs().max() / 2688.0).reshape(())
        xv = nv64(x, xg)[2]
    else:
        codes, sf = moe.quantize_mxfp4(wide)
        wg = xg = None
        wv, xv = mx64(wide), mx64(x)
    big = torch.zeros(N, codes.shape[1] + 48, dtype=torch.uint8, device="cuda")
    big[:, 16: 16 + codes.shape[1]] = codes
    bsf = torch.zeros(sf.shape[1], N + 5, dtype=torch.uint8, device="cuda")
    bsf[:, :N] = sf.view(torch.uint8).t()
    for buf, view in ((torch.full((T, N + 7), 7.0, dtype=BF, device="cuda"), lambda b: b[:, :N]),
                      (torch.full((T + 1, 2 * N), 7.0, dtype=BF, device="cuda"), lambda b: b[:T, ::2]),
                      (torch.full((T, N + 14), 7.0, dtype=BF, device="cuda"), lambda b: b[:, 8: 8 + N])):
        out = view(buf)
        moe.linear_fp4(x, big[:, 16: 16 + codes.shape[1]], bsf.t()[:N].view(sf.dtype), x_global=xg, w_global=wg, out=out)
        check(out, xv, wv)
        mask = torch.ones_like(buf, dtype=torch.bool)
        view(mask).fill_(False)
        assert bool((buf[mask] == 7.0).all())


def test_linear_none_and_empty():
    codes, sf, wg, wv = weight(1, 64, 64, "nv")
    assert moe.linear_fp4(rows(1, 0, 64), codes, sf, x_global=wg).shape == (0, 64)
    x = rows(2, 9, 64)
    xg = torch.tensor([0.004], device="cuda")  # larger values saturate
    check(moe.linear_fp4(x, codes, sf, x_global=xg), nv64(x, xg)[2], wv / wg.to(D))


def test_linear_graph_and_stream():
    codes, sf, wg, wv = weight(1, 300, 256, "nv")
    for T in (2, 70):
        x = rows(T, T, 256)
        xg = (x.float().abs().max() / 2688.0).reshape(1)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        on_stream = moe.linear_fp4(x, codes, sf, x_global=xg, w_global=wg, stream=s)
        s.synchronize()
        ws = torch.empty(max(1, moe.linear_fp4_workspace_bytes(T, 300, 256, moe.SCALE_E4M3_16)), dtype=torch.uint8, device="cuda")
        out = torch.empty(T, 300, dtype=BF, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.linear_fp4(x, codes, sf, x_global=xg, w_global=wg, out=out, workspace=ws)
        for seed in (5, 6):
            x.copy_(rows(seed, T, 256))
            ws.fill_(255)  # nothing is kept from one call for the next
            graph.replay()
            check(out, nv64(x, xg)[2], wv)
        x.copy_(rows(T, T, 256))
        graph.replay()
        assert torch.equal(out, on_stream)


def test_linear_two_streams():
    """Calls at once on two streams, a workspace each (made by the call on its stream)."""
    codes, sf, wg, _ = weight(1, 512, 512, "nv")
    xs = [rows(i, 3 + 40 * (i % 3), 512) for i in range(12)]
    xg = torch.tensor([0.01], device="cuda")
    want = [moe.linear_fp4(x, codes, sf, x_global=xg, w_global=wg) for x in xs]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [moe.linear_fp4(x, codes, sf, x_global=xg, w_global=wg, stream=st[i % 2]) for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_linear_far_offsets():
    """An output of more than 2^31 elements: its last rows are the ones a small call gives."""
    T, N, K = 1 << 19, 4104, 64
    codes, sf, wg, _ = weight(5, N, K, "nv")
    tail = rows(6, 300, K)
    x = torch.zeros(T, K, dtype=BF, device="cuda")
    x[-300:] = tail
    xg = (tail.float().abs().max() / 2688.0).reshape(1)
    out = moe.linear_fp4(x, codes, sf, x_global=xg, w_global=wg)
    assert out.numel() > 1 << 31
    assert torch.equal(out[-300:], moe.linear_fp4(tail, codes, sf, x_global=xg, w_global=wg))
    assert int(out[: T - 300].count_nonzero()) == 0


def test_quantise_then_multiply():
    """The activations' quantiser and the linear layer agree: a layer of the quantised values alone."""
    x, w = rows(1, 130, 256), rows(2, 200, 256, F32)
    xc, xs, xg = moe.quantize_nvfp4(x)
    wc, ws, wg = moe.quantize_nvfp4(w)
    code = unpack(xc)
    v = GRID.cuda()[code & 7] * torch.where(code >= 8, -1.0, 1.0) * (xs.double().repeat_interleave(16, 1) * xg.double())
    check(moe.linear_fp4(x, wc, ws, x_global=xg, w_global=wg), v, nv64(w, wg)[2])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("form", ["nv", "mx"])
@pytest.mark.parametrize("T", [2, 150])
def test_linear_non_finite(T, form, dt):
    """A NaN in a token makes its outputs NaN and no other's; an infinity saturates as the rule says."""
    N, K = 72, 320
    x = rows(1, T, K, dt)
    codes, sf, wg, wv = weight(2, N, K, form)
    xg = (x.float().abs().max() / 2688.0).reshape(1) if form == "nv" else None
    clean = moe.linear_fp4(x, codes, sf, x_global=xg, w_global=wg)
    bad = x.clone()
    bad[1, 37] = float("nan")
    out = moe.linear_fp4(bad, codes, sf, x_global=xg, w_global=wg)
    assert bool(out[1].isnan().all())
    keep = torch.arange(T, device="cuda") != 1
    assert torch.equal(out[keep], clean[keep])
    if form == "nv":
        bad[1, 37] = float("inf")
        big = bad.clone()
        big[1, 37] = 1e30  # far beyond scale 448 and code 6: the same codes
        assert torch.equal(moe.linear_fp4(bad, codes, sf, x_global=xg, w_global=wg),
                           moe.linear_fp4(big, codes, sf, x_global=xg, w_global=wg))
        assert bool(moe.quantize_nvfp4(torch.full((1, 32), float("nan"), dtype=dt, device="cuda"), xg)[1].float().isnan().all())


@pytest.mark.parametrize("T", [1, 2, 4, 40, 300])
def test_linear_nan_scale_in_the_weight(T):
    """The e8m0 code 255 is NaN: every token's output of that weight row is, in both forms of the
    kernel, and no other."""
    N, K = 72, 320
    x = rows(1, T, K)
    codes, sf, _, _ = weight(2, N, K, "mx")
    clean = moe.linear_fp4(x, codes, sf)
    sf[5, 3] = 255
    out = moe.linear_fp4(x, codes, sf)
    assert bool(out[:, 5].isnan().all())
    keep = torch.arange(N, device="cuda") != 5
    assert torch.equal(out[:, keep], clean[:, keep])


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("ex,ew", [(100, 100), (125, -60), (-100, 90), (-127, 120), (-60, -50), (120, -127)])
def test_linear_far_scales(T, ex, ew):
    """Scales whose product, or either with a partial sum, leaves fp32's range: a block whose products
    cancel adds nothing, and the others are exact powers of two times their sums."""
    K = 64
    codes = torch.full((2, K // 2), 0xA2, dtype=torch.uint8, device="cuda")  # 1, -1, 1, -1, ...: cancels
    codes[1] = 0x22
    codes[1, 16:] = 0                                                        # row 1: 32 ones, then zeros
    sf = torch.full((2, 2), ew + 127, dtype=torch.uint8, device="cuda")
    x = torch.full((T, K), 4.0, dtype=F32, device="cuda") * 2.0 ** max(ex, -126)
    x *= 2.0 ** (ex - max(ex, -126))                                         # scale 2^ex, code 4 = the sixth
    out = moe.linear_fp4(x, codes, sf)
    assert bool((out[:, 0] == 0).all())
    want = torch.tensor(128.0, dtype=D) * 2.0 ** (ex + ew)
    assert bool((out[:, 1].cpu() == want.to(BF)).all())


@pytest.mark.parametrize("form", ["nv", "mx"])
@pytest.mark.parametrize("T,N,K,launches", [(1, 8, 72800, 1), (1, 8, 72832, 2), (2, 5, 36384, 1), (2, 5, 36416, 2),
                                            (3, 7, 24256, 1), (3, 7, 24288, 2), (4, 24, 18176, 1), (4, 24, 18208, 2),
                                            (16, 3, 18176, 1), (16, 3, 18208, 2)])
def test_linear_on_both_sides_of_the_one_launch_forms_shared_memory(T, N, K, launches, form):
    x = rows(T + N, T, K)
    codes, sf, wg, wv = weight(K + N, N, K, form)
    xg = (x.float().abs().max() / 2688.0).reshape(1) if form == "nv" else None
    out = moe.linear_fp4(x, codes, sf, x_global=xg, w_global=wg)
    assert moe.last_launch_count() == launches
    check(out, nv64(x, xg)[2] if form == "nv" else mx64(x), wv)
