"""The products with MXFP4 weights against a 64-bit reference on the values that codes and scales stand for: rows in bf16
and in MXFP4, sizes that fill no tile, experts without rows, rows past the last expert, NaN.

Tolerances as in training_ref: a sum of n products is off by at most n 2^-23 sum |a||b|, a result by one rounding."""
import pytest
import torch

import gpu_harness as H
import mxfp4_ref as mx
import token_dispatch_expert_amd as moe
import training_ref as ref

pytestmark = pytest.mark.gpu

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def dev():
    return H.require_gpu()


def held(shape, dev, seed, scale=1.0):
    """Codes and scales of random matrices, and their values in 64 bits; bytes of groups past the end are NaN scales."""
    g = torch.Generator(device=dev).manual_seed(seed)
    w = torch.randn(shape, generator=g, device=dev) * scale
    w *= torch.exp2(torch.randint(-3, 4, (*shape[:-1], shape[-1] // 32), generator=g, device=dev).float()).repeat_interleave(32, -1)
    codes, scales = mx.quantize(w)
    v = mx.values(codes, scales)
    groups = shape[-1] // 32
    if groups % 8:
        scales[..., -1, :, groups % 8:] = 255
    return codes, scales, v


def rows_in(kind, rows, K, dev, seed, used):
    """x as the call takes it (x, x_scales) and its values; rows from `used` on hold NaN."""
    if kind == "mxfp4":
        codes, scales, v = held((rows, K), dev, seed)
        scales[:, used:] = 255
        return codes, scales, v
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((rows, K), generator=g, device=dev).to(BF)
    x[used:] = float("nan")
    return x, None, x.double()


def product_error(x, w, counts):
    """n 2^-23 sum |a||b| for each element of the product."""
    return x.shape[1] * 2.0 ** -23 * ref.forward(x.abs(), w.abs(), counts)


COUNTS = [
    [1], [0, 3, 0], [16, 0, 1, 33], [5] * 8, [70, 1, 0, 129], [300], [0, 0, 257, 512, 1], [260, 0, 31, 700],
]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("N, K", [(8, 32), (40, 96), (264, 800), (128, 256), (1544, 1056), (520, 4128)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
def test_product(dev, counts, N, K, kind, out):
    used, E = sum(counts), len(counts)
    rows = used + 5
    w, ws, wv = held((E, N, K), dev, 1, K ** -0.5)
    x, xs, xv = rows_in(kind, rows, K, dev, 2, used)
    y, whole = ref.guarded((rows, N), out, dev)
    moe.moe_grouped_gemm_mxfp4(x, ref.offsets_of(counts, dev), w, ws, y, x_scales=xs)
    torch.cuda.synchronize()
    assert ref.guards_intact(whole, rows * N)
    assert torch.isnan(y[used:]).all()  # rows of no expert stay as they were
    want = ref.forward(xv[:used], wv, counts)
    e = product_error(xv[:used], wv, counts)
    tol = e + ref.u(out) * (want.abs() + e) + 1e-37
    assert ((y[:used].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("N, K", [(8, 32), (40, 96), (264, 800), (128, 256), (1544, 1056), (4104, 544)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
def test_input_gradient(dev, counts, N, K, out, pair):
    used, E = sum(counts), len(counts)
    rows = used + 5
    weights = [held((E, N, K), dev, 1 + i, K ** -0.5) for i in range(1 + pair)]
    dys = [rows_in("bf16", rows, N, dev, 7 + i, used)[0] for i in range(1 + pair)]
    more = dict(dy2=dys[1], w2=weights[1][0], w2_scales=weights[1][1]) if pair else {}
    dx, whole = ref.guarded((rows, K), out, dev)
    moe.moe_grouped_gemm_mxfp4_dgrad(dys[0], ref.offsets_of(counts, dev), weights[0][0], weights[0][1], dx, **more)
    torch.cuda.synchronize()
    assert ref.guards_intact(whole, rows * K)
    assert torch.isnan(dx[used:]).all()
    want = e = 0
    for (_, _, wv), dy in zip(weights, dys):
        across = wv.transpose(1, 2).contiguous()
        want = want + ref.forward(dy[:used], across, counts)
        e = e + (1 + pair) * N * 2.0 ** -23 * ref.forward(dy[:used].abs(), across.abs(), counts)
    tol = e + ref.u(out) * (want.abs() + e) + 1e-37
    assert ((dx[:used].double() - want).abs() <= tol).all()


def test_input_gradient_nan(dev):
    """A NaN group of W reaches its 32 columns of that expert's rows alone, a NaN in dy its row."""
    counts, N, K = [20, 300], 72, 544
    w, ws, _ = held((2, N, K), dev, 1)
    ws[1, 1, 7, 3] = 255                      # expert 1, row 7, columns 352 .. 383
    dy = rows_in("bf16", 320, N, dev, 2, 320)[0]
    dy[2, 70] = float("nan")
    dx = torch.zeros((320, K), device=dev)
    moe.moe_grouped_gemm_mxfp4_dgrad(dy, ref.offsets_of(counts, dev), w, ws, dx)
    want = torch.zeros_like(dx, dtype=torch.bool)
    want[2] = True
    want[20:, 352:384] = True
    assert torch.equal(torch.isnan(dx), want)


def test_input_gradient_by_differences(dev):
    """The gradient is that of the forward call: linear, so a difference along any direction is exact but for rounding."""
    counts, N, K = [9, 0, 30], 96, 160
    w, ws, wv = held((3, N, K), dev, 1, K ** -0.5)
    offsets = ref.offsets_of(counts, dev)
    x, _, xv = rows_in("bf16", 39, K, dev, 2, 39)
    dy, _, dyv = rows_in("bf16", 39, N, dev, 3, 39)
    step, _, sv = rows_in("bf16", 39, K, dev, 4, 39)
    y0, y1, dx = (torch.empty((39, n), device=dev) for n in (N, N, K))
    both = (x.float() + step.float()).to(BF)
    moe.moe_grouped_gemm_mxfp4(x, offsets, w, ws, y0)
    moe.moe_grouped_gemm_mxfp4(both, offsets, w, ws, y1)
    moe.moe_grouped_gemm_mxfp4_dgrad(dy, offsets, w, ws, dx)
    moved = both.double() - xv                # what the step became in bf16
    left = ((y1.double() - y0.double()) * dyv).sum(1)
    right = (dx.double() * moved).sum(1)
    size = ((ref.forward(both.double().abs(), wv.abs(), counts) + ref.forward(xv.abs(), wv.abs(), counts)) * dyv.abs()).sum(1)
    back = (ref.forward(dyv.abs(), wv.abs().transpose(1, 2).contiguous(), counts) * moved.abs()).sum(1)
    assert ((left - right).abs() <= (K + 1) * 2.0 ** -23 * size + (N + 1) * 2.0 ** -23 * back).all()


def silu(g):
    return g * torch.sigmoid(g)


def swiglu_reference(xv, gv, uv, counts):
    """h in 64 bits and how far fp32 arithmetic may be off before the last rounding: the sums (|silu'| <= 1.1), and the
    activation's own roundings, exp2 and reciprocal ((8 + |g|) 2^-22 of h is more than all of them)."""
    g, u = ref.forward(xv, gv, counts), ref.forward(xv, uv, counts)
    eg, eu = product_error(xv, gv, counts), product_error(xv, uv, counts)
    h = silu(g) * u
    e = 1.1 * eg * (u.abs() + eu) + silu(g).abs() * eu + (8 + g.abs()) * 2.0 ** -22 * h.abs()
    return h, e


def check_mxfp4(codes, scales, h, e):
    """codes and scales hold h (known to within e): the scale is the smallest that holds the group, each code the nearest."""
    got = mx.values(codes, scales)
    b = mx.rows_of(scales, h.shape[1] // 32).long()
    s = mx.power(b - 127)
    g, eg = h.reshape(*s.shape, 32), e.reshape(*s.shape, 32)
    low, high = (g.abs() - eg).amax(-1), (g.abs() + eg).amax(-1)
    assert (low <= 6 * s).all()
    assert ((high > 3 * s) | ((b == 2) & (high <= 6 * s)) | ((b == 127) & (low <= 0))).all()
    v = (g.abs() + eg) / s[..., None]
    half = torch.where(v <= 2, 0.25, torch.where(v <= 4, 0.5, 1.0)) * s[..., None]
    assert ((got.reshape(g.shape) - g).abs() <= half + eg * (1 + 1e-6)).all()


@pytest.mark.parametrize("kind, out", [("bf16", "bf16"), ("bf16", "mxfp4"), ("mxfp4", "bf16"), ("mxfp4", "mxfp4")])
@pytest.mark.parametrize("f, d", [(32, 32), (96, 288), (288, 800), (544, 1056), (1536, 2048)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
def test_swiglu(dev, counts, f, d, kind, out):
    used, E = sum(counts), len(counts)
    rows = used + 3
    w, ws, wv = held((E, f, d), dev, 1, d ** -0.5)
    v, vs, vv = held((E, f, d), dev, 3, d ** -0.5)
    x, xs, xv = rows_in(kind, rows, d, dev, 2, used)
    offsets = ref.offsets_of(counts, dev)
    want, e = swiglu_reference(xv[:used], wv, vv, counts)
    if out == "bf16":
        h, whole = ref.guarded((rows, f), BF, dev)
        moe.moe_grouped_swiglu_mxfp4(x, offsets, w, ws, v, vs, h, x_scales=xs)
        torch.cuda.synchronize()
        assert ref.guards_intact(whole, rows * f) and torch.isnan(h[used:]).all()
        assert ((h[:used].double() - want).abs() <= e + ref.u(BF) * (want.abs() + e) + 1e-37).all()
        return
    codes, scales = moe.mxfp4_buffers((rows, f), device=dev)
    codes.fill_(0xAB)
    scales.fill_(0xAB)
    moe.moe_grouped_swiglu_mxfp4(x, offsets, w, ws, v, vs, codes, x_scales=xs, h_scales=scales)
    torch.cuda.synchronize()
    assert (codes[used:] == 0xAB).all() and (scales[:, used:] == 0xAB).all()
    if f // 32 % 8:
        assert (scales[-1, :, f // 32 % 8:] == 0xAB).all()
    check_mxfp4(codes[:used], scales[:, :used], want, e)


def test_swiglu_far_gates(dev):
    """Gates far below zero: the sigmoid is no normal fp32 number, u is large."""
    d = f = 32
    x = torch.zeros((1, d), device=dev)
    x[0, 0], x[0, 1] = 1.0, 1.0
    wg, wu = torch.zeros((1, f, d), device=dev), torch.zeros((1, f, d), device=dev)
    # each row of W is a group of its own: one element a power of two (times 1.5) is held exactly
    gates = [-64.0, -96.0, -128.0, -192.0, -256.0, -384.0, 96.0, 0.0] * 4
    wg[0, :, 0] = torch.tensor(gates)
    wu[0, :, 1] = 2.0 ** 120
    (cg, sg), (cu, su) = mx.quantize(wg), mx.quantize(wu)
    h = torch.empty((1, f), dtype=BF, device=dev)
    moe.moe_grouped_swiglu_mxfp4(x.to(BF), ref.offsets_of([1], dev), cg, sg, cu, su, h)
    g = torch.tensor(gates, dtype=torch.float64, device=dev)
    want = (g * torch.sigmoid(g) * 2.0 ** 120)
    # the power's error is |g| 2^-24 of its exponent, and those of exp2 and the reciprocal
    tol = (ref.u(BF) + (8 + g.abs()) * 2.0 ** -22) * want.abs() + 2.0 ** -134
    assert ((h[0].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_nan(dev, kind):
    """A NaN scale of a weight group makes that output column NaN, one of a row that row; nothing else is."""
    counts, N, K = [20, 300], 96, 544
    w, ws, wv = held((2, N, K), dev, 1)
    x, xs, xv = rows_in(kind, 320, K, dev, 2, 320)
    ws[1, 1, 7, 3] = 255          # expert 1, row 7, group 11
    if kind == "mxfp4":
        xs[0, 2, 5] = 255
    else:
        x[2, 170] = float("nan")
    y = torch.zeros((320, N), device=dev)
    moe.moe_grouped_gemm_mxfp4(x, ref.offsets_of(counts, dev), w, ws, y, x_scales=xs)
    want = torch.zeros_like(y, dtype=torch.bool)
    want[2] = True
    want[20:, 7] = True
    assert torch.equal(torch.isnan(y), want)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_ends_of_the_scales(dev, kind):
    """Small and large scales that meet: products within fp32 come out right."""
    N, K = 64, 256
    for sw, sx in ((2, 250), (250, 2), (3, 130), (200, 60)):
        g = torch.Generator(device=dev).manual_seed(sw)
        w = torch.randint(0, 256, (1, N, K // 2), generator=g, device=dev, dtype=U8)
        ws = torch.full((1, 1, N, 8), sw, dtype=U8, device=dev)
        codes = torch.randint(0, 256, (40, K // 2), generator=g, device=dev, dtype=U8)
        scales = torch.full((1, 40, 8), sx, dtype=U8, device=dev)
        xv = mx.values(codes, scales)
        y = torch.empty((40, N), device=dev)
        x, xs = (codes, scales) if kind == "mxfp4" else (xv.to(BF), None)
        moe.moe_grouped_gemm_mxfp4(x, ref.offsets_of([40], dev), w, ws, y, x_scales=xs)
        wv = mx.values(w, ws)
        want = ref.forward(xv, wv, [40])
        tol = product_error(xv, wv, [40]) + ref.u(F32) * want.abs() + 1e-37
        assert ((y.double() - want).abs() <= tol).all(), (sw, sx)


def test_no_rows(dev):
    w, ws, _ = held((3, 64, 96), dev, 1)
    offsets = torch.zeros(4, dtype=torch.int32, device=dev)
    moe.moe_grouped_gemm_mxfp4(torch.empty((0, 96), dtype=BF, device=dev), offsets, w, ws, torch.empty((0, 64), device=dev))
    y = torch.full((5, 64), 3.0, device=dev)
    moe.moe_grouped_gemm_mxfp4(torch.ones((5, 96), dtype=BF, device=dev), offsets, w, ws, y)
    assert (y == 3).all()


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_repeated_and_captured(dev, kind):
    """Repeated calls are bit-identical; a captured call replays on what its inputs hold then, beside eager calls."""
    counts, N, K = [3, 0, 40, 90], 264, 800
    w, ws, wv = held((4, N, K), dev, 1)
    offsets = ref.offsets_of(counts, dev)
    x, xs, xv = rows_in(kind, 133, K, dev, 2, 133)
    y, again = torch.empty((133, N), device=dev), torch.empty((133, N), device=dev)
    moe.moe_grouped_gemm_mxfp4(x, offsets, w, ws, y, x_scales=xs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_grouped_gemm_mxfp4(x, offsets, w, ws, again, x_scales=xs)
    for i in range(3):
        nx, ns, _ = rows_in(kind, 133, K, dev, 10 + i, 133)
        x.copy_(nx)
        if xs is not None:
            xs.copy_(ns)
        again.zero_()
        graph.replay()
        moe.moe_grouped_gemm_mxfp4(x, offsets, w, ws, y, x_scales=xs)
        torch.cuda.synchronize()
        assert torch.equal(y, again)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_offsets_past_32_bits(dev, kind):
    """Rows, weights and results of more than 2^31 bytes, and weights of more than 2^32 elements: the last expert's last row."""
    E, N, K = 150, 4104, 7168   # 4.4e9 elements
    counts = [0] * E
    counts[0], counts[-1] = 300000, 40
    w = torch.zeros((E, N, K // 2), dtype=U8, device=dev)
    ws = torch.zeros((E, K // 256, N, 8), dtype=U8, device=dev)
    last, lasts, wv = held((1, N, K), dev, 1, K ** -0.5)
    w[-1], ws[-1] = last[0], lasts[0]
    tail, tails, xv = rows_in(kind, 40, K, dev, 2, 40)
    rows = sum(counts)
    if kind == "mxfp4":
        x = torch.zeros((rows, K // 2), dtype=U8, device=dev)
        xs = torch.zeros((K // 256, rows, 8), dtype=U8, device=dev)
        x[-40:], xs[:, -40:] = tail, tails
    else:
        x, xs = torch.zeros((rows, K), dtype=BF, device=dev), None
        x[-40:] = tail
    y = torch.full((rows, N), 3.0, dtype=F32, device=dev)
    moe.moe_grouped_gemm_mxfp4(x, ref.offsets_of(counts, dev), w, ws, y, x_scales=xs)
    want = ref.forward(xv, wv, [40])
    tol = product_error(xv, wv, [40]) + ref.u(F32) * want.abs() + 1e-37
    assert ((y[-40:].double() - want).abs() <= tol).all()
    assert (y[:300000] == 0).all()
