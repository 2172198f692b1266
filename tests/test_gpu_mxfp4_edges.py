"""The MXFP4 products at the ends of what they take: the widest rows and weights, the most experts, the smallest and largest
scales, infinities and NaN. References and tolerances as in test_gpu_mxfp4_products."""
import pytest
import torch

import gpu_harness as H
import mxfp4_ref as mx
import token_dispatch_expert_amd as moe
import training_ref as ref
from test_gpu_mxfp4_products import check_mxfp4, held, product_error, rows_in, swiglu_reference

pytestmark = pytest.mark.gpu

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
WIDEST = 1 << 20


@pytest.fixture(scope="module")
def dev():
    return H.require_gpu()


def sparse(t, dim, n=160):
    """t with all but n elements along `dim` set to zero, the first and last 32 among the others: sums of n products."""
    size = t.shape[dim]
    g = torch.Generator().manual_seed(size)
    keep = torch.zeros(size, dtype=torch.bool)
    keep[torch.randint(0, size, (n - 64,), generator=g)] = True
    keep[:32] = keep[-32:] = True
    shape = [1] * t.dim()
    shape[dim] = size
    return torch.where(keep.to(t.device).view(shape), t, torch.zeros_like(t)), n


def close(got, want, e):
    assert got.shape == want.shape
    assert ((got.double() - want).abs() <= e + ref.u(got.dtype) * (want.abs() + e) + 1e-37).all()


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("counts", [[2, 7], [20, 300]], ids=lambda c: "-".join(map(str, c)))
def test_longest_contraction(dev, counts, kind):
    R, N, K = sum(counts), 32, WIDEST
    w, ws, wv = held((2, N, K), dev, 1)
    v, vs, vv = held((2, N, K), dev, 3, 1e-3)
    x, n = sparse(torch.randn((R, K), device=dev).to(BF), 1)
    xs, xv = None, x.double()
    if kind == "mxfp4":
        x, xs = mx.quantize(x)
        xv = mx.values(x, xs)
    offsets = ref.offsets_of(counts, dev)
    y = torch.full((R, N), float("nan"), device=dev)
    moe.moe_grouped_gemm_mxfp4(x, offsets, w, ws, y, x_scales=xs)
    close(y, ref.forward(xv, wv, counts), n * 2.0 ** -23 * ref.forward(xv.abs(), wv.abs(), counts))
    h = torch.full((R, N), float("nan"), dtype=BF, device=dev)
    moe.moe_grouped_swiglu_mxfp4(x, offsets, w, ws, v, vs, h, x_scales=xs)
    want, e = swiglu_reference(xv, wv, vv, counts)  # (its bound is that of K products: more than n need)
    close(h, want, e)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("counts", [[2, 7], [20, 300]], ids=lambda c: "-".join(map(str, c)))
def test_widest_results(dev, counts, kind):
    R, N, K = sum(counts), WIDEST, 32
    w, ws, wv = held((2, N, K), dev, 1)
    x, xs, xv = rows_in(kind, R, K, dev, 2, R)
    y = torch.full((R, N), float("nan"), device=dev)
    moe.moe_grouped_gemm_mxfp4(x, ref.offsets_of(counts, dev), w, ws, y, x_scales=xs)
    close(y, ref.forward(xv, wv, counts), product_error(xv, wv, counts))


@pytest.mark.parametrize("counts", [[2, 7], [20, 300]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("N, K", [(WIDEST, 32), (8, WIDEST)])
def test_widest_gradients(dev, counts, N, K):
    R, offsets = sum(counts), ref.offsets_of(counts, dev)
    pairs = [held((2, N, K), dev, 1 + i) for i in range(2)]
    dys = [sparse(torch.randn((R, N), device=dev).to(BF), 1) if N > 1000 else (torch.randn((R, N), device=dev).to(BF), N) for _ in range(2)]
    dx = torch.full((R, K), float("nan"), device=dev)
    moe.moe_grouped_gemm_mxfp4_dgrad(dys[0][0], offsets, pairs[0][0], pairs[0][1], dx, dy2=dys[1][0], w2=pairs[1][0],
                                     w2_scales=pairs[1][1])
    want = e = 0
    for (dy, n), (_, _, wv) in zip(dys, pairs):
        want = want + ref.dgrad(dy, wv, counts)
        e = e + 2 * n * 2.0 ** -23 * ref.dgrad(dy.abs(), wv.abs(), counts)
    close(dx, want, e)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("rows", [700, 9000])
def test_most_experts(dev, rows, kind):
    E, N, K = 1024, 64, 288
    g = torch.Generator().manual_seed(rows)
    counts = torch.bincount(torch.randint(0, E, (rows,), generator=g), minlength=E).tolist()
    counts[0], counts[-1] = 0, counts[-1] + counts[0]
    offsets = ref.offsets_of(counts, dev)
    w, ws, wv = held((E, N, K), dev, 1, K ** -0.5)
    v, vs, vv = held((E, N, K), dev, 3, K ** -0.5)
    x, xs, xv = rows_in(kind, rows, K, dev, 2, rows)
    y = torch.full((rows, N), float("nan"), device=dev)
    moe.moe_grouped_gemm_mxfp4(x, offsets, w, ws, y, x_scales=xs)
    close(y, ref.forward(xv, wv, counts), product_error(xv, wv, counts))
    codes, scales = moe.mxfp4_buffers((rows, N), device=dev)
    moe.moe_grouped_swiglu_mxfp4(x, offsets, w, ws, v, vs, codes, x_scales=xs, h_scales=scales)
    check_mxfp4(codes, scales, *swiglu_reference(xv, wv, vv, counts))
    dy = rows_in("bf16", rows, N, dev, 4, rows)[0]
    dx = torch.full((rows, K), float("nan"), device=dev)
    moe.moe_grouped_gemm_mxfp4_dgrad(dy, offsets, w, ws, dx)
    close(dx, ref.dgrad(dy, wv, counts), N * 2.0 ** -23 * ref.dgrad(dy.abs(), wv.abs(), counts))


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("counts", [[1], [3, 14], [40], [300, 257]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("sw, sx", [(0, 252), (1, 251), (0, 200), (252, 1)])
def test_smallest_scales(dev, counts, kind, sw, sx):
    """Weights (or 4-bit rows) of scale 2^-127, whose values are no normal numbers, meet large ones."""
    E, R, N, K = len(counts), sum(counts), 264, 544
    g = torch.Generator(device=dev).manual_seed(sw)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device=dev, dtype=U8)
    ws = torch.full((E, -(-K // 256), N, 8), sw, dtype=U8, device=dev)
    codes = torch.randint(0, 256, (R, K // 2), generator=g, device=dev, dtype=U8)
    scales = torch.full((-(-K // 256), R, 8), sx, dtype=U8, device=dev)
    xv, wv = mx.values(codes, scales), mx.values(w, ws)
    x, xs = (codes, scales) if kind == "mxfp4" else (xv.to(BF), None)
    if kind == "bf16":
        assert torch.equal(x.double(), xv)
    y = torch.full((R, N), float("nan"), device=dev)
    moe.moe_grouped_gemm_mxfp4(x, ref.offsets_of(counts, dev), w, ws, y, x_scales=xs)
    close(y, ref.forward(xv, wv, counts), product_error(xv, wv, counts))


def same_kind(got, want):
    """Finite, infinite of either sign or NaN in the same places."""
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.where(torch.isinf(got), got.sign(), 0), torch.where(torch.isinf(want), want.sign(), 0).to(got.dtype))


@pytest.mark.parametrize("counts", [[1], [3, 14], [40], [300, 257]], ids=lambda c: "-".join(map(str, c)))
def test_infinite_rows(dev, counts):
    """An infinity in a row meets every weight of its column: infinite where that is not zero, NaN where it is."""
    E, R, N, K = len(counts), sum(counts), 264, 800
    w, ws, wv = held((E, N, K), dev, 1)
    x, _, _ = rows_in("bf16", R, K, dev, 2, R)
    x[0, 3], x[R - 1, K - 1] = float("inf"), -float("inf")
    dy, _, _ = rows_in("bf16", R, N, dev, 3, R)
    dy[0, N - 1] = float("inf")
    offsets = ref.offsets_of(counts, dev)
    y, dx = torch.zeros((R, N), device=dev), torch.zeros((R, K), device=dev)
    moe.moe_grouped_gemm_mxfp4(x, offsets, w, ws, y)
    moe.moe_grouped_gemm_mxfp4_dgrad(dy, offsets, w, ws, dx)
    assert (wv == 0).any()

    def by_rows(a, weights):  # a row at a time: library products need not treat infinities so
        a = a.double()
        out = torch.zeros((R, weights.shape[1]), dtype=torch.float64, device=dev)
        for e, p, q in ref.spans(counts):
            for r in range(p, q):
                if not torch.isfinite(a[r]).all():
                    out[r] = (a[r] * weights[e]).sum(1)
        return out

    same_kind(y, by_rows(x, wv))
    same_kind(dx, by_rows(dy, wv.transpose(1, 2)))


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("counts", [[1, 2], [3, 14], [20, 300]], ids=lambda c: "-".join(map(str, c)))
def test_swiglu_nan(dev, counts, kind):
    """A NaN group of gate or up reaches its column of h for that expert's rows, of h in 4 bits the group of 32 around it; a NaN in a
    row all of it; nothing else."""
    E, R, f, d = 2, sum(counts), 544, 800
    a = counts[0]
    w, ws, _ = held((E, f, d), dev, 1, d ** -0.5)
    v, vs, _ = held((E, f, d), dev, 3, d ** -0.5)
    ws[0, 1, 7, 3] = 255        # expert 0, column 7
    vs[1, 3, 540, 0] = 255      # expert 1, column 540, its last group
    x, xs, _ = rows_in(kind, R, d, dev, 2, R)
    if kind == "mxfp4":
        xs[0, R - 1, 5] = 255
    else:
        x[R - 1, d - 1] = float("nan")
    offsets = ref.offsets_of(counts, dev)
    h = torch.zeros((R, f), dtype=BF, device=dev)
    moe.moe_grouped_swiglu_mxfp4(x, offsets, w, ws, v, vs, h, x_scales=xs)
    want = torch.zeros_like(h, dtype=torch.bool)
    want[:a, 7] = want[a:, 540] = want[R - 1] = True
    assert torch.equal(torch.isnan(h), want)
    codes, scales = moe.mxfp4_buffers((R, f), device=dev)
    moe.moe_grouped_swiglu_mxfp4(x, offsets, w, ws, v, vs, codes, x_scales=xs, h_scales=scales)
    want[:a, :32] = want[a:, 512:544] = True
    assert torch.equal(torch.isnan(mx.values(codes, scales)), want)
    assert (codes.view(R, f // 32, 16)[want.view(R, f // 32, 32)[:, :, 0]] == 0).all()
