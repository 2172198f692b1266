"""Quantisation to MXFP4 and back against the 64-bit reference: codes and scales are compared bit for bit."""
import pytest
import torch

import gpu_harness as H
import mxfp4_ref as mx
import token_dispatch_expert_amd as moe

pytestmark = pytest.mark.gpu

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
MARK = 0xAB


@pytest.fixture(scope="module")
def dev():
    return H.require_gpu()


def marked(shape, dev, pad=256):
    """A byte tensor inside a larger one of marks: (view, whole)."""
    n = 1
    for s in shape:
        n *= s
    whole = torch.full((n + 2 * pad,), MARK, dtype=U8, device=dev)
    return whole[pad:pad + n].view(shape), whole


def intact(whole, pad=256):
    return bool((whole[:pad] == MARK).all() and (whole[len(whole) - pad:] == MARK).all())


def sample(rows, d, dtype, dev, seed=0):
    """Values of many sizes, with the groups that a conversion can get wrong."""
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((rows, d), generator=g, device=dev) * torch.exp2(
        torch.randint(-12, 12, (rows, d // 32), generator=g, device=dev).float()).repeat_interleave(32, 1)
    special = [
        [0.0] * 32, [-0.0] * 32, [6.0, 5.0, -5.0, 3.5, -3.5, 2.5, 1.75, 1.25, 0.75, -0.75, 0.25, -0.25, 0.2500001] + [0.0] * 19,
        [6.0000005] + [0.5] * 31, [7.5, -0.5] * 16, [2.0 ** -149, 2.0 ** -127] * 16, [2.0 ** -126, -(2.0 ** -128)] * 16,
        [3.3e38, -1e38, 1e37, 3e36] * 8, [float("nan")] + [1.0] * 31, [1.0] * 31 + [float("inf")],
        [-float("inf"), float("nan")] * 16, [1e-30] * 32, [6 * 2.0 ** 125, 6 * 2.0 ** 124] * 16]
    flat = x.reshape(-1, 32)
    for i, s in enumerate(special):
        if i < flat.shape[0]:
            flat[(i * 37) % flat.shape[0]] = torch.tensor(s, device=dev)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows, d", [(0, 256), (1, 32), (3, 64), (7, 96), (130, 224), (5, 256), (33, 288), (129, 512),
                                     (2, 1056), (65, 2080), (130, 5152), (40, 7168), (3, 65568)])
def test_rows(dev, rows, d, dtype):
    x = sample(rows, d, dtype, dev) if rows else torch.empty((0, d), dtype=dtype, device=dev)
    codes, wc = marked((rows, d // 2), dev)
    scales, ws = marked((-(-d // 256), rows, 8), dev)
    moe.moe_mxfp4_quantize(x, codes, scales)
    torch.cuda.synchronize()
    assert intact(wc) and intact(ws)
    if not rows:
        return
    want_c, want_s = mx.quantize(x)
    assert torch.equal(scales, want_s)
    assert torch.equal(codes, want_c)
    for out_dtype in (BF, F32):
        whole = torch.full((rows * d + 256,), 7.0, dtype=out_dtype, device=dev)
        out = whole[128:128 + rows * d].view(rows, d)
        moe.moe_mxfp4_dequantize(codes.view(torch.float4_e2m1fn_x2), scales.view(torch.float8_e8m0fnu), out)
        want = mx.values(codes, scales)
        torch.testing.assert_close(out.double(), want, rtol=0, atol=0, equal_nan=True)
        assert (whole[:128] == 7).all() and (whole[-128:] == 7).all()


def test_every_value(dev):
    """All 256 code bytes under all 256 scale bytes; fp32 holds each but 6 * 2^127, bf16 too."""
    codes = torch.arange(256, dtype=U8, device=dev).repeat(256, 1)
    scales = mx.blocked(torch.arange(256, dtype=U8, device=dev)[:, None].expand(256, 16).contiguous())
    want = mx.values(codes, scales)
    for dtype in (BF, F32):
        out = torch.empty((256, 512), dtype=dtype, device=dev)
        moe.moe_mxfp4_dequantize(codes, scales, out)
        torch.testing.assert_close(out.double(), want.to(dtype).double(), rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E, N, K", [(1, 8, 32), (3, 40, 96), (5, 24, 1056), (8, 130, 512)])
def test_matrices(dev, E, N, K, dtype):
    w = sample(E * N, K, dtype, dev, seed=E).view(E, N, K)
    codes, scales = moe.mxfp4_buffers((E, N, K), device=dev)
    moe.moe_mxfp4_quantize(w, codes, scales)
    want_c, want_s = mx.quantize(w)
    assert torch.equal(codes, want_c) and torch.equal(scales, want_s)
    out = torch.empty((E, N, K), dtype=dtype, device=dev)
    moe.moe_mxfp4_dequantize(codes, scales, out)
    torch.testing.assert_close(out.double(), mx.values(codes, scales), rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T, k, d", [(1, 1, 32), (1, 8, 4096), (5, 3, 96), (130, 8, 5152), (67, 7, 288), (300, 32, 256)])
def test_sorted_rows(dev, T, k, d, dtype):
    """Each token's row in its k sorted rows; dropped assignments are skipped, rows that none names stay."""
    x = sample(T, d, dtype, dev, seed=k)
    R = T * k
    g = torch.Generator(device=dev).manual_seed(3)
    f2s = torch.randperm(R, generator=g, device=dev).to(torch.int32)
    f2s[torch.randperm(R, generator=g, device=dev)[: R // 5]] = -1
    if R > 40:
        f2s[11] = R      # outside: skipped as well
        f2s[12] = -2 ** 31
    codes, wc = marked((R, d // 2), dev)
    scales, ws = marked((-(-d // 256), R, 8), dev)
    moe.moe_mxfp4_quantize(x, codes, scales, flat_to_sorted=f2s)
    torch.cuda.synchronize()
    assert intact(wc) and intact(ws)
    c, s = mx.quantize(x)
    want_c = torch.full_like(codes, MARK)
    want_s = torch.full_like(scales, MARK)
    at = torch.nonzero((f2s >= 0) & (f2s < R)).reshape(-1)
    want_c[f2s[at].long()] = c[at // k]
    want_s[:, f2s[at].long()] = s[:, at // k]
    assert torch.equal(codes, want_c) and torch.equal(scales, want_s)


def test_offsets_past_32_bits(dev):
    """More than 2^32 elements: the last rows, on both ways."""
    rows, d = (1 << 32) // 7168 + 40, 7168
    part = sample(64, d, BF, dev, seed=9)
    part = torch.where(torch.isfinite(part), part, torch.ones_like(part))
    x = torch.empty((rows, d), dtype=BF, device=dev)
    x[:64] = part
    x[-64:] = part
    codes, scales = moe.mxfp4_buffers((rows, d), device=dev)
    moe.moe_mxfp4_quantize(x, codes, scales)
    want_c, want_s = mx.quantize(part)
    for at in (slice(0, 64), slice(rows - 64, rows)):
        assert torch.equal(codes[at], want_c) and torch.equal(scales[:, at], want_s)
    x.zero_()
    moe.moe_mxfp4_dequantize(codes, scales, x)
    assert torch.equal(x[-64:].double(), mx.values(want_c, want_s)) and torch.equal(x[:64], x[-64:])


def test_other_stream_and_graph(dev):
    """On a stream of the caller's, and captured: each replay works on what its inputs hold then."""
    x = sample(40, 288, BF, dev)
    codes, scales = moe.mxfp4_buffers((40, 288), device=dev)
    out = torch.empty((40, 288), dtype=F32, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_mxfp4_quantize(x, codes, scales, stream=s)
    s.synchronize()
    assert torch.equal(codes, mx.quantize(x)[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_mxfp4_quantize(x, codes, scales)
        moe.moe_mxfp4_dequantize(codes, scales, out)
    for i in range(3):
        x.copy_(sample(40, 288, BF, dev, seed=i + 20))
        graph.replay()
        torch.cuda.synchronize()
        want_c, want_s = mx.quantize(x)
        assert torch.equal(codes, want_c) and torch.equal(scales, want_s)
        torch.testing.assert_close(out.double(), mx.values(want_c, want_s), rtol=0, atol=0, equal_nan=True)
