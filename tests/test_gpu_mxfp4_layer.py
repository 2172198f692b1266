"""The MXFP4 calls as they are used together: a layer with 4-bit weights, the same with 4-bit rows between the calls, and
a training step through weights that stay as they are. Every stage is checked in 64 bits on what the stage before
left behind, within its own arithmetic's bound."""
import pytest
import torch

import gpu_harness as H
import mxfp4_ref as mx
import token_dispatch_expert_amd as moe
import training_ref as ref
from test_gpu_mxfp4_products import check_mxfp4, held, product_error, swiglu_reference
from token_dispatch_expert_amd.binding import layer_buffers

pytestmark = pytest.mark.gpu

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
F4, E8 = torch.float4_e2m1fn_x2, torch.float8_e8m0fnu


@pytest.fixture(scope="module")
def dev():
    return H.require_gpu()


def weights(E, d, f, dev):
    return {n: held((E, *s), dev, i, s[1] ** -0.5) for i, (n, s) in enumerate(
        dict(gate=(f, d), up=(f, d), down=(d, f)).items())}


def counts_of(out, E):
    return out["counts"].cpu().tolist()


def expect_layer(x, out, W, k, y_dtype, capacity=None):
    """y of a layer with bf16 rows, from the router's choice in `out`, and how far it may be off: h's arithmetic and
    rounding pass through the down product, whose own sum and the combine's k terms follow."""
    E = W["gate"][0].shape[0]
    counts = counts_of(out, E)
    kept = sum(counts)
    T = x.shape[0]
    s2f = out["sorted_to_flat"][:kept].long()
    xs = x.double()[s2f // k]
    h, e = swiglu_reference(xs, W["gate"][2], W["up"][2], counts)
    eh = e + ref.u(BF) * (h.abs() + e)
    ys = ref.forward(h, W["down"][2], counts)
    ey = ref.forward(eh, W["down"][2].abs(), counts) + product_error(h.abs() + eh, W["down"][2], counts)
    gates = out["topk_gates"].double().reshape(-1)[s2f][:, None]
    y = torch.zeros((T, x.shape[1]), dtype=torch.float64, device=x.device).index_add_(0, s2f // k, gates * ys)
    size = torch.zeros_like(y).index_add_(0, s2f // k, gates * (ys.abs() + ey))
    tol = torch.zeros_like(y).index_add_(0, s2f // k, gates * ey) + (k + 1) * 2.0 ** -23 * size
    return y, tol + ref.u(y_dtype) * (y.abs() + tol) + 1e-37


@pytest.mark.parametrize("y_dtype", [F32, BF])
@pytest.mark.parametrize("T, E, k, d, f, capacity", [
    (1, 8, 2, 256, 96, None), (1, 16, 8, 2048, 1536, None), (40, 16, 4, 288, 544, None), (700, 8, 2, 800, 320, None),
    (700, 8, 3, 544, 288, 200), (0, 8, 2, 256, 96, None)])
def test_layer(dev, T, E, k, d, f, capacity, y_dtype):
    W = weights(E, d, f, dev)
    g = torch.Generator(device=dev).manual_seed(T)
    logits = torch.randn((T, E), generator=g, device=dev)
    x = torch.randn((T, d), generator=g, device=dev).to(BF)
    out = layer_buffers(T, E, k, d, BF, device=dev, y_dtype=y_dtype)
    ws = moe.Workspace(moe.moe_layer_workspace_size(T, E, k, d, f, BF, F4), device=dev)
    call = [W[n][0].view(F4) for n in ("gate", "up", "down")]
    scales = dict(s_gate=W["gate"][1], s_up=W["up"][1].view(E8), s_down=W["down"][1])
    moe.moe_layer(logits, x, *call, k, out, ws, capacity=capacity, **scales)
    torch.cuda.synchronize()
    if T == 0:
        return
    if capacity is not None:
        assert max(counts_of(out, E)) == capacity
    y, tol = expect_layer(x, out, W, k, y_dtype)
    assert ((out["y"].double() - y).abs() <= tol).all()
    # the layer's parts, called one by one, give the same bits
    ys = torch.full_like(out["y_sorted"], float("nan"))
    fw = moe.Workspace(moe.moe_ffn_workspace_size(T * k, E, d, f, BF, F4), device=dev)
    moe.moe_grouped_ffn(out["x_sorted"], out["offsets"], *call, ys, fw, **scales)
    kept = sum(counts_of(out, E))
    assert torch.equal(ys[:kept], out["y_sorted"][:kept]) and torch.isnan(ys[kept:]).all()


def test_layer_captured(dev):
    """Two layers that share weights, each with its own workspace, captured and replayed beside eager calls."""
    T, E, k, d, f = 12, 8, 2, 544, 288
    W = weights(E, d, f, dev)
    args = [W[n][0].view(F4) for n in ("gate", "up", "down")]
    scales = dict(s_gate=W["gate"][1], s_up=W["up"][1], s_down=W["down"][1])
    logits = [torch.randn((T, E), device=dev) for _ in range(2)]
    xs = [torch.randn((T, d), device=dev).to(BF) for _ in range(2)]
    outs = [layer_buffers(T, E, k, d, BF, device=dev) for _ in range(3)]
    size = moe.moe_layer_workspace_size(T, E, k, d, f, BF, F4)
    wss = [moe.Workspace(size, device=dev) for _ in range(3)]
    moe.moe_layer(logits[0], xs[0], *args, k, outs[2], wss[2], **scales)
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_layer(logits[i], xs[i], *args, k, outs[i], wss[i], **scales)
        graphs.append(g)
    for _ in range(3):
        for i in range(2):
            logits[i].normal_()
            xs[i].normal_()
            outs[i]["y"].zero_()
        for g in graphs:
            g.replay()
        for i in range(2):
            moe.moe_layer(logits[i], xs[i], *args, k, outs[2], wss[2], **scales)
            torch.cuda.synchronize()
            assert torch.equal(outs[i]["y"], outs[2]["y"])


@pytest.mark.parametrize("T, E, k, d, f", [(1, 8, 2, 256, 96), (40, 16, 4, 288, 544), (700, 8, 3, 800, 320)])
def test_rows_in_4_bits(dev, T, E, k, d, f):
    """Serving with 4-bit rows: the token quantised once into its sorted rows, gate and up give h in 4 bits, down takes it."""
    W = weights(E, d, f, dev)
    R = T * k
    logits, x = torch.randn((T, E), device=dev), torch.randn((T, d), device=dev).to(BF)
    b = layer_buffers(T, E, k, d, BF, device=dev)
    moe.moe_route(logits, k, b["topk_ids"], b["topk_gates"])
    moe.moe_permute(x, b["topk_ids"], E, b["counts"], b["offsets"], b["sorted_to_flat"], b["flat_to_sorted"],
                    b["x_sorted"], moe.Workspace(moe.moe_permute_workspace_size(T, E, k), device=dev))
    x4, xs = moe.mxfp4_buffers((R, d), device=dev)
    h4, hs = moe.mxfp4_buffers((R, f), device=dev)
    moe.moe_mxfp4_quantize(x, x4, xs, flat_to_sorted=b["flat_to_sorted"])
    moe.moe_grouped_swiglu_mxfp4(x4, b["offsets"], W["gate"][0], W["gate"][1], W["up"][0], W["up"][1], h4, x_scales=xs,
                                 h_scales=hs)
    moe.moe_grouped_gemm_mxfp4(h4, b["offsets"], W["down"][0], W["down"][1], b["y_sorted"], x_scales=hs)
    moe.moe_combine(b["y_sorted"], b["flat_to_sorted"], b["topk_gates"], b["y"])
    torch.cuda.synchronize()
    counts = b["counts"].cpu().tolist()
    want_c, want_s = mx.quantize(b["x_sorted"])
    assert torch.equal(x4, want_c)
    assert torch.equal(mx.rows_of(xs, d // 32), mx.rows_of(want_s, d // 32))
    h, e = swiglu_reference(mx.values(x4, xs), W["gate"][2], W["up"][2], counts)
    check_mxfp4(h4, hs, h, e)
    hv = mx.values(h4, hs)
    ys = ref.forward(hv, W["down"][2], counts)
    tol = product_error(hv, W["down"][2], counts) + ref.u(F32) * ys.abs() + 1e-37
    assert ((b["y_sorted"].double() - ys).abs() <= tol).all()
    rows = b["y_sorted"].double()[b["flat_to_sorted"].long()].reshape(T, k, d) * b["topk_gates"].double()[:, :, None]
    assert ((b["y"].double() - rows.sum(1)).abs() <= (k + 1) * 2.0 ** -23 * rows.abs().sum(1) + 1e-37).all()


def test_training_step_through_frozen_weights(dev):
    """Forward and the gradient to the layer's input, each product within its bound of 64 bits on its own inputs."""
    T, E, k, d, f = 300, 6, 2, 544, 352
    W = weights(E, d, f, dev)
    R = T * k
    logits, x = torch.randn((T, E), device=dev), torch.randn((T, d), device=dev).to(BF)
    dy = (torch.randn((T, d), device=dev) * 1e-3).to(BF)
    b = layer_buffers(T, E, k, d, BF, device=dev)
    moe.moe_route(logits, k, b["topk_ids"], b["topk_gates"])
    moe.moe_permute(x, b["topk_ids"], E, b["counts"], b["offsets"], b["sorted_to_flat"], b["flat_to_sorted"],
                    b["x_sorted"], moe.Workspace(moe.moe_permute_workspace_size(T, E, k), device=dev))
    off, f2s = b["offsets"], b["flat_to_sorted"]
    z = lambda shape, t: torch.empty(shape, dtype=t, device=dev)  # noqa: E731
    g, u, h, dh, dg, du = (z((R, f), BF) for _ in range(6))
    dys, dxs, dx = z((R, d), BF), z((R, d), BF), z((T, d), F32)
    moe.moe_grouped_gemm_mxfp4(b["x_sorted"], off, W["gate"][0], W["gate"][1], g)
    moe.moe_grouped_gemm_mxfp4(b["x_sorted"], off, W["up"][0], W["up"][1], u)
    moe.moe_swiglu(g, u, h, offsets=off)
    moe.moe_grouped_gemm_mxfp4(h, off, W["down"][0], W["down"][1], b["y_sorted"])
    moe.moe_combine_backward(dy, None, f2s, b["topk_gates"], dys, None)
    moe.moe_grouped_gemm_mxfp4_dgrad(dys, off, W["down"][0], W["down"][1], dh)
    moe.moe_swiglu_backward(dh, g, u, dg, du, offsets=off)
    moe.moe_grouped_gemm_mxfp4_dgrad(dg, off, W["gate"][0], W["gate"][1], dxs, dy2=du, w2=W["up"][0], w2_scales=W["up"][1])
    moe.moe_permute_backward(dxs, f2s, k, dx)
    torch.cuda.synchronize()
    counts = b["counts"].cpu().tolist()

    def close(got, want, e):
        assert ((got.double() - want).abs() <= e + ref.u(got.dtype) * (want.abs() + e) + 1e-37).all()

    xs = b["x_sorted"].double()
    for got, n, a in ((g, "gate", xs), (u, "up", xs), (b["y_sorted"], "down", h.double())):
        close(got, ref.forward(a, W[n][2], counts), product_error(a, W[n][2], counts))
    across = {n: W[n][2].transpose(1, 2).contiguous() for n in W}
    close(dh, ref.forward(dys, across["down"], counts), product_error(dys.double(), across["down"], counts))
    close(dxs, ref.forward(dg, across["gate"], counts) + ref.forward(du, across["up"], counts),
          2 * product_error(dg.double(), across["gate"], counts) + 2 * product_error(du.double(), across["up"], counts))
    want = dxs.double()[f2s.long()].reshape(T, k, d)
    close(dx, want.sum(1), k * 2.0 ** -23 * want.abs().sum(1))
