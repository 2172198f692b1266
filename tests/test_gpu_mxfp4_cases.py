"""The cases of perf/more_operators.py, listed and drawn, through the library's calls and against their definition in 64 bits;
and sizes that between them take every kernel of the products."""
import importlib.util
import os
import random

import pytest
import torch

import gpu_harness as H
import mxfp4_ref as mx
import token_dispatch_expert_amd as moe
import training_ref as ref
from test_gpu_measured_cases import norms, within
from test_gpu_mxfp4_products import check_mxfp4, held, rows_in, silu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
_spec = importlib.util.spec_from_file_location(
    "more_operators", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py"))
ops = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(ops)


@pytest.fixture(scope="module")
def dev():
    return H.require_gpu()


@pytest.fixture(autouse=True)
def own(monkeypatch):
    monkeypatch.setattr(ops, "own", True)


def drawn(n):
    rng, cases = random.Random(21), []
    while len(cases) < n:
        c = ops.draw(rng)
        cases.append(dict(c, name=f"drawn-{len(cases)}-{c['op']}"))
    return cases


def sum_error(x, w, spans, length, axis=1):
    """length 2^-23 |x[r]| |w_e[n]| >= length 2^-23 sum |a||b| for each row and output of its expert (w [E, N, K] or a function)."""
    size = None
    for e, a, b in spans:
        if b == a:
            continue
        we = w(e)
        if size is None:
            size = torch.zeros((x.shape[0], we.shape[1 - axis]), dtype=torch.float64, device=x.device)
        size[a:b] = (norms(x[a:b], 1)[:, None] * norms(we, axis)[None, :]).double()
    return length * 2.0 ** -23 * size


def swiglu_tolerance(g, u, eg, eu):
    """As swiglu_reference in test_gpu_mxfp4_products, for the result in bf16."""
    h = silu(g) * u
    e = 1.1 * eg * (u.abs() + eu) + silu(g).abs() * eu + (8 + g.abs()) * 2.0 ** -22 * h.abs()
    return h, e


@pytest.mark.parametrize("case", ops.listed() + drawn(16), ids=lambda c: c["name"])
def test_case(dev, case):
    print(case, flush=True)
    seed = 5
    st = ops.prepare(case, seed)
    want, got = ops.exact(case, seed), ops.run(st)
    torch.cuda.synchronize()
    if case["op"] == "quantize":  # one rounding, the code's; values are exact in either format
        assert torch.equal(got.double(), want)
        return
    spans = list(ref.spans([q - p for p, q in zip(st["bounds"], st["bounds"][1:])]))
    values = lambda w, s: lambda e: mx.values(st[w][e], st[s][e])  # noqa: E731
    if case["op"] == "dgrad":
        e = (sum_error(st["dy"], values("w", "ws"), spans, 2 * case["N"], axis=0)
             + sum_error(st["dy2"], values("w2", "w2s"), spans, 2 * case["N"], axis=0))
    else:
        x = st["x"].double() if st["xs"] is None else mx.values(st["x"], st["xs"])
        e = sum_error(x, values("w", "ws"), spans, x.shape[1])
        if case["op"] == "swiglu":
            g, u = torch.zeros_like(want), torch.zeros_like(want)
            for k, a, b in spans:
                g[a:b] = x[a:b] @ mx.values(st["w"][k], st["ws"][k]).t()
                u[a:b] = x[a:b] @ mx.values(st["w2"][k], st["w2s"][k]).t()
            e = swiglu_tolerance(g, u, e, sum_error(x, values("w2", "w2s"), spans, x.shape[1]))[1]
    within(case["op"], got, want, e + ref.u(got.dtype) * (want.abs() + e) + 1e-37)


# (experts, rows, how uneven, N, K): from a few tiles on some of the CUs to many on all
SIZES = [(8, 8, 0.0, 4096, 1536), (4, 40, 0.0, 2080, 800), (1, 200, 0.0, 2048, 1056), (1, 400, 0.0, 4128, 544), (16, 600, 0.6, 1056, 1056),
         (64, 300, 1.2, 2080, 544), (64, 900, 1.2, 2080, 800), (8, 1200, 0.6, 2080, 544), (1, 1999, 0.0, 2080, 544),
         (32, 3000, 1.2, 2080, 1056), (3, 9000, 0.6, 96, 2080), (3, 30000, 0.6, 1000, 320), (5, 9000, 1.2, 2080, 1056),
         (5, 5, 0.0, 3296, 288), (32, 23683, 0.6, 288, 288), (1, 32048, 0.0, 320, 800), (32, 10978, 0.6, 576, 544), (64, 2850, 0.6, 32, 544),
         (64, 3648, 0.6, 32, 288), (64, 757, 0.0, 264, 1184)]


def dealt(E, rows, zipf, seed):
    share = [(r + 1.0) ** -zipf for r in range(E)]
    counts = [int(rows * s / sum(share)) for s in share]
    random.Random(seed).shuffle(counts)
    return counts


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("E, rows, zipf, N, K", SIZES)
def test_product_sizes(dev, E, rows, zipf, N, K, kind):
    counts = dealt(E, rows, zipf, rows)
    used = sum(counts)
    offsets, spans = ref.offsets_of(counts, dev), list(ref.spans(counts))
    w, ws, wv = held((E, N, K), dev, 1, K ** -0.5)
    x, xs, xv = rows_in(kind, rows, K, dev, 2, used)
    y = torch.full((rows, N), float("nan"), device=dev)
    moe.moe_grouped_gemm_mxfp4(x, offsets, w, ws, y, x_scales=xs)
    assert torch.isnan(y[used:]).all()
    want = ref.forward(xv[:used], wv, counts)
    e = sum_error(xv[:used], lambda k: wv[k], spans, K)
    within("product", y[:used], want, e + ref.u(F32) * (want.abs() + e) + 1e-37)
    if kind == "bf16":
        dy = rows_in("bf16", rows, N, dev, 3, used)[0]
        dx = torch.full((rows, K), float("nan"), device=dev)
        moe.moe_grouped_gemm_mxfp4_dgrad(dy, offsets, w, ws, dx)
        assert torch.isnan(dx[used:]).all()
        want = ref.forward(dy[:used], wv.transpose(1, 2).contiguous(), counts)
        e = sum_error(dy[:used], lambda k: wv[k], spans, N, axis=0)
        within("gradient", dx[:used], want, e + ref.u(F32) * (want.abs() + e) + 1e-37)


@pytest.mark.parametrize("kind, out", [("bf16", "bf16"), ("bf16", "mxfp4"), ("mxfp4", "bf16"), ("mxfp4", "mxfp4")])
@pytest.mark.parametrize("E, rows, zipf, N, K", SIZES)
def test_swiglu_sizes(dev, E, rows, zipf, N, K, kind, out):
    f = max(32, N // 64 * 32)
    counts = dealt(E, rows, zipf, rows)
    used = sum(counts)
    offsets, spans = ref.offsets_of(counts, dev), list(ref.spans(counts))
    w, ws, wv = held((E, f, K), dev, 1, K ** -0.5)
    v, vs, vv = held((E, f, K), dev, 3, K ** -0.5)
    x, xs, xv = rows_in(kind, rows, K, dev, 2, used)
    xv = xv[:used]
    g, u = ref.forward(xv, wv, counts), ref.forward(xv, vv, counts)
    want, e = swiglu_tolerance(g, u, sum_error(xv, lambda k: wv[k], spans, K), sum_error(xv, lambda k: vv[k], spans, K))
    if out == "bf16":
        h = torch.full((rows, f), float("nan"), dtype=BF, device=dev)
        moe.moe_grouped_swiglu_mxfp4(x, offsets, w, ws, v, vs, h, x_scales=xs)
        assert torch.isnan(h[used:]).all()
        within("h", h[:used], want, e + ref.u(BF) * (want.abs() + e) + 1e-37)
        return
    codes, scales = moe.mxfp4_buffers((rows, f), device=dev)
    codes.fill_(0xAB)
    scales.fill_(0xAB)
    moe.moe_grouped_swiglu_mxfp4(x, offsets, w, ws, v, vs, codes, x_scales=xs, h_scales=scales)
    assert (codes[used:] == 0xAB).all() and (scales[:, used:] == 0xAB).all()
    check_mxfp4(codes[:used], scales[:, :used], want, e)


@pytest.mark.parametrize("rows", [5, 40, 400])
def test_few_rows_past_32_bits(dev, rows):
    """Weights of more than 2^32 elements: the last expert's rows, in the kernels for few rows."""
    E, N, K = 150, 4104, 7168
    counts = [0] * (E - 1) + [rows]
    offsets = ref.offsets_of(counts, dev)
    w = torch.zeros((E, N, K // 2), dtype=torch.uint8, device=dev)
    ws = torch.zeros((E, K // 256, N, 8), dtype=torch.uint8, device=dev)
    last, lasts, wv = held((1, N, K), dev, 1, K ** -0.5)
    w[-1], ws[-1] = last[0], lasts[0]
    for kind in ("bf16", "mxfp4"):
        x, xs, xv = rows_in(kind, rows, K, dev, 2, rows)
        y = torch.full((rows, N), float("nan"), device=dev)
        moe.moe_grouped_gemm_mxfp4(x, offsets, w, ws, y, x_scales=xs)
        want = ref.forward(xv, wv, [rows])
        e = sum_error(xv, lambda k: wv[0], [(0, 0, rows)], K)
        within(kind, y, want, e + ref.u(F32) * (want.abs() + e) + 1e-37)
    dy = rows_in("bf16", rows, N, dev, 3, rows)[0]
    dx = torch.full((rows, K), float("nan"), device=dev)
    moe.moe_grouped_gemm_mxfp4_dgrad(dy, offsets, w, ws, dx)
    want = ref.forward(dy, wv.transpose(1, 2).contiguous(), [rows])
    e = sum_error(dy, lambda k: wv[0], [(0, 0, rows)], N, axis=0)
    within("gradient", dx, want, e + ref.u(F32) * (want.abs() + e) + 1e-37)


@pytest.mark.parametrize("counts", [[3, 0, 14], [40, 1], [300, 257]], ids=lambda c: "-".join(map(str, c)))
def test_gradient_of_nan_and_small_scales(dev, counts):
    """A group of NaN reaches its columns of its expert's rows and nothing else, a row of dy its own row; scales of 2^-127 are exact."""
    E, N, K, R = len(counts), 264, 800, sum(counts)
    w, ws, _ = held((E, N, K), dev, 1)
    ws[E - 1, :, :, :] = torch.where(ws[E - 1] == 255, ws[E - 1], torch.zeros_like(ws[E - 1]))
    dy = (rows_in("bf16", R, N, dev, 3, R)[0].float() * 2.0 ** 20).to(BF)
    wv = torch.stack([mx.values(w[k], ws[k]) for k in range(E)])
    offsets = ref.offsets_of(counts, dev)
    dx = torch.empty((R, K), device=dev)
    moe.moe_grouped_gemm_mxfp4_dgrad(dy, offsets, w, ws, dx)
    want = ref.forward(dy, wv.transpose(1, 2).contiguous(), counts)
    e = sum_error(dy, lambda k: wv[k], list(ref.spans(counts)), N, axis=0)
    within("small scales", dx, want, e + ref.u(F32) * (want.abs() + e) + 1e-37)
    ws[0, 1, 77, 3] = 255          # columns 352 .. 383 of row 77 of the first expert
    dy[R - 1, 5] = float("nan")
    moe.moe_grouped_gemm_mxfp4_dgrad(dy, offsets, w, ws, dx)
    nan = torch.zeros_like(dx, dtype=torch.bool)
    nan[: counts[0], 352:384] = True
    nan[R - 1] = True
    assert torch.equal(torch.isnan(dx), nan)
