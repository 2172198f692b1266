"""Every kernel that the MXFP4 products choose between, with each format of the result and, for the input gradient, one pair and
two (test_mxfp4_choice checks on the host that the sizes here take them all); large cases and drawn ones of every operator.

Besides the bound of each element, which has to allow n 2^-23 sum |a||b| for n products (see training_ref), the error's root mean
square over the whole result is checked. An addition is off by at most 2^-23 of its partial sum, and with operands of random
signs no partial sum is larger, in the root mean square, than the whole one; so the error's is at most n 2^-23 of the result's (a quarter
is added for the finite sample), beside the rounding to the result's format. Sums in fewer bits or a product left out are above that."""
import random

import pytest
import torch

import gpu_harness as H
import mxfp4_ref as mx
import test_gpu_mxfp4_cases as listed
import token_dispatch_expert_amd as moe
import training_ref as ref
from test_gpu_measured_cases import within
from test_gpu_mxfp4_cases import dealt, ops, sum_error, swiglu_tolerance
from test_gpu_mxfp4_products import check_mxfp4, held, rows_in, silu

BF, F32 = torch.bfloat16, torch.float32

# (experts, rows, N, K), one for each kernel in the order of its table: products of bf16 rows and of 4-bit ones
PRODUCTS = {
    "bf16": [(8, 13, 264, 1056), (32, 33, 776, 544), (1, 613, 264, 544), (128, 144, 392, 544), (1, 1456, 264, 800), (1, 2278, 272, 544),
             (2, 3877, 392, 544), (1, 8537, 264, 544), (64, 21483, 264, 544)],
    "mxfp4": [(8, 13, 264, 1056), (1, 702, 296, 544), (1, 862, 328, 544), (128, 131, 328, 544), (5, 4734, 264, 544), (64, 18392, 272, 544)],
}
# (experts, rows, d_ff, d) of gate and up, by the formats of rows and of h
SWIGLU = {
    ("bf16", "bf16"): [(8, 13, 256, 1056), (1, 209, 416, 544), (1, 292, 608, 544), (128, 135, 1504, 544), (3, 1266, 288, 544),
                       (64, 713, 2016, 544), (16, 4503, 352, 544), (4, 21284, 288, 800)],
    ("bf16", "mxfp4"): [(8, 13, 256, 1056), (1, 602, 640, 544), (1, 1795, 288, 544), (1, 16826, 288, 544)],
    ("mxfp4", "bf16"): [(8, 13, 256, 1056), (1, 212, 480, 544), (1, 306, 512, 544), (8, 9, 2752, 544), (128, 129, 3424, 544),
                        (1, 9286, 352, 544), (8, 13526, 288, 544)],
    ("mxfp4", "mxfp4"): [(8, 13, 256, 1056), (3, 1647, 384, 544), (1, 5683, 288, 800), (64, 9521, 288, 544)],
}
# (experts, rows, N, K) of the input gradient, of one pair and of two
GRADIENTS = {
    1: [(8, 13, 264, 544), (128, 182, 264, 800), (8, 10, 264, 4128), (4, 727, 264, 544), (5, 1527, 288, 544), (8, 1442, 264, 544),
        (4, 5760, 272, 544), (64, 9194, 272, 544)],
    2: [(8, 13, 264, 544), (128, 182, 264, 800), (8, 10, 264, 4128), (4, 727, 264, 544), (3, 1572, 264, 544), (5, 2444, 264, 544),
        (8, 6312, 264, 544), (64, 9194, 272, 544)],
}


def rms(t):
    return float(t.double().square().mean().sqrt())


def check_rms(got, want, sums):
    """sums: root mean square of what the fp32 sums may be off."""
    rounding = rms(want.to(got.dtype).double() - want)
    assert rms(got.double() - want) <= 1.05 * rounding + 1.25 * sums


@pytest.fixture(scope="module")
def dev():
    return H.require_gpu()


@pytest.fixture(autouse=True)
def own(monkeypatch):
    monkeypatch.setattr(ops, "own", True)


def setting(E, rows, dev):
    """counts of the experts (a few rows belong to none), offsets, spans."""
    counts = dealt(E, rows, 0.6, rows)
    return counts, sum(counts), ref.offsets_of(counts, dev), list(ref.spans(counts))


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("kind, size", [(k, s) for k, sizes in PRODUCTS.items() for s in sizes])
def test_product(dev, kind, size, out):
    E, rows, N, K = size
    counts, used, offsets, spans = setting(E, rows, dev)
    w, ws, wv = held((E, N, K), dev, 1, K ** -0.5)
    x, xs, xv = rows_in(kind, rows, K, dev, 2, used)
    y = torch.full((rows, N), float("nan"), dtype=out, device=dev)
    moe.moe_grouped_gemm_mxfp4(x, offsets, w, ws, y, x_scales=xs)
    assert torch.isnan(y[used:]).all()
    want = ref.forward(xv[:used], wv, counts)
    e = sum_error(xv[:used], lambda k: wv[k], spans, K)
    within("product", y[:used], want, e + ref.u(out) * (want.abs() + e) + 1e-37)
    check_rms(y[:used], want, K * 2.0 ** -23 * rms(want))


@pytest.mark.gpu
@pytest.mark.parametrize("kind, h_kind, size", [(*k, s) for k, sizes in SWIGLU.items() for s in sizes])
def test_swiglu(dev, kind, h_kind, size):
    E, rows, f, d = size
    counts, used, offsets, spans = setting(E, rows, dev)
    w, ws, wv = held((E, f, d), dev, 1, d ** -0.5)
    v, vs, vv = held((E, f, d), dev, 3, d ** -0.5)
    x, xs, xv = rows_in(kind, rows, d, dev, 2, used)
    xv = xv[:used]
    g, u = ref.forward(xv, wv, counts), ref.forward(xv, vv, counts)
    want, e = swiglu_tolerance(g, u, sum_error(xv, lambda k: wv[k], spans, d), sum_error(xv, lambda k: vv[k], spans, d))
    if h_kind == "mxfp4":
        codes, scales = moe.mxfp4_buffers((rows, f), device=dev)
        codes.fill_(0xAB)
        scales.fill_(0xAB)
        moe.moe_grouped_swiglu_mxfp4(x, offsets, w, ws, v, vs, codes, x_scales=xs, h_scales=scales)
        assert (codes[used:] == 0xAB).all() and (scales[:, used:] == 0xAB).all()
        check_mxfp4(codes[:used], scales[:, :used], want, e)
        return
    h = torch.full((rows, f), float("nan"), dtype=BF, device=dev)
    moe.moe_grouped_swiglu_mxfp4(x, offsets, w, ws, v, vs, h, x_scales=xs)
    assert torch.isnan(h[used:]).all()
    within("h", h[:used], want, e + ref.u(BF) * (want.abs() + e) + 1e-37)
    check_rms(h[:used], want, swiglu_sums(g, u, d))


def swiglu_sums(g, u, d):
    """What the two sums' errors, d 2^-23 of their rows' root mean squares, make of h (|silu'| <= 1.1), and the activation's own."""
    eg, eu = (d * 2.0 ** -23 * t.square().mean(1, keepdim=True).sqrt() for t in (g, u))
    return rms(1.1 * eg * u.abs() + silu(g).abs() * eu + (8 + g.abs()) * 2.0 ** -22 * (silu(g) * u).abs())


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("pairs, size", [(p, s) for p, sizes in GRADIENTS.items() for s in sizes])
def test_gradient(dev, pairs, size, out):
    E, rows, N, K = size
    counts, used, offsets, spans = setting(E, rows, dev)
    weights = [held((E, N, K), dev, 1 + i, K ** -0.5) for i in range(pairs)]
    dys = [rows_in("bf16", rows, N, dev, 7 + i, used)[0] for i in range(pairs)]
    more = dict(dy2=dys[1], w2=weights[1][0], w2_scales=weights[1][1]) if pairs == 2 else {}
    dx = torch.full((rows, K), float("nan"), dtype=out, device=dev)
    moe.moe_grouped_gemm_mxfp4_dgrad(dys[0], offsets, weights[0][0], weights[0][1], dx, **more)
    assert torch.isnan(dx[used:]).all()
    want = e = 0
    for (_, _, wv), dy in zip(weights, dys):
        want = want + ref.dgrad(dy[:used], wv, counts)
        e = e + sum_error(dy[:used], lambda k: wv[k], spans, pairs * N, axis=0)  # noqa: B023
    within("gradient", dx[:used], want, e + ref.u(out) * (want.abs() + e) + 1e-37)
    check_rms(dx[:used], want, pairs * N * 2.0 ** -23 * rms(want))


# ----------------------------------------------------------------------------------------
# large and drawn cases, as the benchmark makes them
# ----------------------------------------------------------------------------------------
def case_of(name, **change):
    return dict({c["name"]: c for c in ops.listed()}[name], **change)


LARGE = [case_of("gemm_prefill"), case_of("gemm_prefill", out="f32"), case_of("gemm_prefill_4bit", out="f32"),
         case_of("gemm_prefill", N=7168, K=2048, out="f32"), case_of("gemm_prefill_4bit", N=7168, K=2048),
         case_of("gemm_decode"), case_of("dgrad_train"), case_of("dgrad_train", out="f32"), case_of("swiglu_prefill_4bit"),
         case_of("swiglu_prefill_4bit", x="bf16")]


@pytest.mark.gpu
@pytest.mark.parametrize("case", LARGE, ids=lambda c: "-".join(str(c.get(k, "")) for k in ("name", "N", "x", "out")))
def test_sums_of_large_cases(dev, case):
    print(case, flush=True)
    st = ops.prepare(case, 6)
    want, got = ops.exact(case, 6), ops.run(st)
    torch.cuda.synchronize()
    if case["op"] != "swiglu":
        n = 2 * case["N"] if case["op"] == "dgrad" else case["K"]
        return check_rms(got, want, n * 2.0 ** -23 * rms(want))
    x = st["x"].double() if st["xs"] is None else mx.values(st["x"], st["xs"])
    g, u = torch.zeros_like(want), torch.zeros_like(want)
    for e, a, b in ref.spans([q - p for p, q in zip(st["bounds"], st["bounds"][1:])]):
        g[a:b] = x[a:b] @ mx.values(st["w"][e], st["ws"][e]).t()
        u[a:b] = x[a:b] @ mx.values(st["w2"][e], st["w2s"][e]).t()
    check_rms(got, want, swiglu_sums(g, u, case["d"]))


def drawn(each):
    """The same number of every operator and every format of its rows."""
    rng, found = random.Random(22), {}
    kinds = [("quantize", None), ("dgrad", None)] + [(op, x) for op in ("gemm", "swiglu") for x in ("bf16", "mxfp4")]
    while any(len(found.get(k, [])) < each for k in kinds):
        c = ops.draw(rng)
        k = (c["op"], None if c["op"] in ("quantize", "dgrad") else c["x"])
        have = found.setdefault(k, [])
        if len(have) < each:
            have.append(dict(c, name=f"drawn-{c['op']}-{k[1] or ''}-{len(have)}"))
    return [c for k in kinds for c in found[k]]


@pytest.mark.gpu
@pytest.mark.parametrize("case", drawn(4), ids=lambda c: c["name"])
def test_drawn(dev, case):
    listed.test_case(dev, case)
