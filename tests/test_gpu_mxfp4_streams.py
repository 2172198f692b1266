"""The MXFP4 products on streams of the caller's, on two at once, and captured: the calls keep no state of their own, so every
output equals the one computed alone, bit for bit."""
import pytest
import torch

import gpu_harness as H
import token_dispatch_expert_amd as moe
import training_ref as ref
from test_gpu_mxfp4_products import held, rows_in

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# few rows per expert and many: the kernels for both
COUNTS = [[1, 0, 2, 5, 0, 1, 1, 16], [300, 0, 700, 31, 1, 258, 0, 513]]
N, K = 544, 1056


@pytest.fixture(scope="module")
def dev():
    return H.require_gpu()


def calls(counts, dev, seed):
    """name -> (the call on outputs and a stream, outputs); the inputs that a caller may change."""
    R, offsets, E = sum(counts), ref.offsets_of(counts, dev), len(counts)
    w, ws, _ = held((E, N, K), dev, seed, K ** -0.5)
    v, vs, _ = held((E, N, K), dev, seed + 1, K ** -0.5)
    x = rows_in("bf16", R, K, dev, seed + 2, R)[0]
    c, cs, _ = rows_in("mxfp4", R, K, dev, seed + 3, R)
    dy = rows_in("bf16", R, N, dev, seed + 4, R)[0]
    new = lambda n, t: torch.empty((R, n), dtype=t, device=dev)  # noqa: E731
    return {
        "product": (lambda o, s: moe.moe_grouped_gemm_mxfp4(x, offsets, w, ws, o[0], stream=s), [new(N, F32)]),
        "product of codes": (lambda o, s: moe.moe_grouped_gemm_mxfp4(c, offsets, w, ws, o[0], x_scales=cs, stream=s), [new(N, BF)]),
        "swiglu": (lambda o, s: moe.moe_grouped_swiglu_mxfp4(x, offsets, w, ws, v, vs, o[0], stream=s), [new(N, BF)]),
        "swiglu to codes": (lambda o, s: moe.moe_grouped_swiglu_mxfp4(c, offsets, w, ws, v, vs, o[0], x_scales=cs, h_scales=o[1], stream=s),
                            list(moe.mxfp4_buffers((R, N), device=dev))),
        "gradient": (lambda o, s: moe.moe_grouped_gemm_mxfp4_dgrad(dy, offsets, w, ws, o[0], stream=s), [new(K, F32)]),
        "gradient of two": (lambda o, s: moe.moe_grouped_gemm_mxfp4_dgrad(dy, offsets, w, ws, o[0], dy2=dy, w2=v, w2_scales=vs, stream=s),
                            [new(K, BF)]),
    }, (x, c, dy)


def poison(outs):
    for o in outs:
        o.fill_(0 if o.dtype is torch.uint8 else float("nan"))


def same(a, b):
    return all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))


@pytest.mark.parametrize("counts", COUNTS, ids=["few", "many"])
def test_two_streams_at_once(dev, counts):
    sets = [calls(counts, dev, s)[0] for s in (10, 20)]
    alone = []
    for c in sets:
        for f, outs in c.values():
            poison(outs)
            f(outs, None)
        alone.append({k: [o.clone() for o in outs] for k, (f, outs) in c.items()})
    torch.cuda.synchronize()
    streams, copies = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for rep in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                for name, (f, outs) in sets[i].items():
                    poison(outs)
                    f(outs, s)
                    copies.append((i, name, [o.clone() for o in outs]))
    torch.cuda.synchronize()
    for i, name, got in copies:
        assert same(got, alone[i][name]), name


@pytest.mark.parametrize("counts", COUNTS, ids=["few", "many"])
def test_captured(dev, counts):
    """One graph of all calls, replayed on other values in the same tensors, with eager calls of the same between the replays."""
    c, inputs = calls(counts, dev, 30)
    for f, outs in c.values():
        f(outs, None)
    torch.cuda.synchronize()
    kept = {k: [torch.empty_like(o) for o in outs] for k, (f, outs) in c.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for name, (f, _) in c.items():
            f(kept[name], None)
    for rep in range(4):
        inputs[0].mul_(-0.5)
        inputs[1].bitwise_xor_(0x88)  # every code's sign
        inputs[2].add_(1.0)
        for f, outs in c.values():
            poison(outs)
            f(outs, None)
        for outs in kept.values():
            poison(outs)
        graph.replay()
        torch.cuda.synchronize()
        for name, (f, outs) in c.items():
            assert same(outs, kept[name]), (rep, name)
