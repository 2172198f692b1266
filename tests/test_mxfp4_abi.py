"""Host-only checks of the MXFP4 calls: every invalid argument is refused with the documented status before any HIP
call (no GPU needed), the binding refuses wrong tensors, and the tests' reference is the format."""
import os

import pytest
import torch

import mxfp4_ref as mx
import token_dispatch_expert_amd as moe
from token_dispatch_expert_amd import binding as B
from test_training_abi import refuses

P, P2, P3, MIS = 0x7F0000000000, 0x7F0000100000, 0x7F0000200000, 0x7F0000000002
INV, UNS = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED
BF, F32, F8, MX = B.MOE_BF16, B.MOE_F32, B.MOE_FP8_E4M3FN, B.MOE_MXFP4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.library_path()):
        pytest.fail("library missing: run __graft_entry__.build()")
    return B.load_library()


def test_reference_is_the_format():
    """Every code under every scale, and scales and codes of chosen groups by hand."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).reshape(256, 256)  # 512 elements a row
    scales = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 16)
    v = mx.values(codes, mx.blocked(scales.contiguous()))
    low = [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    for b in (0, 1, 126, 127, 128, 254):
        assert v[b, 0::2].tolist() == [low[c & 15] * 2.0 ** (b - 127) for c in range(256)]
        assert v[b, 1::2].tolist() == [low[c >> 4] * 2.0 ** (b - 127) for c in range(256)]
    assert torch.isnan(v[255]).all()
    x = torch.zeros(1, 256)
    x[0, 0:4] = torch.tensor([6.0, 2.5, 3.5, -5.0])           # scale 1; ties to 2, 4 and -4
    x[0, 32:35] = torch.tensor([6.5, 0.5, -1.5])              # scale 2; 3.25, 0.25 and -0.75 become 3, 0 and -1
    x[0, 64] = 2.0 ** -140                                    # under the smallest scale
    x[0, 96] = float("inf")
    x[0, 128] = 3.4e38                                        # past the largest scale: stops at 6 * 2^125
    s = mx.scale_of(x)
    assert s[0].tolist() == [127, 128, 2, 255, 252, 127, 127, 127]
    c = mx.codes_of(x, s)
    v = mx.values(c, mx.blocked(s))
    assert v[0, 0:4].tolist() == [6, 2, 4, -4] and v[0, 32:35].tolist() == [6, 0, -2]
    assert v[0, 64] == 0 and torch.isnan(v[0, 96:128]).all() and v[0, 128] == 6 * 2.0 ** 125


def test_quantize(lib):
    ok = dict(x=P, t=BF, E=1, rows=8, k=2, d=256, f2s=P2, c=P3, s=P, st=None)
    refuses(lib.moe_mxfp4_quantize, ok, [
        (dict(x=None), INV), (dict(c=None), INV), (dict(s=None), INV), (dict(x=MIS), INV), (dict(c=MIS), INV),
        (dict(s=MIS), INV), (dict(f2s=MIS + 1), INV), (dict(f2s=None), INV), (dict(E=2), INV), (dict(E=0), INV),
        (dict(rows=-1), INV), (dict(k=0), INV), (dict(k=33), INV), (dict(d=0), INV), (dict(d=100), UNS),
        (dict(d=48), UNS), (dict(d=(1 << 20) + 32), INV), (dict(t=F8), UNS), (dict(t=MX), UNS), (dict(t=11), INV),
        (dict(rows=1 << 30, k=2), INV), (dict(rows=(1 << 31) - 1, k=1, d=1 << 20), UNS)])
    refuses(lib.moe_mxfp4_quantize, dict(ok, E=4, k=1, f2s=None), [
        (dict(x=None), INV), (dict(k=2), INV), (dict(E=1 << 16, rows=1 << 16), INV)])


def test_dequantize(lib):
    ok = dict(c=P, s=P2, E=2, rows=8, d=256, o=P3, t=BF, st=None)
    refuses(lib.moe_mxfp4_dequantize, ok, [
        (dict(c=None), INV), (dict(s=None), INV), (dict(o=None), INV), (dict(c=MIS), INV), (dict(s=MIS), INV),
        (dict(o=MIS), INV), (dict(E=0), INV), (dict(rows=-1), INV), (dict(d=16), UNS), (dict(d=-32), INV),
        (dict(t=MX), UNS), (dict(t=6), INV), (dict(E=1 << 16, rows=1 << 16), INV), (dict(rows=1 << 29, d=1 << 20), UNS)])


def test_other_calls_refuse_the_format(lib):
    refuses(lib.moe_checkpoint_pack, dict(x=P, t=BF, rows=8, d=256, c=P2, sc=P3, s=None), [(dict(t=MX), UNS)])
    refuses(lib.moe_grouped_gemm, dict(x=P, xt=BF, off=P2, rows=64, E=4, N=128, K=256, w=P3, wt=BF, y=P, yt=F32, s=None),
            [(dict(wt=MX), UNS), (dict(xt=MX), UNS), (dict(yt=MX), UNS)])
    ws = lib.moe_permute_workspace_size(64, 8, 2)
    assert lib.moe_permute(P, MX, P2, 64, 8, 2, 256, P3, P3, P3, P3, P, P2, ws, None) == UNS


def meta(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype)  # host tensors: refused last, for where they are


@pytest.mark.parametrize("change, error", [
    (dict(x=meta(8, 256, dtype=torch.float16)), TypeError),
    (dict(x=meta(256, dtype=torch.bfloat16)), ValueError),
    (dict(codes=meta(16, 128, dtype=torch.int8)), TypeError),
    (dict(codes=meta(8, 128)), ValueError),
    (dict(scales=meta(1, 16, 8, dtype=torch.float32)), TypeError),
    (dict(scales=meta(16, 8)), ValueError),
    (dict(scales=meta(1, 8, 8)), ValueError),
    (dict(f=meta(15, dtype=torch.int32)), ValueError),
    (dict(f=meta(0, dtype=torch.int32)), ValueError),
    (dict(f=meta(16, dtype=torch.int64)), TypeError),
    (dict(), ValueError),
])
def test_binding_refuses(change, error):
    a = dict(x=meta(8, 256, dtype=torch.bfloat16), codes=meta(16, 128), scales=meta(1, 16, 8), f=meta(16, dtype=torch.int32))
    a.update(change)
    with pytest.raises(error):
        moe.moe_mxfp4_quantize(a["x"], a["codes"], a["scales"], flat_to_sorted=a["f"])


def test_binding_refuses_out():
    for out, codes, scales, error in (
            (meta(8, 256, dtype=torch.float16), meta(8, 128), meta(1, 8, 8), TypeError),
            (meta(8, 256, dtype=torch.float32), meta(8, 256), meta(1, 8, 8), ValueError),
            (meta(2, 8, 288, dtype=torch.float32), meta(2, 8, 144), meta(2, 1, 8, 8), ValueError),
            (meta(256, dtype=torch.float32), meta(128), meta(1, 8), ValueError)):
        with pytest.raises(error):
            moe.moe_mxfp4_dequantize(codes, scales, out)


def test_buffers():
    c, s = moe.mxfp4_buffers((3, 8, 288), device="cpu")
    assert c.shape == (3, 8, 144) and s.shape == (3, 2, 8, 8) and c.dtype == s.dtype == torch.uint8
    c, s = moe.mxfp4_buffers((8, 256), device="cpu")
    assert c.shape == (8, 128) and s.shape == (1, 8, 8)


def test_grouped_gemm(lib):
    ok = dict(x=P, xs=None, xt=BF, off=P2, rows=64, E=4, N=128, K=256, w=P3, ws=P2, y=P, yt=F32, s=None)
    refuses(lib.moe_grouped_gemm_mxfp4, ok, [
        (dict(x=None), INV), (dict(off=None), INV), (dict(w=None), INV), (dict(ws=None), INV), (dict(y=None), INV),
        (dict(x=MIS), INV), (dict(w=MIS), INV), (dict(ws=MIS), INV), (dict(y=MIS), INV), (dict(off=MIS + 1), INV),
        (dict(xs=P), INV), (dict(xt=MX), INV), (dict(xt=MX, xs=MIS), INV), (dict(xt=F32), UNS), (dict(xt=F8), UNS), (dict(xt=5), INV),
        (dict(yt=MX), UNS), (dict(yt=F8), UNS), (dict(yt=9), INV), (dict(rows=-1), INV), (dict(E=0), INV), (dict(E=1025), UNS),
        (dict(N=0), INV), (dict(N=132), UNS), (dict(K=0), INV), (dict(K=248), UNS), (dict(K=16), UNS),
        (dict(N=(1 << 20) + 8), INV), (dict(K=(1 << 20) + 32), INV), (dict(rows=(1 << 31) - 1, N=1 << 20), UNS)])
    assert lib.moe_grouped_gemm_mxfp4(*dict(ok, rows=0, x=None, y=None).values()) == B.MOE_OK


def test_grouped_gemm_dgrad(lib):
    ok = dict(dy=P, dy2=None, t=BF, off=P2, rows=64, E=4, N=128, K=256, w=P3, ws=P2, w2=None, w2s=None, dx=P, xt=F32, s=None)
    two = dict(dy2=P, w2=P3, w2s=P2)
    refuses(lib.moe_grouped_gemm_mxfp4_dgrad, ok, [
        (dict(dy=None), INV), (dict(w=None), INV), (dict(ws=None), INV), (dict(dx=None), INV), (dict(off=None), INV),
        (dict(dy=MIS), INV), (dict(w=MIS), INV), (dict(ws=MIS), INV), (dict(dx=MIS), INV),
        (dict(two, dy2=None), INV), (dict(two, w2=None), INV), (dict(two, w2s=None), INV),
        (dict(two, dy2=MIS), INV), (dict(two, w2=MIS), INV), (dict(two, w2s=MIS), INV),
        (dict(t=F32), UNS), (dict(t=MX), UNS), (dict(t=5), INV), (dict(xt=MX), UNS), (dict(xt=9), INV), (dict(rows=-1), INV),
        (dict(E=0), INV), (dict(E=1025), UNS), (dict(N=12), UNS), (dict(K=40), UNS), (dict(K=0), INV),
        (dict(rows=(1 << 31) - 1, K=1 << 20), UNS)])
    assert lib.moe_grouped_gemm_mxfp4_dgrad(*dict(ok, rows=0, dy=None, dx=None).values()) == B.MOE_OK


def test_grouped_swiglu(lib):
    ok = dict(x=P, xs=None, xt=BF, off=P2, rows=64, E=4, f=128, d=256, wg=P3, gs=P2, wu=P3, us=P2, h=P, hs=None, ht=BF, s=None)
    refuses(lib.moe_grouped_swiglu_mxfp4, ok, [
        (dict(x=None), INV), (dict(wg=None), INV), (dict(gs=None), INV), (dict(wu=None), INV), (dict(us=None), INV), (dict(h=None), INV),
        (dict(x=MIS), INV), (dict(wg=MIS), INV), (dict(gs=MIS), INV), (dict(wu=MIS), INV), (dict(us=MIS), INV), (dict(h=MIS), INV),
        (dict(off=None), INV), (dict(xs=P), INV), (dict(xt=MX), INV), (dict(xt=F32), UNS), (dict(xt=5), INV),
        (dict(hs=P), INV), (dict(ht=MX), INV), (dict(ht=MX, hs=MIS), INV), (dict(ht=F32), UNS), (dict(ht=5), INV),
        (dict(f=136), UNS), (dict(d=40), UNS), (dict(f=0), INV), (dict(d=0), INV), (dict(rows=-1), INV), (dict(E=0), INV),
        (dict(E=1025), UNS), (dict(rows=(1 << 31) - 1, f=1 << 20), UNS)])
    assert lib.moe_grouped_swiglu_mxfp4(*dict(ok, rows=0, x=None, h=None).values()) == B.MOE_OK


def test_grouped_ffn(lib):
    need = lib.moe_ffn_workspace_size(64, 4, 256, 128, BF, MX)
    assert need == 64 * 128 * 2 and lib.moe_ffn_workspace_size(0, 4, 256, 128, BF, MX) == 0
    ok = dict(x=P, t=BF, off=P2, rows=64, E=4, d=256, f=128, wg=P3, wu=P3, wd=P3, wt=MX, sg=P2, su=P2, sd=P2, y=P,
              ws=P, n=need, s=None)
    refuses(lib.moe_grouped_ffn, ok, [
        (dict(t=F32), UNS), (dict(t=MX), UNS), (dict(sg=None), INV), (dict(su=None), INV), (dict(sd=None), INV), (dict(sg=MIS), INV),
        (dict(sd=MIS), INV), (dict(wg=None), INV), (dict(wd=MIS), INV), (dict(d=264), UNS), (dict(f=136), UNS), (dict(E=1025), UNS),
        (dict(n=need - 1), B.MOE_ERR_WORKSPACE), (dict(ws=None), B.MOE_ERR_WORKSPACE), (dict(wt=5), UNS),
        (dict(rows=(1 << 31) - 1, f=1 << 20, n=1 << 62), UNS)])


def test_layer(lib):
    T, E, k, d, f = 16, 8, 2, 256, 128
    need = lib.moe_layer_workspace_size(T, E, k, d, f, BF, MX)
    assert need == lib.moe_permute_workspace_size(T, E, k) + lib.moe_ffn_workspace_size(T * k, E, d, f, BF, MX)
    ok = dict(logits=P, x=P, t=BF, T=T, E=E, k=k, d=d, f=f, cap=0, wg=P3, wu=P3, wd=P3, wt=MX, sg=P2, su=P2, sd=P2, ids=P, g=P,
              c=P, off=P, s2f=P, f2s=P, xs=P, ys=P, y=P, yt=BF, ws=P, n=need, s=None)
    refuses(lib.moe_layer_capped, ok, [
        (dict(sg=None), INV), (dict(su=MIS), INV), (dict(t=F32, n=1 << 30), UNS), (dict(d=264), UNS), (dict(f=136, n=1 << 30), UNS), (dict(yt=MX), INV),
        (dict(n=need - 1), B.MOE_ERR_WORKSPACE)])


def weights(E=2, N=64, K=288):
    return meta(E, N, K // 2), meta(E, (K + 255) // 256, N, 8)


bf = lambda *s: meta(*s, dtype=torch.bfloat16)  # noqa: E731
i32 = lambda *s: meta(*s, dtype=torch.int32)  # noqa: E731


@pytest.mark.parametrize("change, error", [
    (dict(x=meta(8, 288, dtype=torch.float16)), TypeError),
    (dict(x=bf(8, 256)), ValueError),
    (dict(x=bf(9, 288)), ValueError),
    (dict(x=meta(8, 144)), TypeError),                              # codes come with their scales
    (dict(x=meta(8, 144), x_scales=meta(1, 8, 8)), ValueError),     # two blocks of 256 elements
    (dict(x_scales=meta(2, 8, 8)), TypeError),                      # and bf16 rows without
    (dict(w=meta(2, 64, 288)), ValueError),
    (dict(w_scales=meta(2, 64, 9)), ValueError),
    (dict(w_scales=None), TypeError),
    (dict(y=meta(8, 64, dtype=torch.float16)), TypeError),
    (dict(y=bf(8, 72)), ValueError),
    (dict(offsets=i32(2)), ValueError),
    (dict(offsets=meta(3, dtype=torch.int64)), TypeError),
    (dict(), ValueError),
])
def test_binding_refuses_products(change, error):
    w, s = weights()
    a = dict(x=bf(8, 288), offsets=i32(3), w=w, w_scales=s, y=bf(8, 64))
    with pytest.raises(error):
        moe.moe_grouped_gemm_mxfp4(**dict(a, **change))


@pytest.mark.parametrize("change, error", [
    (dict(dy=meta(8, 64, dtype=torch.float32)), TypeError),
    (dict(dy=bf(8, 72)), ValueError),
    (dict(dx=bf(8, 256)), ValueError),
    (dict(dy2=None), ValueError),
    (dict(w2=None), ValueError),
    (dict(w2_scales=None), (TypeError, ValueError)),
    (dict(dy2=bf(8, 72)), ValueError),
    (dict(w2=meta(2, 64, 128)), ValueError),
    (dict(), ValueError),
])
def test_binding_refuses_gradient(change, error):
    w, s = weights()
    a = dict(dy=bf(8, 64), offsets=i32(3), w=w, w_scales=s, dx=bf(8, 288), dy2=bf(8, 64), w2=w, w2_scales=s)
    with pytest.raises(error):
        moe.moe_grouped_gemm_mxfp4_dgrad(**dict(a, **change))


@pytest.mark.parametrize("change, error", [
    (dict(w_up=meta(2, 32, 144)), ValueError),
    (dict(up_scales=meta(2, 1, 64, 8)), ValueError),
    (dict(h=meta(8, 64, dtype=torch.float32)), TypeError),
    (dict(h=bf(8, 32)), ValueError),
    (dict(h_scales=meta(1, 8, 8)), TypeError),
    (dict(h=meta(8, 32)), TypeError),
    (dict(), ValueError),
])
def test_binding_refuses_swiglu(change, error):
    w, s = weights()
    a = dict(x=bf(8, 288), offsets=i32(3), w_gate=w, gate_scales=s, w_up=w, up_scales=s, h=bf(8, 64))
    with pytest.raises(error):
        moe.moe_grouped_swiglu_mxfp4(**dict(a, **change))


@pytest.mark.parametrize("change, error", [
    (dict(s_up=None), ValueError),
    (dict(weights_blocked=True), TypeError),
    (dict(w_down=meta(2, 288, 64, dtype=torch.bfloat16)), (TypeError, ValueError)),
    (dict(s_gate=meta(2, 64, 16)), ValueError),
])
def test_binding_refuses_ffn(change, error):
    w, s = weights()
    wd, sd = weights(2, 288, 64)
    f4 = lambda t: t.view(torch.float4_e2m1fn_x2)  # noqa: E731
    a = dict(x_sorted=bf(8, 288), offsets=i32(3), w_gate=f4(w), w_up=f4(w), w_down=f4(wd), y_sorted=meta(8, 288, dtype=torch.float32),
             workspace=meta(1 << 16), s_gate=s, s_up=s, s_down=sd)
    a.update(change)
    with pytest.raises(error):
        moe.moe_grouped_ffn(**a)
