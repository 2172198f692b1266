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
