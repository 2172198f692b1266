"""Host-only checks of the training step's calls: every invalid argument is refused with the documented
status before any HIP call (no GPU needed), and the binding refuses wrong tensors."""
import os

import pytest
import torch

import token_dispatch_expert_amd as moe
from token_dispatch_expert_amd import binding as B

P, P2, P3, MIS = 0x7F0000000000, 0x7F0000100000, 0x7F0000200000, 0x7F0000000002
INV, UNS = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED
BF, F32, F8 = B.MOE_BF16, B.MOE_F32, B.MOE_FP8_E4M3FN


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.library_path()):
        pytest.fail("library missing: run __graft_entry__.build()")
    return B.load_library()


def refuses(f, ok, cases):
    """Each case: arguments changed from a call that is valid but for them, and the status."""
    for change, status in cases:
        assert set(change) <= set(ok)
        assert f(*dict(ok, **change).values()) == status, change


def test_grouped_gemm(lib):
    ok = dict(x=P, xt=BF, off=P2, rows=64, E=4, N=128, K=256, w=P3, wt=BF, y=P, yt=F32, s=None)
    refuses(lib.moe_grouped_gemm, ok, [
        (dict(x=None), INV), (dict(off=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(x=MIS), INV),
        (dict(w=MIS), INV), (dict(y=MIS), INV), (dict(off=P2 + 2), INV), (dict(rows=-1), INV), (dict(E=0), INV),
        (dict(E=1025), UNS), (dict(N=0), INV), (dict(K=0), INV), (dict(N=132), UNS), (dict(K=260), UNS),
        (dict(N=(1 << 20) + 8), INV), (dict(xt=F8), UNS), (dict(xt=9), INV), (dict(wt=F32), UNS), (dict(wt=9), INV),
        (dict(wt=B.MOE_BF16_BLOCKED), UNS), (dict(yt=F8), UNS), (dict(yt=-1), INV),
        (dict(rows=(1 << 31) - 1, N=1 << 20), UNS)])


def test_grouped_gemm_dgrad(lib):
    ok = dict(dy=P, dy2=None, t=BF, off=P2, rows=64, E=4, N=128, K=256, w=P3, w2=None, wt=BF, dx=P, xt=F32, s=None)
    refuses(lib.moe_grouped_gemm_dgrad, ok, [
        (dict(dy=None), INV), (dict(w=None), INV), (dict(dx=None), INV), (dict(dy2=P), INV), (dict(w2=P), INV),
        (dict(dy2=MIS, w2=P), INV), (dict(dy2=P, w2=MIS), INV), (dict(t=F32), UNS), (dict(xt=F8), UNS), (dict(N=12), UNS),
        (dict(rows=(1 << 31) - 1, K=1 << 20), UNS)])


def test_grouped_gemm_wgrad(lib):
    ok = dict(dy=P, x=P2, t=BF, off=P3, rows=64, E=4, N=128, K=256, dw=P, dt=F32, acc=0, s=None)
    refuses(lib.moe_grouped_gemm_wgrad, ok, [
        (dict(dy=None), INV), (dict(x=None), INV), (dict(dw=None), INV), (dict(off=None), INV), (dict(acc=2), INV),
        (dict(acc=-1), INV), (dict(t=F8), UNS), (dict(dt=F8), UNS), (dict(dt=7), INV), (dict(K=20), UNS), (dict(E=2000), UNS),
        (dict(E=1024, N=1 << 20, K=1 << 20), UNS)])


def test_checkpoints(lib):
    refuses(lib.moe_checkpoint_pack, dict(x=P, t=BF, rows=8, d=256, c=P2, sc=P3, s=None), [
        (dict(x=None), INV), (dict(c=None), INV), (dict(sc=None), INV), (dict(x=MIS), INV), (dict(c=MIS), INV),
        (dict(rows=-1), INV), (dict(d=0), INV), (dict(d=100), UNS), (dict(t=F8), UNS), (dict(t=11), INV),
        (dict(rows=(1 << 31) - 1, d=1 << 20), UNS)])
    refuses(lib.moe_checkpoint_unpack, dict(c=P, sc=P2, T=8, k=2, d=256, f2s=P3, out=P, t=BF, s=None), [
        (dict(c=None), INV), (dict(sc=None), INV), (dict(out=None), INV), (dict(f2s=None), INV), (dict(k=0), INV),
        (dict(k=33), INV), (dict(T=-1), INV), (dict(T=1 << 30, k=2), INV), (dict(d=12), UNS), (dict(t=F8), UNS),
        (dict(f2s=MIS + 1), INV), (dict(out=MIS), INV)])


def test_swiglu(lib):
    ok = dict(g=P, u=P2, t=BF, off=P3, E=4, rows=8, f=256, h=P, gc=P, gs=P2, uc=P3, us=P, s=None)
    refuses(lib.moe_swiglu, ok, [
        (dict(g=None), INV), (dict(u=None), INV), (dict(h=None), INV), (dict(gc=None), INV), (dict(gs=None), INV),
        (dict(uc=None), INV), (dict(us=None), INV), (dict(gc=MIS), INV), (dict(f=12), UNS), (dict(rows=-2), INV),
        (dict(t=F8), UNS), (dict(E=0), INV), (dict(E=1025), UNS), (dict(off=MIS), INV)])
    ok = dict(dh=P, t=BF, g=P2, u=P3, gt=F8, gs=P, us=P2, off=None, E=0, rows=8, f=256, dg=P, du=P2, h=None, s=None)
    refuses(lib.moe_swiglu_backward, ok, [
        (dict(dh=None), INV), (dict(g=None), INV), (dict(dg=None), INV), (dict(du=None), INV), (dict(gs=None), INV),
        (dict(us=None), INV), (dict(gt=BF), INV), (dict(gt=F32, gs=None, us=None), UNS), (dict(gt=8), INV),
        (dict(gt=B.MOE_FP8_E4M3FN_BLOCKED), UNS), (dict(h=MIS), INV), (dict(off=P, E=0), INV), (dict(t=F8), UNS)])


def test_token_gradients(lib):
    ok = dict(dy=P, t=BF, ys=P2, f2s=P3, gates=P, T=8, k=2, d=256, dys=P2, dt=BF, dg=P3, s=None)
    refuses(lib.moe_combine_backward, ok, [
        (dict(dy=None), INV), (dict(ys=None), INV), (dict(dg=None), INV), (dict(f2s=None), INV), (dict(gates=None), INV),
        (dict(dys=None), INV), (dict(dys=MIS), INV), (dict(k=0), INV), (dict(k=40), INV), (dict(T=-1), INV),
        (dict(T=1 << 30), INV), (dict(d=4), UNS), (dict(t=F8), UNS), (dict(dt=F8), UNS)])
    refuses(lib.moe_permute_backward, dict(dxs=P, t=BF, f2s=P2, T=8, k=2, d=256, dx=P3, dt=F32, s=None), [
        (dict(dxs=None), INV), (dict(f2s=None), INV), (dict(dx=None), INV), (dict(dx=MIS), INV), (dict(k=0), INV),
        (dict(d=20), UNS), (dict(t=F8), UNS), (dict(dt=5), INV)])
    refuses(lib.moe_route_backward, dict(dg=P, ids=P2, gates=P3, T=8, E=16, k=2, dl=P, s=None), [
        (dict(dg=None), INV), (dict(ids=None), INV), (dict(gates=None), INV), (dict(dl=None), INV), (dict(k=17), INV),
        (dict(E=1025), UNS), (dict(T=-1), INV), (dict(dl=MIS), INV)])


def test_binding_refuses_wrong_tensors():
    """Shapes, dtypes, layouts and pairs are checked on the tensors' metadata; host tensors never reach the library."""
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    i = lambda n: z(n, t=torch.int32)  # noqa: E731
    f32, f8 = torch.float32, torch.float8_e4m3fn
    bad = [
        (ValueError, moe.moe_grouped_gemm, (z(4, 16), i(3), z(2, 8, 16), z(4, 8)), {}),                  # on the host
        (TypeError, moe.moe_grouped_gemm, (z(4, 16), i(3), z(2, 8, 16, t=f32), z(4, 8)), {}),            # two dtypes
        (ValueError, moe.moe_grouped_gemm, (z(4, 16), i(3), z(2, 8, 24), z(4, 8)), {}),                  # K differs
        (ValueError, moe.moe_grouped_gemm, (z(4, 16), i(4), z(2, 8, 16), z(4, 8)), {}),                  # offsets
        (ValueError, moe.moe_grouped_gemm, (z(4, 16), i(3), z(2, 8, 16), z(5, 8)), {}),                  # y
        (TypeError, moe.moe_grouped_gemm, (z(4, 16), z(3, t=torch.int64), z(2, 8, 16), z(4, 8)), {}),
        (ValueError, moe.moe_grouped_gemm_dgrad, (z(4, 8), i(3), z(2, 8, 16), z(4, 16)), dict(dy2=z(4, 8))),
        (ValueError, moe.moe_grouped_gemm_dgrad, (z(4, 8), i(3), z(2, 8, 16), z(4, 16)), dict(dy2=z(3, 8), w2=z(2, 8, 16))),
        (ValueError, moe.moe_grouped_gemm_wgrad, (z(4, 8), z(5, 16), i(3), z(2, 8, 16)), {}),
        (TypeError, moe.moe_grouped_gemm_wgrad, (z(4, 8, t=f32), z(4, 16), i(3), z(2, 8, 16)), {}),
        (TypeError, moe.moe_checkpoint_pack, (z(4, 16), z(4, 16), z(4, 1, t=f32)), {}),                  # codes not 8 bits
        (ValueError, moe.moe_checkpoint_pack, (z(4, 16), z(4, 16, t=f8), z(4, 2, t=f32)), {}),           # scales
        (ValueError, moe.moe_checkpoint_unpack, (z(4, 16, t=f8), z(4, 1, t=f32), z(7, 16)), dict(flat_to_sorted=i(7))),
        (TypeError, moe.moe_checkpoint_unpack, (z(4, 16, t=f8), z(4, 1, t=f32), z(4, 16, t=torch.float16)), {}),
        (ValueError, moe.moe_swiglu, (z(4, 16), z(4, 16), z(4, 16)), dict(g_codes=z(4, 16, t=f8))),
        (ValueError, moe.moe_swiglu_backward, (z(4, 16), z(4, 16), z(4, 16), z(4, 16), z(4, 16)), dict(g_scales=z(4, 1, t=f32))),
        (ValueError, moe.moe_swiglu, (z(4, 16), z(4, 16), z(4, 16)), dict(offsets=i(0))),                # of no expert
        (ValueError, moe.moe_swiglu, (z(4, 16), z(4, 16), z(4, 16)), dict(offsets=i(1))),
        (ValueError, moe.moe_swiglu, (z(4, 16), z(4, 16), z(4, 16)), dict(offsets=i(4).reshape(2, 2))),
        (TypeError, moe.moe_swiglu_backward, (z(4, 16), z(4, 16, t=f32), z(4, 16, t=f32), z(4, 16), z(4, 16)), {}),
        (ValueError, moe.moe_combine_backward, (z(4, 16), None, i(8), z(4, 2, t=f32), z(8, 16), z(4, 2, t=f32)), {}),
        (ValueError, moe.moe_permute_backward, (z(8, 16), i(8), 3, z(4, 16)), {}),
        (TypeError, moe.moe_route_backward, (z(4, 2), i(8).reshape(4, 2), z(4, 2, t=f32), z(4, 8, t=f32)), {}),
    ]
    for error, f, args, kw in bad:
        with pytest.raises(error):
            f(*args, **kw)
    with pytest.raises(ValueError):  # not contiguous
        moe.moe_permute_backward(z(16, 8).t(), i(8), 2, z(4, 16))
