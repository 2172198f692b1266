"""SwiGLU and its gradient far down the sigmoid, where s = 1 / (1 + e^-g) is no normal fp32 number (g under
-87.3) or e^-g overflows (under -88.7): what s is multiplied with may be large, and the result is then an
ordinary number."""
import pytest
import torch

import token_dispatch_expert_amd as moe

import gpu_harness as H
import training_ref as ref

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
LOW = [-80.0, -86.5, -87.0, -87.3, -87.5, -88.0, -88.5, -88.75, -89.0, -90.0, -95.0, -103.0, -104.0, -110.0, -150.0,
       -174.0, -200.0, -260.0, -348.0, -350.0, -1000.0, -3e38]
FACTORS = [(1e38, 1e-2), (1e20, 1e18), (3e38, 1.0), (1.0, 3e38), (1.0, 1.0), (-3e37, 2.5), (0.0, 1.0), (1e-30, 3e38)]


@pytest.fixture(scope="module")
def dev():
    return H.require_gpu()


def tail_inputs(dtype, dev, width=64):
    """Every g with every (u, dh), padded with ordinary values to rows of `width`; 64-bit copies of what was stored."""
    rows = [(g, u_, dh) for g in LOW for u_, dh in FACTORS]
    fill = (-len(rows)) % width
    rows += [(0.5 + 0.01 * i, 1.0, 1.0) for i in range(fill)]
    cols = torch.tensor(rows, dtype=torch.float64).reshape(-1, width, 3)
    # neighbours of a low g in a thread's 8 elements: both low and ordinary ones
    cols = torch.cat([cols, cols.flatten(0, 1)[torch.randperm(cols.shape[0] * width, generator=torch.Generator().manual_seed(1))]
                      .reshape(cols.shape)])
    return [ref.put(cols[:, :, i].to(dtype).to(dev), dtype, dev) for i in range(3)]


def check(name, got, want, rel, dtype):
    """Relative to the value: `rel` of the computation and one rounding to the format; where the format
    has only subnormals left, one step of those (2^-133 in bf16, 2^-149 in fp32; twice, for the 64-bit
    result's way through fp32). A result past the range is infinite."""
    assert got.dtype == dtype
    step = {BF: 2.0 ** -133, F32: 2.0 ** -149}[dtype]
    most = torch.finfo(dtype).max
    g = got.double()
    tol = want.abs() * (rel + ref.u(dtype)) + 2 * step
    over = want.abs() > most
    bad = torch.where(over, (g != torch.sign(want) * float("inf")) & (g.abs() < most), (g - want).abs() > tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} values, first got {g[bad][0].item():.6g}, want {want[bad][0].item():.6g}"


# fp32: s from e^(g/4), within 2 units, to the fourth power, or from e^-g, a sum and a division; up to eight
# products of one unit (2^-23) each: under 2^-19. bf16: the product with log2 e is off by |g| 2^-24, so e^-g by
# up to 1000 2^-24 where anything is left of it: under 2^-13, and rounding comes on top.
REL = {F32: 2.0 ** -19, BF: 2.0 ** -13}


@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_and_gradient_down_the_tail(dev, dtype):
    g, u_, dh = tail_inputs(dtype, dev)
    gd, ud, dhd = g.double(), u_.double(), dh.double()
    out = {n: ref.guarded(tuple(g.shape), dtype, dev) for n in ("forward", "dg", "du", "h")}
    moe.moe_swiglu(g, u_, out["forward"][0])
    moe.moe_swiglu_backward(dh, g, u_, out["dg"][0], out["du"][0], h=out["h"][0])
    want = dict(zip(("dg", "du", "h"), ref.swiglu_backward(dhd, gd, ud)), forward=ref.swiglu(gd, ud))
    for n, (got, whole) in out.items():
        assert ref.guards_intact(whole, got.numel()), n
        check(n, got, want[n], REL[dtype], dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_of_held_values_down_the_tail(dev, dtype):
    """g and u held in 8 bits, each in rows of its own size (a row's group has one scale): the gradient on
    what the codes stand for."""
    g = torch.tensor([-80.0, -88.0, -96.0, -104.0], device=dev).repeat_interleave(32).repeat(3, 1).to(dtype)
    u_ = torch.tensor([2.0 ** 100, 2.0 ** 120, -1.75 * 2.0 ** 124], device=dev)[:, None].expand(3, 128).to(dtype).contiguous()
    dh = torch.full((3, 128), 0.5, dtype=dtype, device=dev)
    h, dg, du, h2 = (torch.full((3, 128), float("nan"), dtype=dtype, device=dev) for _ in range(4))
    codes = [torch.empty((3, 128), dtype=F8, device=dev) for _ in range(2)]
    scales = [torch.empty((3, 1), device=dev) for _ in range(2)]
    moe.moe_swiglu(g, u_, h, codes[0], scales[0], codes[1], scales[1])
    gd, ud = ref.held(g)[0].to(dev), ref.held(u_)[0].to(dev)
    assert torch.equal(gd, g.double()) and torch.equal(ud, u_.double())  # all of them have codes
    moe.moe_swiglu_backward(dh, codes[0], codes[1], dg, du, h=h2, g_scales=scales[0], u_scales=scales[1])
    want = dict(zip(("dg", "du", "h"), ref.swiglu_backward(dh.double(), gd, ud)), forward=ref.swiglu(gd, ud))
    for n, got in dict(dg=dg, du=du, h=h2, forward=h).items():
        check(n, got, want[n], REL[dtype], dtype)
        assert (got != 0).any(), n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinities_and_nan_beside_low_values(dev, dtype):
    """A low g in a thread's 8 elements changes nothing for a NaN or an infinity beside it."""
    inf, nan = float("inf"), float("nan")
    g = torch.tensor([-100.0, nan, inf, -inf, 1.0, -1.0, 0.0, 30.0], dtype=dtype, device=dev).reshape(1, 8)
    one = torch.ones_like(g)
    h, dg, du = (torch.empty_like(g) for _ in range(3))
    moe.moe_swiglu(g, one, h)
    moe.moe_swiglu_backward(one, g, one, dg, du)
    alone = [torch.empty_like(g) for _ in range(3)]
    g1 = g.clone()
    g1[0, 0], g1[0, 3] = 2.0, 2.0
    moe.moe_swiglu(g1, one, alone[0])
    moe.moe_swiglu_backward(one, g1, one, alone[1], alone[2])
    for a, b in zip((h, dg, du), alone):
        same = [1, 2, 4, 5, 6, 7]
        assert torch.equal(a[0, same].nan_to_num(7.0), b[0, same].nan_to_num(7.0))
        assert torch.isnan(a[0, 1]) and torch.isnan(a[0, 3])
