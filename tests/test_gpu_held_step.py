"""A training step on held activations (test_gpu_training.Step with held=True), on the values that are held: every
call of the backward pass against 64 bits on the very buffers it was given, and the whole backward pass against
64 bits from the held x, g and u on. A step that used the exact activations, or another row's, fails both."""
import pytest
import torch

import gpu_harness as H
import training_ref as ref
from test_gpu_training import Step, relative, swiglu_tolerances

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    return H.require_gpu()


def stored(codes, scales):
    """What 8-bit rows stand for, from their codes."""
    v = ref.code_values().to(codes.device)[codes.view(torch.uint8).long()]
    return v * scales.double().repeat_interleave(128, 1)[:, :codes.shape[1]]


class Rows:
    """The step's rows by expert and by token, in 64 bits."""

    def __init__(self, s):
        self.counts = (s.b["offsets"][1:] - s.b["offsets"][:-1]).tolist()
        self.n = sum(self.counts)
        T, k = s.b["ids"].shape
        self.f2s = s.b["f2s"].reshape(T, k).long()
        self.kept = self.f2s >= 0
        self.row = self.f2s.clamp(min=0)

    def sorted_rows(self, per_token, scale=None):
        """[n, d]: token rows (times scale[t, j]) where their assignments went."""
        out = torch.full((self.n, per_token.shape[1]), float("nan"), dtype=torch.float64, device=per_token.device)
        for j in range(self.f2s.shape[1]):
            on = self.kept[:, j]
            v = per_token[on] if scale is None else per_token[on] * scale[on, j:j + 1]
            out[self.f2s[on, j]] = v
        return out

    def token_sums(self, rows):
        pick = torch.where(self.kept[:, :, None], rows[self.row], torch.zeros(1, dtype=rows.dtype, device=rows.device))
        return pick.sum(1)


def close(name, got, want, tol):
    off = (got.double() - want).abs()
    assert (off <= tol).all(), f"{name}: {((off / tol.clamp(min=1e-300)).max()).item():.3f} of its bound"


def sums(n, size, want, dtype):
    """A sum of n products in fp32, rounded to dtype (see training_ref)."""
    e = n * 2.0 ** -23 * size
    return e + ref.u(dtype) * (want.abs() + e) + 1e-37


CASES = [(40, 8, 2, 136, 264, BF), (700, 16, 4, 256, 384, BF), (600, 4, 2, 1032, 520, BF), (96, 16, 4, 256, 384, F32)]


@pytest.mark.parametrize("T,E,k,d,f,dtype", CASES)
@pytest.mark.parametrize("capacity", [None, 50])
def test_every_call_of_the_step(dev, T, E, k, d, f, dtype, capacity):
    s = Step(T, E, k, d, f, dtype, dev, held=True, capacity=capacity)
    s.forward()
    g, u_ = s.b["g"].clone(), s.b["u"].clone()
    s.backward()
    b, r = s.b, Rows(s)
    n = slice(0, r.n)
    # held in the forward pass, brought back in the backward pass: exactly
    x = stored(*b["x8"])
    gh, uh = stored(*b["g8"])[n], stored(*b["u8"])[n]
    assert torch.equal(x, ref.held(s.x)[0].to(dev))
    assert torch.equal(gh, ref.held(g[n])[0].to(dev)) and torch.equal(uh, ref.held(u_[n])[0].to(dev))
    assert torch.equal(b["xs"][n].double(), r.sorted_rows(x))
    # each call on its own inputs
    want = r.sorted_rows(s.dy.double(), b["gates"].double())
    close("dys", b["dys"][n], want, (ref.u(dtype) + 2 * ref.u(F32)) * want.abs() + 1e-37)
    dys, dh = b["dys"][n].double(), b["dh"][n].double()
    want = ref.dgrad(dys, s.wd, r.counts)
    close("dh", dh, want, sums(d, ref.dgrad(dys.abs(), s.wd.abs(), r.counts), want, dtype))
    tol = swiglu_tolerances(gh, uh, dh, dtype)
    for name, key, want in zip(("dg", "du", "h"), ("dg", "du", "h2"), ref.swiglu_backward(dh, gh, uh)):
        close(key, b[key][n], want, tol[name])
    dg, du, h2 = (b[m][n].double() for m in ("dg", "du", "h2"))
    xs, most = r.sorted_rows(x), max(r.counts)
    for name, a, c in (("dwd", dys, h2), ("dwg", dg, xs), ("dwu", du, xs)):
        want = ref.wgrad(a, c, r.counts)
        close(name, b[name], want, sums(most, ref.wgrad(a.abs(), c.abs(), r.counts), want, F32))
    want = ref.dgrad(dg, s.wg, r.counts) + ref.dgrad(du, s.wu, r.counts)
    size = ref.dgrad(dg.abs(), s.wg.abs(), r.counts) + ref.dgrad(du.abs(), s.wu.abs(), r.counts)
    close("dxs", b["dxs"][n], want, sums(2 * f, size, want, F32))
    dxs = b["dxs"][n].double()
    close("dx", b["dx"], r.token_sums(dxs), sums(2 * k, r.token_sums(dxs.abs()), r.token_sums(dxs), F32))


@pytest.mark.parametrize("T,E,k,d,f,dtype", CASES)
@pytest.mark.parametrize("capacity", [None, 50])
def test_the_backward_pass_sees_the_held_values(dev, T, E, k, d, f, dtype, capacity):
    """From dy to the gradients in 64 bits on the held x, g and u, without any rounding between the calls. bf16: a
    gradient passes at most 8 roundings to bf16 on its way, 2^-8 of an element each, 3.2e-2 together; fp32: 1e-4,
    as for the step without held values. The held values themselves are off by up to 2^-4."""
    s = Step(T, E, k, d, f, dtype, dev, held=True, capacity=capacity)
    s.forward()
    s.backward()
    b, r = s.b, Rows(s)
    n = slice(0, r.n)
    x, gh, uh = stored(*b["x8"]), stored(*b["g8"])[n], stored(*b["u8"])[n]
    dys = r.sorted_rows(s.dy.double(), b["gates"].double())
    dg, du, h = ref.swiglu_backward(ref.dgrad(dys, s.wd, r.counts), gh, uh)
    xs = r.sorted_rows(x)
    want = dict(dwd=ref.wgrad(dys, h, r.counts), dwg=ref.wgrad(dg, xs, r.counts), dwu=ref.wgrad(du, xs, r.counts),
                dx=r.token_sums(ref.dgrad(dg, s.wg, r.counts) + ref.dgrad(du, s.wu, r.counts)))
    for name, w in want.items():
        err = relative(b[name], w)
        print(f"T={T} {dtype} capacity={capacity} {name}: {err:.2e}", flush=True)
        assert err <= (3.2e-2 if dtype == BF else 1e-4), name
