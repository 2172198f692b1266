"""The cases of perf/operators.py, listed and drawn, through the library's calls and against their definition in 64
bits: the sizes that the documents give times for."""
import importlib.util
import os
import random

import pytest
import torch

import gpu_harness as H
import training_ref as ref
from test_gpu_held_step import stored
from test_gpu_training import swiglu_tolerances

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
_spec = importlib.util.spec_from_file_location(
    "operators", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py"))
ops = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(ops)


@pytest.fixture(scope="module")
def dev():
    return H.require_gpu()


@pytest.fixture(autouse=True)
def own(monkeypatch):
    monkeypatch.setattr(ops, "own", True)


def drawn(n):
    rng, cases = random.Random(20), []
    while len(cases) < n:
        c = ops.draw(rng)
        cases.append(dict(c, name=f"drawn-{len(cases)}-{c['op']}"))
    return cases


def norms(t, axis):
    """Euclidean lengths: a sum |a||b| is at most the product of the two (fp32, and 1% more for its rounding)."""
    return t.float().norm(dim=axis) * 1.01


def product_bound(case, st, want):
    """n 2^-23 sum |a||b| for n products, and one rounding of the result (see training_ref)."""
    out = ops.DTYPES[case["out"]]
    size = torch.empty(want.shape, dtype=F32, device=want.device)
    length = 0
    for e, a, b in ref.spans([q - p for p, q in zip(st["bounds"], st["bounds"][1:])]):
        if case["op"] == "wgrad":
            size[e] = norms(st["dy"][a:b], 0)[:, None] * norms(st["x"][a:b], 0)[None, :]
            length = max(length, b - a)
        elif b > a:
            pairs = [("x", "w")] if case["dir"] == "forward" else [("dy", "w"), ("dy2", "w2")]
            axis = 1 if case["dir"] == "forward" else 0
            size[a:b] = sum(norms(st[m][a:b], 1)[:, None] * norms(st[w][e], axis)[None, :] for m, w in pairs)
            length = len(pairs) * (case["K"] if case["dir"] == "forward" else case["N"])
    e = length * 2.0 ** -23 * size
    return e + ref.u(out) * (want.abs() + e) + 1e-37


def within(name, got, want, tol):
    assert got.shape == want.shape, name
    for g, w, t in zip(got.split(4096), want.split(4096), tol.split(4096)):
        assert ((g.double() - w).abs() <= t).all(), name


@pytest.mark.parametrize("case", ops.listed() + drawn(12), ids=lambda c: c["name"])
def test_case(dev, case):
    print(case, flush=True)
    seed = 5
    st = ops.prepare(case, seed)
    want, got = ops.exact(case, seed), ops.run(st)
    torch.cuda.synchronize()
    assert want is not None
    if case["op"] in ("gemm", "wgrad"):
        return within(case["op"], got, want, product_bound(case, st, want))
    if case["op"] == "checkpoint":  # one rounding, the code's; values are exact in either format
        assert torch.equal(got.double(), want)
        return
    if case["op"] == "swiglu":
        dt = ops.DTYPES[case["dtype"]]
        for part in torch.arange(case["T"] * case["k"], device=dev).split(8192):
            g, u_, dh = (st[n][part].double() for n in ("g", "u", "dh"))
            within("h", got["h"][part], want["h"][part], swiglu_tolerances(g, u_, dh, dt)["h"])
            g, u_ = (stored(st[n + "_codes"][part], st[n + "_scales"][part]) for n in "gu")
            tol = swiglu_tolerances(g, u_, dh, dt)
            for n, m in (("dg", "dg"), ("du", "du"), ("h2", "h")):
                within(n, got[n][part], want[n][part], tol[m])
        return
    T, k, d, out = case["T"], case["k"], case["d"], ops.DTYPES[case["out"]]
    within("dy_sorted", got["dy_sorted"], want["dy_sorted"], (ref.u(out) + 2 * ref.u(F32)) * want["dy_sorted"].abs() + 1e-40)
    f2s, dy = st["f2s"].reshape(T, k).long(), st["dy"].double()
    gate_size, dx_size = torch.empty_like(want["dgates"]), torch.zeros_like(want["dx"])
    for j in range(k):
        gate_size[:, j] = norms(st["dy"], 1).double() * norms(st["y_sorted"][f2s[:, j]], 1).double()
        dx_size += st["dx_in"][f2s[:, j]].double().abs()
    off = d * 2.0 ** -23 * gate_size
    within("dgates", got["dgates"], want["dgates"], off)
    within("dx", got["dx"], want["dx"], k * 2.0 ** -22 * dx_size + ref.u(out) * want["dx"].abs() + 1e-37)
    gates = st["gates"].double()
    dg = want["dgates"].abs() + off
    mean = (gates * dg).sum(1, keepdim=True)
    slack = gates * (off + (gates * off).sum(1, keepdim=True) + (k + 4) * 2.0 ** -22 * (dg + mean))
    tol = torch.zeros_like(want["dlogits"]).scatter_(1, st["ids"].long(), slack)  # outside the chosen experts: exactly 0
    within("dlogits", got["dlogits"], want["dlogits"], tol)
