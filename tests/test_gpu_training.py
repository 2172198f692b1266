"""The row-wise operators of the training step (8-bit checkpoints, SwiGLU and its gradient, the backward
passes of combine, permute and route) against 64-bit references, and a whole layer's gradient, as a user
puts it together, against autograd in 64 bits."""
import pytest
import torch

import token_dispatch_expert_amd as moe

import gpu_harness as H
import training_ref as ref

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    return H.require_gpu()


def normal(shape, seed, dev, scale=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(shape, generator=g, device=dev) * scale


def held_buffers(rows, d, dev):
    return ref.guarded((rows, d), F8, dev), ref.guarded((rows, -(-d // 128)), F32, dev)


def hard_rows(d, dtype, dev):
    """Rows that a scale has to get right: zeros, one value, the borders of a scale, the type's ends,
    non-finite values among finite ones, and ordinary ones."""
    tiny, huge = torch.finfo(dtype).tiny, torch.finfo(dtype).max
    rows = [torch.zeros(d), torch.full((d,), -0.0), torch.full((d,), 448.0), torch.full((d,), 450.0),
            torch.full((d,), 3.0), torch.full((d,), tiny), torch.full((d,), huge), torch.full((d,), -huge),
            torch.full((d,), 2.0 ** -117 * 448), torch.full((d,), 2.0 ** -126)]
    for seed, scale in enumerate((1.0, 1e-3, 1e4, 1e-30, 1e-36, 1e37)):
        rows.append(torch.randn(d, generator=torch.Generator().manual_seed(seed)) * scale)
    wide = torch.randn(d, generator=torch.Generator().manual_seed(9))
    rows.append(wide * 10.0 ** torch.linspace(-12, 12, d))
    for v in (float("inf"), float("-inf"), float("nan")):
        r = wide.clone()
        r[d // 2] = v
        rows.append(r)
    rows.append(torch.full((d,), float("inf")))
    # every code's value, and the midpoints between them (ties)
    t = ref.code_values()[:127].float()
    ties = torch.cat([t, (t[1:] + t[:-1]) / 2])
    rows.append(torch.nn.functional.pad(ties, (0, max(0, d - ties.numel())))[:d])
    x = torch.stack(rows)
    fine = torch.isfinite(x)  # 10^37 times a normal value may pass the type's range: kept inside
    return torch.where(fine, x.clamp(-huge, huge), x).to(dtype).to(dev)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [8, 64, 120, 128, 136, 256, 392, 1544, 5160])
def test_pack_holds_what_is_documented(dev, dtype, d):
    x = ref.put(hard_rows(d, dtype, dev), dtype, dev)
    (codes, cw), (scales, sw) = held_buffers(x.shape[0], d, dev)
    moe.moe_checkpoint_pack(x, codes, scales)
    want, want_scales = ref.held(x)
    assert ref.guards_intact(cw, codes.numel()) and ref.guards_intact(sw, scales.numel())
    assert torch.equal(scales.double().cpu(), want_scales)
    table = ref.code_values()
    got = table[codes.view(torch.uint8).cpu().long()] * scales.double().cpu().repeat_interleave(128, 1)[:, :d]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))
    # the documented distance from x
    xd = x.double().cpu()
    fine = torch.isfinite(xd)
    s = want_scales.repeat_interleave(128, 1)[:, :d]
    far = (got - xd).abs()[fine]
    allowed = torch.maximum(xd.abs() * 2.0 ** -4, s * 2.0 ** -10)[fine]
    assert (far <= allowed).all()


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("T,k,d", [(1, 1, 8), (1, 8, 264), (37, 3, 128), (130, 8, 1544), (5, 32, 40)])
def test_unpack_gathers_exactly(dev, T, k, d, out):
    x = normal((T, d), 1, dev).to(BF)
    (codes, _), (scales, _) = held_buffers(T, d, dev)
    moe.moe_checkpoint_pack(x, codes, scales)
    want = ref.held(x)[0].to(out).to(dev)
    plain, whole = ref.guarded((T, d), out, dev)
    moe.moe_checkpoint_unpack(codes, scales, plain)
    assert torch.equal(plain, want) and ref.guards_intact(whole, plain.numel())
    f2s = torch.randperm(T * k, generator=torch.Generator().manual_seed(2)).to(torch.int32)
    f2s[::5] = -1                                            # dropped assignments
    if T * k > 7:
        f2s[3] = T * k                                       # an entry that names no row
    f2s = f2s.to(dev)
    rows, whole = ref.guarded((T * k, d), out, dev)
    moe.moe_checkpoint_unpack(codes, scales, rows, flat_to_sorted=f2s)
    assert ref.guards_intact(whole, rows.numel())
    left = torch.ones(T * k, dtype=torch.bool, device=dev)
    for i, p in enumerate(f2s.tolist()):
        if 0 <= p < T * k:
            assert torch.equal(rows[p], want[i // k])
            left[p] = False
    assert torch.isnan(rows[left]).all()


def swiglu_tolerances(g, u_, dh, out):
    """fp32 steps: exp and the two divisions or sums are within 4 units (2^-22) each, s within 2^-20 of itself
    after them; 1 - s and 1 + g (1 - s) lose at most that much of 1 + |g|. Eight roundings follow at most."""
    e = 2.0 ** -20
    s = torch.sigmoid(g)
    h, du = (g * s * u_).abs(), (dh * g * s).abs()
    dg = (dh * u_ * s).abs()
    tiny = 1e-37
    return dict(h=e * h + ref.u(out) * h + tiny, du=e * du + ref.u(out) * du + tiny,
                dg=e * dg * (2 + 2 * g.abs()) + ref.u(out) * dg * (1 + g.abs()) + tiny)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,f", [(1, 8), (3, 128), (130, 264), (77, 1544), (1000, 384)])
@pytest.mark.parametrize("use", ["all", "some", "none"])
def test_swiglu_and_its_gradient(dev, dtype, rows, f, use):
    g, u_, dh = (ref.put(normal((rows, f), i, dev, s), dtype, dev) for i, s in ((1, 3.0), (2, 1.0), (3, 1e-3)))
    g[0, :8] = torch.tensor([0.0, -0.0, 90.0, -90.0, 200.0, -200.0, 1e-30, -1.25], dtype=dtype)
    kept = dict(all=rows, some=rows - rows // 3, none=0)[use]
    offsets = None if use == "all" else ref.offsets_of([kept // 2, 0, kept - kept // 2], dev)
    n = slice(0, kept)

    def outputs(names):
        return {m: ref.guarded((rows, f), dtype, dev) for m in names}

    def within(o, want, tol, names):
        for m in names:
            got, whole = o[m]
            assert ref.guards_intact(whole, got.numel()), m
            assert torch.isnan(got[kept:]).all(), f"{m}: wrote rows of no expert"
            off = (got[n].double() - want[m]).abs()
            assert (off <= tol[m]).all(), f"{m}: {(off / tol[m]).max().item():.3f} of the tolerance"

    held = dict(zip("gu", (held_buffers(rows, f, dev), held_buffers(rows, f, dev))))
    kw = {}
    for m in "gu":
        kw[m + "_codes"], kw[m + "_scales"] = held[m][0][0], held[m][1][0]
    o = outputs(["h"])
    moe.moe_swiglu(g, u_, o["h"][0], offsets=offsets, **kw)
    gd, ud, dhd = g[n].double(), u_[n].double(), dh[n].double()
    within(o, dict(h=ref.swiglu(gd, ud)), swiglu_tolerances(gd, ud, dhd, dtype), ["h"])
    alone = outputs(["h"])
    moe.moe_swiglu(g, u_, alone["h"][0], offsets=offsets)
    assert torch.equal(alone["h"][0][n], o["h"][0][n])
    # held as moe_checkpoint_pack holds them
    hold = {}
    for m, src in (("g", g), ("u", u_)):
        hold[m], scales = ref.held(src[n])
        (codes, cw), (sc, sw) = held[m]
        assert ref.guards_intact(cw, codes.numel()) and ref.guards_intact(sw, sc.numel())
        assert torch.equal(sc[n].double().cpu(), scales) and torch.isnan(sc[kept:]).all()
        assert (codes.view(torch.uint8)[kept:] == 0xAB).all()
        hold[m] = hold[m].to(dev)
    # the gradient on the held values, and on g and u themselves
    for gv, uv, args in ((hold["g"], hold["u"], dict(g_scales=kw["g_scales"], u_scales=kw["u_scales"])), (gd, ud, {})):
        src = (kw["g_codes"], kw["u_codes"]) if args else (g, u_)
        want = dict(zip(("dg", "du", "h"), ref.swiglu_backward(dhd, gv, uv)))
        tol = swiglu_tolerances(gv, uv, dhd, dtype)
        o = outputs(["dg", "du", "h"])
        moe.moe_swiglu_backward(dh, *src, o["dg"][0], o["du"][0], h=o["h"][0], offsets=offsets, **args)
        within(o, want, tol, ["dg", "du", "h"])
        few = outputs(["dg", "du"])
        moe.moe_swiglu_backward(dh, *src, few["dg"][0], few["du"][0], offsets=offsets, **args)
        for m in few:
            assert torch.equal(few[m][0][n], o[m][0][n])


def test_swiglu_gradient_against_differences(dev):
    """dg and du against central differences of the 64-bit forward: the difference with step t is off by
    t^2 / 6 of the third derivative (under 2 |u dh| for silu) and by 64-bit rounding."""
    g, u_, dh = (normal((40, 64), i, dev) for i in (1, 2, 3))
    dg, du = torch.empty_like(g), torch.empty_like(g)
    moe.moe_swiglu_backward(dh, g, u_, dg, du)
    gd, ud, dhd, t = g.double(), u_.double(), dh.double(), 1e-4
    num_g = (ref.swiglu(gd + t, ud) - ref.swiglu(gd - t, ud)) / (2 * t) * dhd
    num_u = (ref.swiglu(gd, ud + t) - ref.swiglu(gd, ud - t)) / (2 * t) * dhd
    tol = swiglu_tolerances(gd, ud, dhd, F32)
    extra = t * t * (ud * dhd).abs() + 1e-10
    assert ((dg.double() - num_g).abs() <= tol["dg"] + extra).all()
    assert ((du.double() - num_u).abs() <= tol["du"] + extra).all()


def maps(T, k, E, seed, dev, drop=0):
    """ids [T, k], gates, flat_to_sorted (some entries dropped), as moe_route and moe_permute write them."""
    logits = normal((T, E), seed, dev) - 0.8 * torch.log(torch.arange(1, E + 1, device=dev, dtype=F32))
    top, ids = torch.topk(logits, k, 1)
    order = torch.argsort(ids.reshape(-1), stable=True)
    f2s = torch.empty_like(order)
    f2s[order] = torch.arange(T * k, device=dev)
    f2s = f2s.to(torch.int32)
    if drop:
        f2s[torch.arange(0, T * k, drop, device=dev)] = -1
        if T * k > 9:
            f2s[7] = T * k  # names no row
    return ids.to(torch.int32), torch.softmax(top, 1).contiguous(), f2s


@pytest.mark.parametrize("dy_t,out", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("T,k,E,d", [(1, 1, 1, 8), (1, 8, 16, 7168), (9, 3, 8, 128), (64, 8, 64, 1032), (130, 32, 40, 264),
                                     (77, 5, 9, 1024)])
@pytest.mark.parametrize("drop", [0, 4])
def test_combine_and_permute_backward(dev, dy_t, out, T, k, E, d, drop):
    _, gates, f2s = maps(T, k, E, 1, dev, drop)
    R = T * k
    dy, ys = ref.put(normal((T, d), 2, dev, 1e-3), dy_t, dev), ref.put(normal((R, d), 3, dev), F32, dev)
    f = f2s.long()
    used = (f >= 0) & (f < R)
    left = torch.ones(R, dtype=torch.bool, device=dev)
    left[f[used]] = False
    ys[left] = float("nan")                                    # rows of dropped assignments hold nothing
    dys, w1 = ref.guarded((R, d), out, dev)
    dgates, w2 = ref.guarded((T, k), F32, dev)
    moe.moe_combine_backward(dy, ys, f2s, gates, dys, dgates)
    assert ref.guards_intact(w1, dys.numel()) and ref.guards_intact(w2, dgates.numel())
    per = dy.double().repeat_interleave(k, 0)
    want = gates.double().reshape(-1, 1) * per
    off = (dys[f[used]].double() - want[used]).abs()
    assert (off <= (ref.u(out) + ref.u(F32) * 2) * want[used].abs() + 1e-40).all()
    assert torch.isnan(dys[left]).all()
    rows = torch.where(used, f, torch.zeros_like(f))
    prod = per * ys[rows].double()
    wg = torch.where(used, prod.sum(1), torch.zeros(1, device=dev, dtype=torch.float64))
    size = torch.where(used, prod.abs().sum(1), torch.zeros(1, device=dev, dtype=torch.float64))
    assert ((dgates.reshape(-1).double() - wg).abs() <= d * 2.0 ** -23 * size).all()
    assert (dgates.reshape(-1)[~used] == 0).all()
    alone, _ = ref.guarded((R, d), out, dev)
    moe.moe_combine_backward(dy, None, f2s, gates, alone, None)
    assert torch.equal(alone.nan_to_num(0), dys.nan_to_num(0))

    dxs = ref.put(normal((R, d), 4, dev), dy_t, dev)
    dxs[left] = float("nan")
    dx, w3 = ref.guarded((T, d), out, dev)
    moe.moe_permute_backward(dxs, f2s, k, dx)
    assert ref.guards_intact(w3, dx.numel())
    part = torch.where(used.reshape(-1, 1), dxs[rows].double(), torch.zeros(1, device=dev, dtype=torch.float64)).reshape(T, k, d)
    want, size = part.sum(1), part.abs().sum(1)
    assert ((dx.double() - want).abs() <= k * 2.0 ** -23 * size * 2 + ref.u(out) * want.abs()).all()


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 8), (5, 2, 8), (64, 8, 63), (65, 8, 64), (130, 3, 65), (33, 32, 1024),
                                   (70, 8, 256)])
def test_route_backward(dev, T, k, E):
    ids, gates, _ = maps(T, k, E, 5, dev)
    dgates = ref.put(normal((T, k), 6, dev), F32, dev)
    dl, whole = ref.guarded((T, E), F32, dev)
    moe.moe_route_backward(dgates, ids, gates, dl)
    assert ref.guards_intact(whole, dl.numel())
    g, dg = gates.double(), dgates.double()
    mean, size = (g * dg).sum(1, keepdim=True), (g * dg.abs()).sum(1, keepdim=True)
    want = torch.zeros((T, E), dtype=torch.float64, device=dev).scatter_(1, ids.long(), g * (dg - mean))
    tol = torch.zeros_like(want).scatter_(1, ids.long(), g * ((k + 2) * 2.0 ** -23 * size + 2.0 ** -22 * dg.abs()))
    assert ((dl.double() - want).abs() <= tol).all()   # outside the chosen experts: exactly 0


def test_route_backward_with_ids_out_of_range_or_twice(dev):
    ids = torch.tensor([[0, 9, 3], [2, 2, 1], [-1, 4, 7]], dtype=torch.int32, device=dev)
    gates = torch.full((3, 3), 1 / 3, device=dev)
    dg = torch.tensor([[1.0, 2.0, 6.0]] * 3, device=dev)
    dl, whole = ref.guarded((3, 8), F32, dev)
    moe.moe_route_backward(dg, ids, gates, dl)
    assert ref.guards_intact(whole, dl.numel())
    v = (dg[0].double() - 3) / 3
    want = torch.zeros((3, 8), dtype=torch.float64, device=dev)
    want[0, 0], want[0, 3] = v[0], v[2]
    want[1, 2], want[1, 1] = v[0] + v[1], v[2]
    want[2, 4], want[2, 7] = v[1], v[2]
    assert (dl.double() - want).abs().max() <= 1e-6


def test_no_tokens(dev):
    e = lambda *s, t=F32: torch.empty(s, dtype=t, device=dev)  # noqa: E731
    i32 = torch.int32
    moe.moe_checkpoint_pack(e(0, 16), e(0, 16, t=F8), e(0, 1))
    moe.moe_checkpoint_unpack(e(0, 16, t=F8), e(0, 1), e(0, 16))
    moe.moe_swiglu(e(0, 16), e(0, 16), e(0, 16))
    moe.moe_swiglu_backward(e(0, 16), e(0, 16), e(0, 16), e(0, 16), e(0, 16))
    moe.moe_combine_backward(e(0, 16), e(0, 16), e(0, t=i32), e(0, 2), e(0, 16), e(0, 2))
    moe.moe_permute_backward(e(0, 16), e(0, t=i32), 2, e(0, 16))
    moe.moe_route_backward(e(0, 2), e(0, 2, t=i32), e(0, 2), e(0, 4))
    torch.cuda.synchronize()


# ----------------------------------------------------------------------------------------------
# a layer's training step
# ----------------------------------------------------------------------------------------------
class Step:
    """One training step of the layer out of the library's calls, with the buffers a user keeps."""

    def __init__(self, T, E, k, d, f, dtype, dev, held, capacity=None, seed=1):
        self.k, self.E, self.held, self.capacity = k, E, held, capacity
        n = lambda shape, s, scale=1.0: normal(shape, seed * 100 + s, dev, scale).to(dtype)  # noqa: E731
        self.logits = normal((T, E), seed * 100, dev)
        self.x, self.dy = n((T, d), 1), n((T, d), 2, 1e-2)
        self.wg, self.wu, self.wd = n((E, f, d), 3, d ** -0.5), n((E, f, d), 4, d ** -0.5), n((E, d, f), 5, f ** -0.5)
        R = T * k
        z = lambda shape, t=dtype: torch.full(shape, float("nan"), dtype=t, device=dev)  # noqa: E731
        i = lambda shape: torch.full(shape, -7, dtype=torch.int32, device=dev)  # noqa: E731
        q = lambda c: (torch.zeros((c[0], c[1]), dtype=F8, device=dev), z((c[0], -(-c[1] // 128)), F32))  # noqa: E731
        self.b = dict(ids=i((T, k)), gates=z((T, k), F32), counts=i((E,)), offsets=i((E + 1,)), s2f=i((R,)), f2s=i((R,)),
                      xs=z((R, d)), g=z((R, f)), u=z((R, f)), h=z((R, f)), ys=z((R, d), F32), y=z((T, d), F32),
                      x8=q((T, d)), g8=q((R, f)), u8=q((R, f)),
                      dys=z((R, d)), dgates=z((T, k), F32), dh=z((R, f)), dg=z((R, f)), du=z((R, f)), h2=z((R, f)),
                      dxs=z((R, d), F32), dx=z((T, d), F32), dlogits=z((T, E), F32),
                      dwg=z((E, f, d), F32), dwu=z((E, f, d), F32), dwd=z((E, d, f), F32))
        self.ws = moe.Workspace(moe.moe_permute_workspace_size(T, E, k), device=dev)

    def forward(self):
        b = self.b
        moe.moe_route(self.logits, self.k, b["ids"], b["gates"])
        moe.moe_permute(self.x, b["ids"], self.E, b["counts"], b["offsets"], b["s2f"], b["f2s"], b["xs"], self.ws,
                        capacity=self.capacity)
        moe.moe_grouped_gemm(b["xs"], b["offsets"], self.wg, b["g"])
        moe.moe_grouped_gemm(b["xs"], b["offsets"], self.wu, b["u"])
        if self.held:
            moe.moe_checkpoint_pack(self.x, *b["x8"])
            moe.moe_swiglu(b["g"], b["u"], b["h"], *b["g8"], *b["u8"], offsets=b["offsets"])
        else:
            moe.moe_swiglu(b["g"], b["u"], b["h"], offsets=b["offsets"])
        moe.moe_grouped_gemm(b["h"], b["offsets"], self.wd, b["ys"])
        moe.moe_combine(b["ys"], b["f2s"], b["gates"], b["y"])

    def backward(self):
        b = self.b
        off = b["offsets"]
        moe.moe_combine_backward(self.dy, b["ys"], b["f2s"], b["gates"], b["dys"], b["dgates"])
        moe.moe_route_backward(b["dgates"], b["ids"], b["gates"], b["dlogits"])
        moe.moe_grouped_gemm_dgrad(b["dys"], off, self.wd, b["dh"])
        if self.held:
            moe.moe_checkpoint_unpack(*b["x8"], b["xs"], flat_to_sorted=b["f2s"])
            moe.moe_swiglu_backward(b["dh"], b["g8"][0], b["u8"][0], b["dg"], b["du"], h=b["h2"], g_scales=b["g8"][1],
                                    u_scales=b["u8"][1], offsets=off)
        else:
            moe.moe_swiglu_backward(b["dh"], b["g"], b["u"], b["dg"], b["du"], h=b["h2"], offsets=off)
        moe.moe_grouped_gemm_wgrad(b["dys"], b["h2"], off, b["dwd"])
        moe.moe_grouped_gemm_wgrad(b["dg"], b["xs"], off, b["dwg"])
        moe.moe_grouped_gemm_wgrad(b["du"], b["xs"], off, b["dwu"])
        moe.moe_grouped_gemm_dgrad(b["dg"], off, self.wg, b["dxs"], dy2=b["du"], w2=self.wu)
        moe.moe_permute_backward(b["dxs"], b["f2s"], self.k, b["dx"])

    def reference(self):
        """y and the gradients by autograd in 64 bits, for the library's routing. With held activations the
        backward pass sees the held x, g and u (straight through the rounding)."""
        leaf = lambda t: t.double().clone().requires_grad_(True)  # noqa: E731
        logits, x = leaf(self.logits), leaf(self.x)
        wg, wu, wd = leaf(self.wg), leaf(self.wu), leaf(self.wd)
        b = self.b
        ids = b["ids"].long()
        gates = torch.softmax(torch.gather(logits, 1, ids), 1)
        y = torch.zeros_like(x)
        f2s = b["f2s"].reshape(ids.shape)
        for e in range(self.E):
            tok, slot = torch.nonzero((ids == e) & (f2s >= 0), as_tuple=True)
            if tok.numel() == 0:
                continue
            h = torch.nn.functional.silu(x[tok] @ wg[e].t()) * (x[tok] @ wu[e].t())
            y = y.index_add(0, tok, gates[tok, slot].unsqueeze(1) * (h @ wd[e].t()))
        y.backward(self.dy.double())
        return dict(y=y.detach(), dx=x.grad, dlogits=logits.grad, dwg=wg.grad, dwu=wu.grad, dwd=wd.grad)


def relative(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("T,E,k,d,f", [(1, 8, 2, 64, 72), (40, 8, 2, 136, 264), (96, 16, 4, 256, 384)])
@pytest.mark.parametrize("capacity", [None, 6])
def test_training_step_f32(dev, T, E, k, d, f, capacity):
    """fp32 throughout. Each of the 8 operators on a gradient's way adds at most n 2^-23 of its sums' absolute
    size (n up to 384: 4.6e-5); sums of random terms cancel to about the root of that, and the bar is 100
    units, 1.2e-5, times 8."""
    s = Step(T, E, k, d, f, F32, dev, held=False, capacity=capacity)
    s.forward()
    s.backward()
    for name, want in s.reference().items():
        err = relative(s.b[name], want)
        print(f"T={T} capacity={capacity} {name}: {err:.2e}", flush=True)
        assert err <= 1e-4, name


@pytest.mark.parametrize("T,E,k,d,f", [(40, 8, 2, 136, 264), (700, 16, 4, 256, 384), (600, 4, 2, 1032, 520)])
@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("capacity", [None, 50])
def test_training_step_bf16(dev, T, E, k, d, f, held, capacity):
    """bf16 activations and gradients: a gradient passes at most 8 roundings to bf16 (2^-9 rms each, 2^-8 at
    most): 8 * 2^-8 = 3.2e-2. Held activations: two more factors with at most 2^-4 each, 1.3e-1 together, on
    what depends on them; y does not."""
    s = Step(T, E, k, d, f, BF, dev, held=held, capacity=capacity)
    s.forward()
    s.backward()
    for name, want in s.reference().items():
        err = relative(s.b[name], want)
        print(f"T={T} held={held} capacity={capacity} {name}: {err:.2e}", flush=True)
        assert err <= (3.2e-2 if not held or name in ("y", "dlogits") else 3.2e-2 + 1.3e-1), name


@pytest.mark.parametrize("T,E,k,d,f,dtype", [(48, 8, 2, 128, 256, BF), (700, 16, 4, 256, 384, BF), (33, 8, 2, 128, 72, F32)])
def test_training_step_captured_and_replayed(dev, T, E, k, d, f, dtype):
    """The whole step in a graph; every replay against the eager step, with new inputs, an eager step of other
    tensors in between, and two graphs that share no buffers replayed in turn."""
    steps = [Step(T, E, k, d, f, dtype, dev, held=True, seed=i + 1) for i in range(2)]
    other = Step(T + 9, E, k, d, f, dtype, dev, held=False, seed=5)
    stream, graphs = torch.cuda.Stream(), []
    for s in steps:
        s.forward(), s.backward()                 # once before the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            s.forward()
            s.backward()
        graphs.append(g)
    names = ("y", "dx", "dlogits", "dwg", "dwu", "dwd")
    for rep in range(4):
        for i, (s, g) in enumerate(zip(steps, graphs)):
            s.x.copy_(normal(tuple(s.x.shape), 1000 + 10 * rep + i, dev))
            s.logits.copy_(normal(tuple(s.logits.shape), 2000 + 10 * rep + i, dev))
            for n in names:
                s.b[n].fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            got = {n: s.b[n].clone() for n in names}
            other.forward(), other.backward()
            s.forward(), s.backward()
            torch.cuda.synchronize()
            for n in names:
                assert torch.equal(got[n], s.b[n]), (rep, i, n)


def test_two_training_steps_at_once(dev):
    """Two steps of their own tensors, their calls dealt in turn to two streams, against the same steps alone."""
    names = ("y", "dx", "dlogits", "dwg", "dwu", "dwd")
    steps = [Step(700, 16, 4, 256, 384, BF, dev, held=True, seed=1), Step(90, 8, 2, 136, 264, F32, dev, held=True, seed=2)]
    alone = []
    for s in steps:
        s.forward(), s.backward()
        torch.cuda.synchronize()
        alone.append({n: s.b[n].clone() for n in names})
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        for s in steps:
            for n in names:
                s.b[n].fill_(float("nan"))
        torch.cuda.synchronize()
        for part in ("forward", "backward"):
            for s, stream in zip(steps, streams):
                with torch.cuda.stream(stream):
                    getattr(s, part)()
        torch.cuda.synchronize()
        for s, want in zip(steps, alone):
            for n in names:
                assert torch.equal(s.b[n], want[n]), (rep, n)


def test_calls_run_on_the_stream_they_are_given(dev):
    """Inputs arrive late on a side stream that is not the current one; only calls on that stream see them."""
    T, E, k, d = 200, 8, 2, 264
    R, side = T * k, torch.cuda.Stream()
    f2s = torch.randperm(R, generator=torch.Generator().manual_seed(3)).to(dev, torch.int32)
    off = ref.offsets_of([R // E] * E, dev)
    gates, ids = torch.rand((T, k), device=dev), torch.arange(R, device=dev).reshape(T, k).remainder(E).to(torch.int32)
    late = {n: normal(shape, 40 + i, dev) for i, (n, shape) in enumerate(dict(x=(T, d), r=(R, d), q=(R, d), g=(T, k), w=(E, d, d)).items())}
    slow = torch.zeros((4096, 4096), device=dev)

    def run(t, stream):
        z = lambda *s, t=F32: torch.empty(s, dtype=t, device=dev)  # noqa: E731
        held = lambda n: (z(n, d, t=F8), z(n, -(-d // 128)))  # noqa: E731
        o = dict(xc=held(T), up=z(R, d), gc=held(R), uc=held(R), h=z(R, d), dg=z(R, d), du=z(R, d), dys=z(R, d), dgates=z(T, k),
                 dx=z(T, d), dl=z(T, E), y=z(R, d), dxs=z(R, d), dw=z(E, d, d))
        torch.cuda.current_stream().synchronize()  # the buffers' earlier uses are over
        moe.moe_checkpoint_pack(t["x"], *o["xc"], stream=stream)
        moe.moe_checkpoint_unpack(*o["xc"], o["up"], flat_to_sorted=f2s, stream=stream)
        moe.moe_swiglu(t["r"], t["q"], o["h"], *o["gc"], *o["uc"], stream=stream)
        moe.moe_swiglu_backward(t["q"], o["gc"][0], o["uc"][0], o["dg"], o["du"], g_scales=o["gc"][1], u_scales=o["uc"][1], stream=stream)
        moe.moe_combine_backward(t["x"], t["r"], f2s, gates, o["dys"], o["dgates"], stream=stream)
        moe.moe_permute_backward(t["r"], f2s, k, o["dx"], stream=stream)
        moe.moe_route_backward(t["g"], ids, gates, o["dl"], stream=stream)
        moe.moe_grouped_gemm(t["r"], off, t["w"], o["y"], stream=stream)
        moe.moe_grouped_gemm_dgrad(t["r"], off, t["w"], o["dxs"], stream=stream)
        moe.moe_grouped_gemm_wgrad(t["r"], t["q"], off, o["dw"], stream=stream)
        return o
    want = run(late, None)
    torch.cuda.synchronize()
    t = {n: torch.zeros_like(v) for n, v in late.items()}
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            slow.addmm_(slow, slow)
        for n, v in t.items():
            v.copy_(late[n])
    got = run(t, side)
    torch.cuda.synchronize()
    for n, v in want.items():
        for a, b in zip(v if isinstance(v, tuple) else (v,), got[n] if isinstance(v, tuple) else (got[n],)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), n


def test_rows_past_32_bits(dev):
    """Element offsets past 2^32 in every row-wise call, checked on the last rows."""
    T, k, d = 75000, 8, 7168                                 # 4.3e9 elements in the sorted rows
    R, m = T * k, 16
    f2s = torch.arange(R, device=dev, dtype=torch.int32)     # token t's rows are t*k .. t*k + k - 1
    gates = torch.full((T, k), 0.5, device=dev)
    x = torch.zeros((T, d), dtype=BF, device=dev)
    x[-2:] = normal((2, d), 1, dev)
    ys = torch.zeros((R, d), device=dev)
    ys[-m:] = normal((m, d), 2, dev)
    rows, dgates = torch.full((R, d), float("nan"), dtype=BF, device=dev), torch.empty((T, k), device=dev)
    moe.moe_combine_backward(x, ys, f2s, gates, rows, dgates)
    last = x[-2:].repeat_interleave(k, 0)
    assert torch.equal(rows[-m:], (last.float() * 0.5).to(BF)) and (rows[:m] == 0).all()
    want = (last.double() * ys[-m:].double()).sum(1)
    assert (dgates[-2:].reshape(-1).double() - want).abs().max() <= d * 2.0 ** -23 * (last.double() * ys[-m:].double()).abs().sum(1).max()
    del ys
    codes, scales = torch.empty((T, d), dtype=F8, device=dev), torch.empty((T, d // 128), device=dev)
    moe.moe_checkpoint_pack(x, codes, scales)
    rows.fill_(float("nan"))
    moe.moe_checkpoint_unpack(codes, scales, rows, flat_to_sorted=f2s)
    assert torch.equal(rows[-m:], ref.held(x[-2:])[0].to(BF).to(dev).repeat_interleave(k, 0)) and not torch.isnan(rows).any()
    dx = torch.empty((T, d), device=dev)
    moe.moe_permute_backward(rows, f2s, k, dx)
    assert torch.equal(dx[-2:].double(), rows[-m:].double().reshape(2, k, d).sum(1)) and (dx[0] == 0).all()
    # 4.4e9 elements of the activations
    g = rows
    g.zero_()
    g[-m:] = normal((m, d), 3, dev)
    u_, h = g.clone(), torch.full_like(g, float("nan"))
    c = [torch.empty((R, d), dtype=F8, device=dev) for _ in range(2)]
    s = [torch.empty((R, d // 128), device=dev) for _ in range(2)]
    moe.moe_swiglu(g, u_, h, c[0], s[0], c[1], s[1])
    gd = g[-m:].double()
    tol = swiglu_tolerances(gd, gd, gd, BF)
    assert ((h[-m:].double() - ref.swiglu(gd, gd)).abs() <= tol["h"]).all() and (h[:m] == 0).all()
    hold = ref.held(g[-m:])[0].to(dev)
    dg, du = u_, g  # (their values are held in 8 bits now)
    dh = h.fill_(0.0)
    dh[-m:] = 1.0
    moe.moe_swiglu_backward(dh, c[0], c[1], dg, du, g_scales=s[0], u_scales=s[1])
    one = torch.ones_like(hold)
    want = dict(zip(("dg", "du", "h"), ref.swiglu_backward(one, hold, hold)))
    tol = swiglu_tolerances(hold, hold, one, BF)
    assert ((dg[-m:].double() - want["dg"]).abs() <= tol["dg"]).all()
    assert ((du[-m:].double() - want["du"]).abs() <= tol["du"]).all()
