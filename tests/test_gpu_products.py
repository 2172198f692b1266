"""Matrix products grouped by expert (forward, input gradient, weight gradient) against 64-bit
references: exactly where whole numbers make the fp32 sums exact, else within the bound derived in
training_ref. Inputs lie in NaN (rows of no expert, weights of experts without rows, memory around
the tensors), outputs in guarded buffers."""
import pytest
import torch

import token_dispatch_expert_amd as moe

import gpu_harness as H
import training_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    return H.require_gpu()


def whole_numbers(shape, seed, dev, most=4):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, dtype=torch.int16).to(dev).float()


def inputs(counts, spare, N, K, dtype, dev, seed, make=whole_numbers):
    """x, dy (spare NaN rows behind the last expert's), w (NaN where an expert has no rows), offsets."""
    n = sum(counts)
    t = dict(offsets=ref.offsets_of(counts, dev))
    for name, c, s in (("x", K, 1), ("dy", N, 2), ("dy2", N, 3)):
        v = torch.full((n + spare, c), float("nan"), device=dev)
        v[:n] = make((n, c), 10 * seed + s, dev)
        t[name] = ref.put(v, dtype, dev)
    for name, s in (("w", 4), ("w2", 5)):
        v = make((len(counts), N, K), 10 * seed + s, dev)
        for e, c in enumerate(counts):
            if c == 0:
                v[e] = float("nan")
        t[name] = ref.put(v, dtype, dev)
    return t


def check(got, whole, want, scale, n_sum, out_dtype, what):
    """got against the 64-bit result `want`; scale: sum |a||b| (None: the sum is exact)."""
    assert ref.guards_intact(whole, got.numel()), f"{what}: wrote outside its buffer"
    n = want.shape[0]
    g = got[:n]
    if scale is None:
        exact = want.to(out_dtype)
        bad = torch.nonzero(g != exact)
        assert bad.numel() == 0, f"{what}: {bad.shape[0]} values differ, first at {bad[0].tolist()}"
    else:
        bound = n_sum * 2.0 ** -23 * scale + ref.u(out_dtype) * (want.abs() + n_sum * 2.0 ** -23 * scale)
        worst = ((g.double() - want).abs() / bound.clamp(min=1e-300)).max().item()
        print(f"{what}: worst error {worst:.3f} of its bound", flush=True)
        assert worst <= 1.0, what
    if got.shape[0] > n:
        assert torch.isnan(got[n:]).all(), f"{what}: wrote rows of no expert"


def run_all(counts, spare, N, K, dtype, out, dev, seed=1, make=whole_numbers, exact=True):
    t = inputs(counts, spare, N, K, dtype, dev, seed, make)
    n, E = sum(counts), len(counts)
    size = lambda f, *a: None if exact else f(*[v[:n].abs() if v.dim() == 2 else v.abs() for v in a], counts)  # noqa: E731
    tag = f"counts {counts if E < 9 else E} N {N} K {K} {dtype} -> {out}"

    y, whole = ref.guarded((n + spare, N), out, dev)
    moe.moe_grouped_gemm(t["x"], t["offsets"], t["w"], y)
    check(y, whole, ref.forward(t["x"], t["w"], counts), size(ref.forward, t["x"], t["w"]), K, out, "forward " + tag)

    dx, whole = ref.guarded((n + spare, K), out, dev)
    moe.moe_grouped_gemm_dgrad(t["dy"], t["offsets"], t["w"], dx)
    one, one_size = ref.dgrad(t["dy"], t["w"], counts), size(ref.dgrad, t["dy"], t["w"])
    check(dx, whole, one, one_size, N, out, "dgrad " + tag)

    dx, whole = ref.guarded((n + spare, K), out, dev)
    moe.moe_grouped_gemm_dgrad(t["dy"], t["offsets"], t["w"], dx, dy2=t["dy2"], w2=t["w2"])
    two_size = None if exact else one_size + size(ref.dgrad, t["dy2"], t["w2"])
    check(dx, whole, one + ref.dgrad(t["dy2"], t["w2"], counts), two_size, 2 * N, out, "dgrad of two " + tag)

    dw, whole = ref.guarded((E, N, K), out, dev)
    moe.moe_grouped_gemm_wgrad(t["dy"], t["x"], t["offsets"], dw)
    want, w_size = ref.wgrad(t["dy"][:n], t["x"][:n], counts), size(ref.wgrad, t["dy"], t["x"])
    most = max(counts, default=0)
    check(dw, whole, want, w_size, most, out, "wgrad " + tag)

    if exact:  # into what is there (whole numbers: one exact sum)
        old = whole_numbers((E, N, K), 77, dev, 100)
        dw, whole = ref.guarded((E, N, K), out, dev)
        dw.copy_(old)
        moe.moe_grouped_gemm_wgrad(t["dy"], t["x"], t["offsets"], dw, accumulate=True)
        check(dw, whole, want + old.double(), None, 0, out, "wgrad accumulated " + tag)


# rows per expert around the tiles' sizes, experts without rows first, between and last
COUNTS = [
    [1], [0, 0, 3, 0], [0, 1, 63, 64, 65, 0], [128, 127, 0, 129, 2], [257, 255, 256, 1, 0, 31],
    [16, 17, 15, 32, 33, 31, 1, 0, 8], [700, 0, 5],
]
WIDTHS = [(8, 8), (64, 72), (136, 264), (256, 512), (264, 40), (520, 1032)]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("N,K", WIDTHS)
def test_bf16_products_exact(dev, counts, N, K):
    run_all(counts, 5, N, K, BF, F32, dev, seed=3)


@pytest.mark.parametrize("counts", [COUNTS[1], COUNTS[3], COUNTS[4]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("N,K", [(8, 8), (136, 264), (264, 40)])
def test_bf16_products_rounded_to_bf16(dev, counts, N, K):
    run_all(counts, 0, N, K, BF, BF, dev, seed=4)


@pytest.mark.parametrize("counts", [COUNTS[1], COUNTS[2], COUNTS[3]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("N,K", [(8, 8), (64, 72), (136, 264), (264, 40)])
@pytest.mark.parametrize("out", [F32, BF])
def test_f32_products_exact(dev, counts, N, K, out):
    run_all(counts, 3, N, K, F32, out, dev, seed=5)


@pytest.mark.parametrize("counts,N,K", [
    ([40] * 3 + [0] * 5, 512, 4096), ([3, 0, 1, 2, 1, 1] * 6, 384, 640), ([600, 100, 0, 36], 1024, 896)])
def test_bf16_products_longer(dev, counts, N, K):
    run_all(counts, 0, N, K, BF, F32, dev, seed=6)


def normal(shape, seed, dev):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(shape, generator=g, device=dev)


@pytest.mark.parametrize("dtype,out", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("counts,N,K", [([5, 300, 0, 77], 200, 328), ([2, 1, 0, 0, 9], 768, 2048), ([1025, 511], 264, 712)])
def test_products_of_normal_values(dev, dtype, out, counts, N, K):
    run_all(counts, 2, N, K, dtype, out, dev, seed=7, make=normal, exact=False)


def test_no_rows(dev):
    """rows = 0, and rows that belong to no expert: nothing is written but the weight gradient's zeros."""
    for rows in (0, 6):
        off = torch.zeros(4, dtype=torch.int32, device=dev)
        x, dy = (torch.full((rows, c), float("nan"), dtype=BF, device=dev) for c in (24, 16))
        w = torch.full((3, 16, 24), float("nan"), dtype=BF, device=dev)
        y, whole_y = ref.guarded((rows, 16), F32, dev)
        dx, whole_x = ref.guarded((rows, 24), F32, dev)
        moe.moe_grouped_gemm(x, off, w, y)
        moe.moe_grouped_gemm_dgrad(dy, off, w, dx)
        assert torch.isnan(whole_y).all() and torch.isnan(whole_x).all()
        dw, whole = ref.guarded((3, 16, 24), F32, dev)
        moe.moe_grouped_gemm_wgrad(dy, x, off, dw, accumulate=True)
        assert torch.isnan(whole).all()
        moe.moe_grouped_gemm_wgrad(dy, x, off, dw)
        assert (dw == 0).all() and ref.guards_intact(whole, dw.numel())


def test_most_experts(dev):
    counts = [(7 * e) % 5 for e in range(1024)]
    run_all(counts, 0, 16, 24, BF, F32, dev, seed=8)
    run_all(counts, 0, 16, 24, F32, F32, dev, seed=8)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_non_finite_values_stay_in_their_place(dev, value):
    """One non-finite x and dy element reaches the outputs that contain it and no others: also where
    tiles hang over an expert's end, into the next expert's rows."""
    counts, N, K = [70, 0, 59, 3], 72, 136
    t = inputs(counts, 0, N, K, BF, dev, seed=9, make=normal)
    clean = {}
    for bad in (False, True):
        if bad:
            t["x"][70, 100] = value   # the first row of expert 2
            t["dy"][70, 3] = value
        y = torch.empty((132, N), device=dev)
        dx, dw = torch.empty((132, K), device=dev), torch.empty((4, N, K), device=dev)
        moe.moe_grouped_gemm(t["x"], t["offsets"], t["w"], y)
        moe.moe_grouped_gemm_dgrad(t["dy"], t["offsets"], t["w"], dx)
        moe.moe_grouped_gemm_wgrad(t["dy"], t["x"], t["offsets"], dw)
        if not bad:
            clean = dict(y=y, dx=dx, dw=dw)
            continue
        for name, got in dict(y=y, dx=dx).items():
            hit = torch.zeros_like(got, dtype=torch.bool)
            hit[70] = True
            assert not torch.isfinite(got[hit]).any(), name
            assert torch.equal(got[~hit], clean[name][~hit]), name
        hit = torch.zeros_like(dw, dtype=torch.bool)
        hit[2, 3, :] = True
        hit[2, :, 100] = True
        assert not torch.isfinite(dw[hit]).any()
        assert torch.equal(dw[~hit], clean["dw"][~hit])


def test_offsets_past_32_bits(dev):
    """Operands and results whose byte and element offsets pass 2^32: the last expert's rows, checked alone."""
    counts, N, K = [65600, 30], 32, 65536     # x: 4.3e9 elements
    n = sum(counts)
    off = ref.offsets_of(counts, dev)
    x = torch.zeros((n, K), dtype=BF, device=dev)
    x[65600:] = whole_numbers((30, K), 1, dev, 1)
    w = whole_numbers((2, N, K), 2, dev, 1).to(BF)
    dy = torch.zeros((n, N), dtype=BF, device=dev)
    dy[65600:] = whole_numbers((30, N), 3, dev, 1)
    y = torch.empty((n, N), device=dev)
    moe.moe_grouped_gemm(x, off, w, y)
    assert torch.equal(y[65600:].double(), x[65600:].double() @ w[1].double().t()) and (y[:65600] == 0).all()
    dx = torch.full((n, K), float("nan"), dtype=BF, device=dev)
    moe.moe_grouped_gemm_dgrad(dy, off, w, dx)
    assert torch.equal(dx[65600:], (dy[65600:].double() @ w[1].double()).to(BF))
    assert not torch.isnan(dx).any()
    del dx
    dw = torch.empty((2, N, K), device=dev)
    moe.moe_grouped_gemm_wgrad(dy, x, off, dw)
    assert torch.equal(dw[1].double(), dy[65600:].double().t() @ x[65600:].double()) and (dw[0] == 0).all()
    del x
    # weights and their gradient
    E, N, K = 70, 8192, 8192                  # 4.7e9 elements
    counts = [0] * (E - 1) + [20]
    off = ref.offsets_of(counts, dev)
    w = torch.zeros((E, N, K), dtype=BF, device=dev)
    w[-1] = whole_numbers((N, K), 4, dev, 1)
    x, dy = whole_numbers((20, K), 5, dev, 1).to(BF), whole_numbers((20, N), 6, dev, 1).to(BF)
    y, dx = torch.empty((20, N), device=dev), torch.empty((20, K), device=dev)
    moe.moe_grouped_gemm(x, off, w, y)
    moe.moe_grouped_gemm_dgrad(dy, off, w, dx)
    assert torch.equal(y.double(), x.double() @ w[-1].double().t())
    assert torch.equal(dx.double(), dy.double() @ w[-1].double())
    w.fill_(float("nan"))
    moe.moe_grouped_gemm_wgrad(dy, x, off, w)
    assert torch.equal(w[-1], (dy.double().t() @ x.double()).to(BF)) and (w[:-1] == 0).all()


def test_same_bits_every_call_and_on_another_stream(dev):
    counts, N, K = [130, 0, 300, 7, 64], 264, 520
    t = inputs(counts, 0, N, K, BF, dev, seed=11, make=normal)
    outs = []
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s in streams:  # the two side streams' calls may overlap
        y = torch.full((sum(counts), N), float("nan"), device=dev)
        dx, dw = torch.full((sum(counts), K), float("nan"), device=dev), torch.full((5, N, K), float("nan"), device=dev)
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        moe.moe_grouped_gemm(t["x"], t["offsets"], t["w"], y, stream=s)
        moe.moe_grouped_gemm_dgrad(t["dy"], t["offsets"], t["w"], dx, stream=s)
        moe.moe_grouped_gemm_wgrad(t["dy"], t["x"], t["offsets"], dw, stream=s)
        outs.append((y, dx, dw))
    torch.cuda.synchronize()
    for o in outs[1:]:
        for a, b in zip(o, outs[0]):
            assert torch.equal(a, b)


# Sizes with enough rows and tiles for each kind of tile that the library chooses among (see the rule in
# grouped_gemm.hip): 256 x 256, 128 x 128, 64 x 128 and the few-row tiles, with partial tiles on every side
@pytest.mark.parametrize("counts,N,K", [
    ([1500, 0, 17, 2579], 2056, 520),           # 256 x 256 forward
    ([1300, 900, 0, 1900], 520, 2056),          # 256 x 256 input gradient
    ([700, 5, 0, 1200, 300, 64, 1, 800], 1800, 2056),   # 256 x 256 weight gradient
    ([150] * 20 + [0, 3, 290], 1032, 1160),     # 128 x 128
    ([30, 0, 55, 70] * 8, 392, 1160),           # 64 x 128
    ([3, 1, 0, 14] * 30, 1544, 264),            # few rows
], ids=["large-forward", "large-dgrad", "large-wgrad", "middle", "small", "few"])
@pytest.mark.parametrize("out", [F32, BF])
def test_every_tile_size_exact(dev, counts, N, K, out):
    run_all(counts, 3, N, K, BF, out, dev, seed=12)


# Few tiles, each with a CU of its own (of 32, 64 and 128 rows), with more steps than the ring has slots, fewer, or a
# part of one; and one case of tiles of 64 rows past that
@pytest.mark.parametrize("counts,N,K", [
    ([40, 0, 3], 1544, 4104), ([1], 4104, 136), ([33], 72, 2056), ([5, 64, 0, 31], 776, 904), ([200], 648, 776), ([7, 9], 392, 520),
    ([300, 500, 0, 900, 260], 1160, 1160), ([30, 0, 55, 70] * 5, 520, 776), ([30, 0, 55, 70] * 8, 2056, 2056), ([1900], 264, 392),
], ids=lambda v: "-".join(map(str, v)) if isinstance(v, list) else str(v))
@pytest.mark.parametrize("out", [F32, BF])
def test_few_tiles_of_long_sums_exact(dev, counts, N, K, out):
    run_all(counts, 2, N, K, BF, out, dev, seed=17)


# fp32: 16 x 64 tiles with the contraction whole and split in four, 64 x 64 ones whole and split in two
@pytest.mark.parametrize("counts,N,K", [
    ([20] * 40 + [0, 47], 1160, 1160), ([3, 0, 1] * 20, 1032, 264), ([26], 3800, 104), ([300, 0, 517, 100], 1032, 1160),
    ([900, 0, 1300, 700], 1032, 1160), ([700, 0, 333], 264, 392),
], ids=["16-rows", "16-rows-split", "16-rows-split-long", "64-rows-split", "64-rows", "wgrad-split"])
@pytest.mark.parametrize("out", [F32, BF])
def test_every_fp32_tile_exact(dev, counts, N, K, out):
    run_all(counts, 3, N, K, F32, out, dev, seed=18)


@pytest.mark.parametrize("N,K", [(136, 1 << 20), (1 << 20, 72)])
@pytest.mark.parametrize("counts,dtype", [([40, 3], BF), ([300, 0], BF), ([40, 3], F32)], ids=["few-bf16", "bf16", "f32"])
def test_widest_matrices_exact(dev, N, K, counts, dtype):
    """The largest width: the longest sums (of -1, 0 and 1, exact in fp32), the farthest offsets within a tile."""
    make = lambda shape, seed, dev: torch.randint(-1, 2, shape, device=dev, dtype=torch.int8,  # noqa: E731
                                                  generator=torch.Generator(device=dev).manual_seed(seed)).float()
    run_all(counts, 1, N, K, dtype, F32, dev, seed=19, make=make)


def test_large_tiles_of_normal_values(dev):
    run_all([1500, 0, 17, 2579], 3, 2056, 520, BF, BF, dev, seed=13, make=normal, exact=False)
    run_all([1300, 900, 0, 1900], 0, 520, 2056, BF, F32, dev, seed=14, make=normal, exact=False)


@pytest.mark.parametrize("counts,N,K", [([1500, 0, 17, 2579], 2056, 520), ([1300, 900, 0, 1900], 520, 2056),
                                        ([150] * 20 + [0, 3, 290], 264, 328), ([3, 1, 0, 14] * 30, 1544, 264)])
def test_products_captured_and_replayed(dev, counts, N, K):
    """Each product in a graph: replays with other inputs, rows dealt anew on the device (the graph holds no
    counts), other eager work in between; every replay against the eager call."""
    n = sum(counts)
    t = inputs(counts, 0, N, K, BF, dev, seed=15, make=normal)
    for w in ("w", "w2"):
        t[w].nan_to_num_(0.5)
    E = len(counts)
    out = dict(y=torch.empty((n, N), device=dev), dx=torch.empty((n, K), dtype=BF, device=dev),
               dw=torch.empty((E, N, K), dtype=BF, device=dev))

    def run(o, stream=None):
        moe.moe_grouped_gemm(t["x"], t["offsets"], t["w"], o["y"])
        moe.moe_grouped_gemm_dgrad(t["dy"], t["offsets"], t["w"], o["dx"], dy2=t["dy2"], w2=t["w2"])
        moe.moe_grouped_gemm_wgrad(t["dy"], t["x"], t["offsets"], o["dw"])
    run(out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(out)
    order = list(counts)
    for rep in range(4):
        order = order[1:] + order[:1]
        t["offsets"].copy_(ref.offsets_of(order, dev))
        t["x"].copy_(normal((n, K), 200 + rep, dev))
        for o in out.values():
            o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        eager = {k: torch.full_like(v, float("nan")) for k, v in out.items()}
        run(eager)
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(out[k], eager[k]), (rep, k)


def test_offsets_that_are_wrong_stay_in_bounds(dev):
    """Offsets that no permutation writes (falling, negative, past the rows) give unspecified results, but
    nothing is read or written outside the buffers."""
    N, K, rows = 136, 264, 300
    t = inputs([100, 100, 100], 0, N, K, BF, dev, seed=16)
    for bad in ([0, 250, 100, 300], [-5, 900, 20, 7], [2 ** 31 - 1] * 4, [300, 200, 100, 0]):
        off = torch.tensor(bad, dtype=torch.int32, device=dev)
        for shape, call in (((rows, N), lambda o: moe.moe_grouped_gemm(t["x"], off, t["w"], o)),
                            ((rows, K), lambda o: moe.moe_grouped_gemm_dgrad(t["dy"], off, t["w"], o)),
                            ((3, N, K), lambda o: moe.moe_grouped_gemm_wgrad(t["dy"], t["x"], off, o))):
            o, whole = ref.guarded(shape, F32, dev)
            call(o)
            torch.cuda.synchronize()
            assert ref.guards_intact(whole, o.numel())
