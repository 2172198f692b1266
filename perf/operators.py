"""The operators of the MoE layer's training step, as cases to measure.

Five operators over expert-sorted rows (expert e owns rows [offsets[e], offsets[e+1])):

  gemm        y[r] = W_e x[r] (forward), dx[r] = W_e^T dy[r] + W2_e^T dy2[r] (input gradient)
  wgrad       dW_e = sum over the expert's rows of dy[r] x[r]^T
  checkpoint  rows held in 8 bits (e4m3fn codes, a power-of-two scale per 128 elements of a row) from the
              forward to the backward pass, where they come back gathered into expert order
  swiglu      h = silu(g) * u with g and u kept in 8 bits, then dg, du and h again from those
  tokens      the backward passes of combine, permute and route, which take a layer's gradient from the
              tokens to the sorted rows and back, and to the router's logits

With `own` false `run` is their plain form in torch; with `own` true it calls the library.
"""
import math

import torch

own = False

GROUP = 128          # elements of a row that share a scale
MIN_SCALE_EXP = -117  # smallest scale: every value of a code is then a normal bf16 number
MAX_SCALE_EXP = 120

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------
def listed():
    return [
        # one decode token through 8 of 128 experts: latency and the stream of eight weight matrices
        dict(name="gemm_forward_one_token", op="gemm", dir="forward", T=1, k=8, E=128, N=1536, K=4096,
             zipf=0.0, dtype="bf16", out="bf16"),
        # a decode batch of 128 tokens: few rows per expert, bound by the weights
        dict(name="gemm_forward_decode", op="gemm", dir="forward", T=128, k=8, E=128, N=1536, K=4096,
             zipf=1.2, dtype="bf16", out="f32"),
        # a training batch on one of eight GPUs (32 of 256 experts): the gate or up product
        dict(name="gemm_forward_train", op="gemm", dir="forward", T=8192, k=8, E=32, N=2048, K=7168,
             zipf=1.2, dtype="bf16", out="bf16"),
        # the same batch's input gradient through gate and up, summed in one pass
        dict(name="gemm_dgrad_train", op="gemm", dir="dgrad", T=8192, k=8, E=32, N=2048, K=7168,
             zipf=1.2, dtype="bf16", out="bf16"),
        # weight gradient of the smallest fp32 layer: latency
        dict(name="wgrad_small_f32", op="wgrad", T=64, k=2, E=8, N=256, K=128, zipf=0.0, dtype="f32", out="f32"),
        # weight gradient of the training batch, fp32 for the optimiser
        dict(name="wgrad_train", op="wgrad", T=8192, k=8, E=32, N=2048, K=7168, zipf=1.2, dtype="bf16", out="f32"),
        # a decode-sized batch's layer input, held and brought back (rows of 40 groups and a part of one)
        dict(name="checkpoint_small", op="checkpoint", T=130, k=8, E=128, d=5160, zipf=1.0, dtype="f32", out="f32"),
        # a training batch's layer input: packed once per token, unpacked for its 8 sorted rows
        dict(name="checkpoint_train", op="checkpoint", T=8192, k=8, E=32, d=7168, zipf=1.2, dtype="bf16", out="bf16"),
        # activations of a decode-sized batch, width no multiple of a group
        dict(name="swiglu_small", op="swiglu", T=125, k=8, E=128, f=1544, zipf=1.2, dtype="f32", out="f32"),
        # activations of the training batch
        dict(name="swiglu_train", op="swiglu", T=8192, k=8, E=32, f=2048, zipf=1.2, dtype="bf16", out="bf16"),
        # the smallest fp32 layer's tokens: three launches
        dict(name="tokens_small", op="tokens", T=64, k=2, E=8, d=128, zipf=0.0, dtype="f32", out="f32"),
        # the training batch's tokens, over all 256 experts
        dict(name="tokens_train", op="tokens", T=8192, k=8, E=256, d=7168, zipf=1.2, dtype="bf16", out="bf16"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "wgrad", "wgrad", "checkpoint", "swiglu", "tokens"])
    E = _log_int(rng, 1, 128)
    k = rng.randint(1, min(8, E))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    out = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
    case = dict(op=op, T=_log_int(rng, 1, 8192), k=k, E=E, zipf=rng.choice([0.0, 0.6, 1.2]), dtype=dtype, out=out)
    if op in ("gemm", "wgrad"):
        case["N"], case["K"] = _log_int(rng, 64, 4096, 8), _log_int(rng, 64, 7168, 8)
        if op == "gemm":
            case["dir"] = rng.choice(["forward", "dgrad"])
        # no more arithmetic and no larger weights than the largest listed cases
        while case["T"] * k * case["N"] * case["K"] * (4 if dtype == "f32" else 1) > 2 ** 39:
            case["T"] = max(1, case["T"] // 2)
        while case["E"] * case["N"] * case["K"] > 32 * 2048 * 7168:
            case["E"] = max(case["k"], case["E"] // 2)
            if case["E"] == case["k"]:
                case["N"] = max(64, case["N"] // 16 * 8)
        return case
    if out == "f32":  # bound by memory: no more bytes than the listed 16-bit cases
        case["T"] = min(case["T"], 4096)
    case["f" if op == "swiglu" else "d"] = _log_int(rng, 64, 2048 if op == "swiglu" else 7168, 8)
    return case


def _counts(case):
    """Rows per expert in order of popularity: shares rank^-zipf of T*k, at most T each."""
    T, k, E = case["T"], case["k"], case["E"]
    share = [(r + 1.0) ** -case["zipf"] for r in range(E)]
    total, left = sum(share), T * k
    counts = [min(T, int(T * k * s / total)) for s in share]
    left -= sum(counts)
    while left > 0:
        for e in range(E):
            add = min(left, max(0, min(T - counts[e], max(1, left // E))))
            counts[e] += add
            left -= add
    return counts


# ----------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype, scale=1.0):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.normal_(0.0, scale, generator=g)
    return t


def _grouping(case, g):
    """offsets [E+1] on the device and on the host: the counts dealt to the experts in a seeded order."""
    counts = torch.tensor(_counts(case), device="cuda")[torch.randperm(case["E"], generator=g, device="cuda")]
    offsets = torch.zeros(case["E"] + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets, offsets.tolist()


def _routing(case, g):
    """A router's choice for T tokens: ids, gates, and the maps between tokens and sorted rows."""
    T, k, E = case["T"], case["k"], case["E"]
    bias = -case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    logits = _normal(g, (T, E), torch.float32) + bias[torch.randperm(E, generator=g, device="cuda")]
    top, ids = torch.topk(logits, k, dim=1)
    order = torch.argsort(ids.reshape(-1), stable=True)
    back = torch.empty_like(order)
    back[order] = torch.arange(T * k, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(ids.reshape(-1), minlength=E), 0)
    return dict(ids=ids.to(torch.int32), gates=torch.softmax(top, 1), offsets=offsets,
                s2f=order.to(torch.int32), f2s=back.to(torch.int32))


def prepare(case, seed):
    g = _generator(seed)
    dt, out = DTYPES[case["dtype"]], DTYPES[case["out"]]
    R = case["T"] * case["k"]
    st = dict(case=case)
    empty = lambda shape, t: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
    if case["op"] in ("gemm", "wgrad"):
        E, N, K = case["E"], case["N"], case["K"]
        st["offsets"], st["bounds"] = _grouping(case, g)
        if case["op"] == "wgrad":
            # gradients of a mean loss are small; the activations are normalised
            st.update(dy=_normal(g, (R, N), dt, 1e-3), x=_normal(g, (R, K), dt), dw=empty((E, N, K), out))
        elif case["dir"] == "forward":
            st.update(x=_normal(g, (R, K), dt), w=_normal(g, (E, N, K), dt, K ** -0.5), y=empty((R, N), out))
        else:
            st.update(dy=_normal(g, (R, N), dt, 1e-3), dy2=_normal(g, (R, N), dt, 1e-3),
                      w=_normal(g, (E, N, K), dt, K ** -0.5), w2=_normal(g, (E, N, K), dt, K ** -0.5),
                      dx=empty((R, K), out))
        return st
    if case["op"] == "swiglu":
        f = case["f"]
        st["offsets"], _ = _grouping(case, g)
        st.update(g=_normal(g, (R, f), dt), u=_normal(g, (R, f), dt), dh=_normal(g, (R, f), dt, 1e-3),
                  h=empty((R, f), dt), dg=empty((R, f), dt), du=empty((R, f), dt), h2=empty((R, f), dt))
        groups = -(-f // GROUP)
        for n in "gu":
            st[n + "_codes"] = empty((R, f), torch.float8_e4m3fn)
            st[n + "_scales"] = empty((R, groups), torch.float32)
        return st
    T, d = case["T"], case["d"]
    st.update(_routing(case, g))
    if case["op"] == "checkpoint":
        # hidden states after a norm: unit size with a few large channels
        x = _normal(g, (T, d), dt)
        x[:, torch.randperm(d, generator=g, device="cuda")[: max(1, d // 256)]] *= 30.0
        st.update(x=x, codes=empty((T, d), torch.float8_e4m3fn), scales=empty((T, -(-d // GROUP)), torch.float32),
                  x_sorted=empty((R, d), out))
    else:
        st.update(dy=_normal(g, (T, d), dt, 1e-3), y_sorted=_normal(g, (R, d), torch.float32),
                  dx_in=_normal(g, (R, d), dt, 1e-3), dy_sorted=empty((R, d), out), dx=empty((T, d), out),
                  dgates=empty((T, case["k"]), torch.float32), dlogits=empty((T, case["E"]), torch.float32))
    return st


# ----------------------------------------------------------------------------------------
# the operators
# ----------------------------------------------------------------------------------------
def _experts(bounds):
    """The experts that have rows: (expert, first row, end)."""
    return [(e, a, b) for e, (a, b) in enumerate(zip(bounds, bounds[1:])) if b > a]


def _gemm(st):
    case = st["case"]
    if own:
        import token_dispatch_expert_amd as moe
        if case["dir"] == "forward":
            moe.moe_grouped_gemm(st["x"], st["offsets"], st["w"], st["y"])
            return st["y"]
        moe.moe_grouped_gemm_dgrad(st["dy"], st["offsets"], st["w"], st["dx"], dy2=st["dy2"], w2=st["w2"])
        return st["dx"]
    rows, cols = case["T"] * case["k"], case["N"] if case["dir"] == "forward" else case["K"]
    out = torch.empty((rows, cols), dtype=DTYPES[case["out"]], device="cuda")
    for e, a, b in _experts(st["bounds"]):
        if case["dir"] == "forward":
            out[a:b] = st["x"][a:b].float() @ st["w"][e].float().t()
        else:
            out[a:b] = st["dy"][a:b].float() @ st["w"][e].float() + st["dy2"][a:b].float() @ st["w2"][e].float()
    return out


def _wgrad(st):
    case = st["case"]
    if own:
        import token_dispatch_expert_amd as moe
        moe.moe_grouped_gemm_wgrad(st["dy"], st["x"], st["offsets"], st["dw"])
        return st["dw"]
    dw = torch.zeros((case["E"], case["N"], case["K"]), dtype=DTYPES[case["out"]], device="cuda")
    for e, a, b in _experts(st["bounds"]):
        dw[e] = st["dy"][a:b].float().t() @ st["x"][a:b].float()
    return dw


def _held(x):
    """fp32 rows as their 8-bit codes stand for them: e4m3fn with a power-of-two scale per group."""
    d = x.shape[1]
    xp = torch.nn.functional.pad(x, (0, -d % GROUP)).reshape(x.shape[0], -1, GROUP)
    mant, exp = torch.frexp(xp.abs().amax(2, keepdim=True))       # amax = mant * 2^exp, mant in [0.5, 1)
    e = (exp - 9 + (mant > 0.875)).clamp(MIN_SCALE_EXP, MAX_SCALE_EXP)  # amax <= 448 * 2^e
    e = torch.where(mant == 0, torch.zeros_like(e), e)
    power = lambda n: ((n + 127) << 23).view(torch.float32)  # noqa: E731  (2^n, exactly)
    q = (xp * power(-e)).to(torch.float8_e4m3fn).float()
    return (q * power(e)).reshape(x.shape[0], -1)[:, :d]


def _checkpoint(st):
    case = st["case"]
    if own:
        import token_dispatch_expert_amd as moe
        moe.moe_checkpoint_pack(st["x"], st["codes"], st["scales"])
        moe.moe_checkpoint_unpack(st["codes"], st["scales"], st["x_sorted"], flat_to_sorted=st["f2s"])
        return st["x_sorted"]
    return _held(st["x"].float()).to(DTYPES[case["out"]])[(st["s2f"] // case["k"]).long()]


def _swiglu(st):
    if own:
        import token_dispatch_expert_amd as moe
        moe.moe_swiglu(st["g"], st["u"], st["h"], g_codes=st["g_codes"], g_scales=st["g_scales"],
                       u_codes=st["u_codes"], u_scales=st["u_scales"], offsets=st["offsets"])
        moe.moe_swiglu_backward(st["dh"], st["g_codes"], st["u_codes"], st["dg"], st["du"], h=st["h2"],
                                g_scales=st["g_scales"], u_scales=st["u_scales"], offsets=st["offsets"])
        return dict(h=st["h"], dg=st["dg"], du=st["du"], h2=st["h2"])
    dt = st["g"].dtype
    g, u, dh = st["g"].float(), st["u"].float(), st["dh"].float()
    h = g / (1 + torch.exp(-g)) * u
    g, u = _held(g), _held(u)
    s = 1 / (1 + torch.exp(-g))
    return dict(h=h.to(dt), dg=(dh * u * s * (1 + g * (1 - s))).to(dt), du=(dh * g * s).to(dt), h2=(g * s * u).to(dt))


def _tokens(st):
    case = st["case"]
    if own:
        import token_dispatch_expert_amd as moe
        moe.moe_combine_backward(st["dy"], st["y_sorted"], st["f2s"], st["gates"], st["dy_sorted"], st["dgates"])
        moe.moe_permute_backward(st["dx_in"], st["f2s"], case["k"], st["dx"])
        moe.moe_route_backward(st["dgates"], st["ids"], st["gates"], st["dlogits"])
        return dict(dy_sorted=st["dy_sorted"], dgates=st["dgates"], dx=st["dx"], dlogits=st["dlogits"])
    T, k, d = case["T"], case["k"], case["d"]
    out = DTYPES[case["out"]]
    dy, gates, f2s = st["dy"].float(), st["gates"], st["f2s"].long()
    dy_sorted = (gates[:, :, None] * dy[:, None, :]).reshape(T * k, d)[st["s2f"].long()].to(out)
    dgates = (dy[:, None, :] * st["y_sorted"][f2s].reshape(T, k, d)).sum(2)
    dx = st["dx_in"][f2s].float().reshape(T, k, d).sum(1).to(out)
    dl = gates * (dgates - (gates * dgates).sum(1, keepdim=True))
    dlogits = torch.zeros((T, case["E"]), device="cuda").scatter_(1, st["ids"].long(), dl)
    return dict(dy_sorted=dy_sorted, dgates=dgates, dx=dx, dlogits=dlogits)


_RUN = dict(gemm=_gemm, wgrad=_wgrad, checkpoint=_checkpoint, swiglu=_swiglu, tokens=_tokens)


def run(state):
    return _RUN[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------
def work(case):
    b, o = (2 if case[n] == "bf16" else 4 for n in ("dtype", "out"))
    T, k, E = case["T"], case["k"], case["E"]
    R = T * k
    if case["op"] in ("gemm", "wgrad"):
        N, K = case["N"], case["K"]
        active = sum(c > 0 for c in _counts(case))
        if case["op"] == "wgrad":
            return dict(bytes=R * (N + K) * b + E * N * K * o, flops=2 * R * N * K)
        if case["dir"] == "forward":
            return dict(bytes=(R * K + active * N * K) * b + R * N * o, flops=2 * R * N * K)
        return dict(bytes=2 * (R * N + active * N * K) * b + R * K * o, flops=4 * R * N * K)
    if case["op"] == "checkpoint":
        d = case["d"]
        held = T * (d + 4 * -(-d // GROUP))
        return dict(bytes=T * d * b + 2 * held + R * d * o, flops=4 * T * d + 2 * R * d)
    if case["op"] == "swiglu":
        f = case["f"]
        held = 2 * R * (f + 4 * -(-f // GROUP))
        return dict(bytes=2 * R * f * b + R * f * b + 2 * held + R * f * b + 3 * R * f * b, flops=40 * R * f)
    d = case["d"]
    return dict(bytes=T * d * b + 4 * R * d + R * d * o + R * d * b + T * d * o + 4 * T * E + 24 * R, flops=5 * R * d)


# ----------------------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------------------
def _code_values(device):
    """The finite magnitudes of e4m3fn, ascending: index = code (3 mantissa bits, bias 7)."""
    c = torch.arange(127, device=device)
    e, m = c // 8, (c % 8).double()
    return torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * _power64(e - 7))


def _power64(n):
    """2^n as a 64-bit float, from its bits: exp2 and pow may be off by one place."""
    return ((n + 1023) << 52).view(torch.float64)


def _held64(x):
    """The held values by search among the codes' values, ties to the even code."""
    table = _code_values(x.device)
    out = torch.empty_like(x)
    for c0 in range(0, x.shape[1], GROUP):
        part = x[:, c0:c0 + GROUP]
        top = part.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 448.0)) / 448.0)).long()
        e = e - ((top <= 448.0 * _power64(e - 1)) & (top > 0)).long()  # log2 may land on either side
        e = (e + (top > 448.0 * _power64(e)).long()).clamp(MIN_SCALE_EXP, MAX_SCALE_EXP)
        s = _power64(e)
        v = part.abs() / s
        hi = torch.searchsorted(table, v.contiguous()).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        below, above = v - table[lo], table[hi] - v
        pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
        out[:, c0:c0 + GROUP] = torch.sign(part) * table[pick] * s
    return out


def exact(case, seed):
    st = prepare(case, seed)
    T, k = case["T"], case["k"]
    R = T * k
    if case["op"] in ("gemm", "wgrad"):
        E, N, K = case["E"], case["N"], case["K"]
        if 2 * R * N * K > 3e12:
            return None
        owner = torch.bucketize(torch.arange(R, device="cuda"), st["offsets"][1:].long(), right=True)
        if case["op"] == "wgrad":
            res = torch.zeros((E, N, K), dtype=torch.float64, device="cuda")
        else:
            res = torch.zeros((R, N if case["dir"] == "forward" else K), dtype=torch.float64, device="cuda")
        for e in torch.unique(owner).tolist():
            mine = torch.nonzero(owner == e).reshape(-1)
            if case["op"] == "wgrad":
                res[e] = torch.mm(st["x"][mine].double().t(), st["dy"][mine].double()).t()
            elif case["dir"] == "forward":
                res[mine] = torch.mm(st["w"][e].double(), st["x"][mine].double().t()).t()
            else:
                both = torch.cat([st["dy"][mine], st["dy2"][mine]], 1).double()
                res[mine] = torch.mm(both, torch.cat([st["w"][e], st["w2"][e]], 0).double())
        return res
    if case["op"] == "checkpoint":
        return _held64(st["x"].double())[torch.div(st["s2f"], k, rounding_mode="floor").long()]
    if case["op"] == "swiglu":
        out = {n: torch.empty((R, case["f"]), dtype=torch.float64, device="cuda") for n in ("h", "dg", "du", "h2")}
        for r in range(0, R, 8192):
            part = slice(r, r + 8192)
            g, u, dh = (st[n][part].double() for n in ("g", "u", "dh"))
            out["h"][part] = g * torch.sigmoid(g) * u
            g, u = _held64(g), _held64(u)
            sig, rest = torch.sigmoid(g), torch.sigmoid(-g)
            out["dg"][part] = dh * u * (sig + g * sig * rest)
            out["du"][part] = dh * g * sig
            out["h2"][part] = g * sig * u
        return out
    d = case["d"]
    dy, gates = st["dy"].double(), st["gates"].double()
    dy_sorted = torch.empty((R, d), dtype=torch.float64, device="cuda")
    dgates = torch.empty((T, k), dtype=torch.float64, device="cuda")
    dx = torch.zeros((T, d), dtype=torch.float64, device="cuda")
    dlogits = torch.zeros((T, case["E"]), dtype=torch.float64, device="cuda")
    f2s = st["f2s"].reshape(T, k).long()
    for j in range(k):
        row = f2s[:, j]
        dy_sorted[row] = gates[:, j:j + 1] * dy
        dgates[:, j] = (dy * st["y_sorted"][row].double()).sum(1)
        dx += st["dx_in"][row].double()
    mean = (gates * dgates).sum(1)
    for j in range(k):
        dlogits[torch.arange(T, device="cuda"), st["ids"][:, j].long()] = gates[:, j] * (dgates[:, j] - mean)
    return dict(dy_sorted=dy_sorted, dgates=dgates, dx=dx, dlogits=dlogits)
