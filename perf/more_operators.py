"""Microscaled 4-bit operators of the MoE layer (MXFP4), as cases to measure.

A row of d elements is d e2m1 codes, two to a byte (the first in the low half), and one e8m0 scale byte b per 32 elements;
an element's value is code * 2^(b - 127). The scales of rows lie in blocks of 256 elements, [ceil(d/256), rows, 8].
Expert e owns rows [offsets[e], offsets[e+1]).

  quantize  rows to MXFP4, each token's row once into its k expert-sorted rows, and back as values
  gemm      y[r] = W_e x[r] with W in MXFP4, x in bf16 or MXFP4
  dgrad     dx[r] = W_e^T dy[r] + W2_e^T dy2[r] with W and W2 in MXFP4
  swiglu    h[r] = silu(Wg_e x[r]) * (Wu_e x[r]) with Wg and Wu in MXFP4, x in bf16 or MXFP4

With `own` false `run` is their plain form in torch; with `own` true it calls the library.
"""
import math

import torch

own = False

GROUP = 32    # elements that share a scale
BLOCK = 256   # elements whose 8 scales lie together
MAX_EXP = 125  # scales lie in 2^-125 .. 2^125

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------
def listed():
    return [
        # the layer input of a small batch: fp32, a last block of scales that is not full
        dict(name="quantize_small", op="quantize", T=130, k=8, E=128, d=5152, zipf=1.0, x="f32", out="f32"),
        # a training or prefill batch's layer input, straight into its sorted rows
        dict(name="quantize_train", op="quantize", T=8192, k=8, E=32, d=7168, zipf=1.2, x="bf16", out="bf16"),
        # one decode token through 8 of 128 experts: latency
        dict(name="gemm_one_token", op="gemm", T=1, k=8, E=128, N=1536, K=4096, zipf=0.0, x="bf16", out="bf16"),
        # a decode batch: the stream of the 4-bit weights
        dict(name="gemm_decode", op="gemm", T=128, k=8, E=128, N=1536, K=4096, zipf=1.2, x="bf16", out="f32"),
        # a prefill batch on one of eight GPUs, rows in bf16
        dict(name="gemm_prefill", op="gemm", T=8192, k=8, E=32, N=2048, K=7168, zipf=1.2, x="bf16", out="bf16"),
        # the down product of a decode batch whose activations are held in 4 bits
        dict(name="gemm_decode_4bit", op="gemm", T=128, k=8, E=128, N=4096, K=1536, zipf=1.2, x="mxfp4", out="f32"),
        # the prefill batch with 4-bit rows: the scaled matrix instructions
        dict(name="gemm_prefill_4bit", op="gemm", T=8192, k=8, E=32, N=2048, K=7168, zipf=1.2, x="mxfp4", out="bf16"),
        # the input gradient of a small layer with frozen 4-bit weights, sizes that fill no tile
        dict(name="dgrad_small", op="dgrad", T=26, k=4, E=8, N=1544, K=800, zipf=0.6, out="f32"),
        # a training batch's input gradient through gate and up
        dict(name="dgrad_train", op="dgrad", T=8192, k=8, E=32, N=2048, K=7168, zipf=1.2, out="bf16"),
        # gate, up and activation of one decode token
        dict(name="swiglu_one_token", op="swiglu", T=1, k=8, E=128, f=1536, d=4096, zipf=0.0, x="bf16"),
        # of a decode batch
        dict(name="swiglu_decode", op="swiglu", T=128, k=8, E=128, f=1536, d=4096, zipf=1.2, x="bf16"),
        # of a prefill batch with 4-bit rows
        dict(name="swiglu_prefill_4bit", op="swiglu", T=8192, k=8, E=32, f=2048, d=7168, zipf=1.2, x="mxfp4"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "gemm", "dgrad", "dgrad", "swiglu", "swiglu"])
    E = _log_int(rng, 1, 128)
    case = dict(op=op, T=_log_int(rng, 1, 8192), k=rng.randint(1, min(8, E)), E=E, zipf=rng.choice([0.0, 0.6, 1.2]))
    if op == "quantize":
        case["x"] = rng.choice(["bf16", "bf16", "f32"])
        case["out"] = rng.choice(["bf16", "f32"])
        case["d"] = _log_int(rng, 64, 7168, 32)
        if case["out"] == "f32":  # bound by memory: no more bytes than the listed 16-bit case
            case["T"] = min(case["T"], 4096)
        return case
    rows, cols = ("f", "d") if op == "swiglu" else ("N", "K")
    case[rows] = _log_int(rng, 64, 2048 if op == "swiglu" else 4096, 32 if op == "swiglu" else 8)
    case[cols] = _log_int(rng, 64, 7168, 32)
    if op != "dgrad":
        case["x"] = rng.choice(["bf16", "mxfp4"])
    if op != "swiglu":
        case["out"] = rng.choice(["bf16", "f32"])
    # no more arithmetic and no larger weights than the largest listed cases
    pairs = 1 if op == "gemm" else 2
    while case["T"] * case["k"] * case[rows] * case[cols] * pairs > 2 ** 40:
        case["T"] = max(1, case["T"] // 2)
    while case["E"] * case[rows] * case[cols] > 32 * 2048 * 7168:
        if case["E"] > case["k"]:
            case["E"] = max(case["k"], case["E"] // 2)
        else:
            case[rows] = max(64, case[rows] // 64 * 32)
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
# the format
# ----------------------------------------------------------------------------------------
def _power(n):
    """2^n for whole n in -126 .. 127, exactly."""
    return ((n.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes(x):
    """fp32 rows [rows, d] as codes [rows, d] (0 .. 15) and exponents [rows, d/32]: the smallest power of two with which
    the group's largest magnitude is at most 6, codes rounded to the nearest, ties to the even code."""
    g = x.reshape(x.shape[0], -1, GROUP)
    mant, exp = torch.frexp(g.abs().amax(2))                    # amax = mant * 2^exp, mant in [0.5, 1)
    e = (exp - 3 + (mant > 0.75).int()).clamp(-MAX_EXP, MAX_EXP)  # 6 = 0.75 * 2^3
    e = torch.where(mant == 0, torch.zeros_like(e), e)
    q = g * _power(-e)[:, :, None]
    a = q.abs()
    c = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
         + (a >= 3.5).byte() + (a > 5).byte() + torch.signbit(q).byte() * 8)
    return c.reshape(x.shape), e


def _pack(c, e):
    """Codes and exponents as they are held: codes [rows, d/2] and scales [ceil(d/256), rows, 8] bytes."""
    rows, groups = e.shape
    b = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -groups % 8))
    return c[:, 0::2] | (c[:, 1::2] << 4), b.reshape(rows, -1, 8).transpose(0, 1).contiguous()


def _table(device):
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)
    return torch.cat([v, -v])


def _values(codes, scales):
    """The fp32 values [rows, d] that codes [rows, d/2] and scales [ceil(d/256), rows, 8] stand for."""
    rows, half = codes.shape
    t = _table(codes.device)
    byte = torch.arange(256, device=codes.device)
    pairs = torch.stack([t[byte & 15], t[byte >> 4]], 1)  # the two elements of each byte
    v = pairs[codes.int()].reshape(rows, -1, GROUP)
    s = _power(scales.transpose(0, 1).reshape(rows, -1)[:, : v.shape[1]].int() - 127)
    return (v * s[:, :, None]).reshape(rows, 2 * half)


# ----------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype, scale=1.0):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.normal_(0.0, scale, generator=g)
    return t


def _weights(g, E, N, K):
    """Weights as a program holds them: quantised once, when they are loaded."""
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, -(-K // BLOCK), N, 8), dtype=torch.uint8, device="cuda")
    for e in range(E):
        codes[e], scales[e] = _pack(*_codes(_normal(g, (N, K), torch.float32, K ** -0.5)))
    return codes, scales


def _hidden(g, rows, d, dtype):
    """Hidden states after a norm: unit size with a few large channels."""
    x = _normal(g, (rows, d), dtype)
    x[:, torch.randperm(d, generator=g, device="cuda")[: max(1, d // 256)]] *= 30.0
    return x


def _grouping(case, g):
    """offsets [E+1] on the device and on the host: the counts dealt to the experts in a seeded order."""
    counts = torch.tensor(_counts(case), device="cuda")[torch.randperm(case["E"], generator=g, device="cuda")]
    offsets = torch.zeros(case["E"] + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets, offsets.tolist()


def _routing(case, g):
    """A router's choice for T tokens, as the sorted row of each assignment and the assignment of each row."""
    T, k, E = case["T"], case["k"], case["E"]
    bias = -case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    logits = _normal(g, (T, E), torch.float32) + bias[torch.randperm(E, generator=g, device="cuda")]
    order = torch.argsort(torch.topk(logits, k, dim=1).indices.reshape(-1), stable=True)
    back = torch.empty_like(order)
    back[order] = torch.arange(T * k, device="cuda")
    return dict(s2f=order.to(torch.int32), f2s=back.to(torch.int32))


def prepare(case, seed):
    g = _generator(seed)
    T, k, E, op = case["T"], case["k"], case["E"], case["op"]
    R = T * k
    st = dict(case=case)
    empty = lambda shape, t: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
    if op == "quantize":
        d = case["d"]
        st.update(_routing(case, g))
        st.update(x=_hidden(g, T, d, DTYPES[case["x"]]), codes=empty((R, d // 2), torch.uint8),
                  scales=empty((-(-d // BLOCK), R, 8), torch.uint8), values=empty((R, d), DTYPES[case["out"]]))
        return st
    st["offsets"], st["bounds"] = _grouping(case, g)
    N, K = (case["f"], case["d"]) if op == "swiglu" else (case["N"], case["K"])
    st["w"], st["ws"] = _weights(g, E, N, K)
    if op != "gemm":
        st["w2"], st["w2s"] = _weights(g, E, N, K)
    if op == "dgrad":  # gradients of a mean loss are small
        st.update(dy=_normal(g, (R, N), torch.bfloat16, 1e-3), dy2=_normal(g, (R, N), torch.bfloat16, 1e-3),
                  dx=empty((R, K), DTYPES[case["out"]]))
        return st
    if case["x"] == "mxfp4":
        st["x"], st["xs"] = _pack(*_codes(_hidden(g, R, K, torch.float32)))
    else:
        st["x"], st["xs"] = _hidden(g, R, K, torch.bfloat16), None
    st["y"] = empty((R, N), torch.bfloat16 if op == "swiglu" else DTYPES[case["out"]])
    return st


# ----------------------------------------------------------------------------------------
# the operators
# ----------------------------------------------------------------------------------------
def _experts(bounds):
    """The experts that have rows: (expert, first row, end)."""
    return [(e, a, b) for e, (a, b) in enumerate(zip(bounds, bounds[1:])) if b > a]


def _quantize(st):
    case = st["case"]
    if own:
        import token_dispatch_expert_amd as moe
        moe.moe_mxfp4_quantize(st["x"], st["codes"], st["scales"], flat_to_sorted=st["f2s"])
        moe.moe_mxfp4_dequantize(st["codes"], st["scales"], st["values"])
        return st["values"]
    c, e = _codes(st["x"].float())
    v = _table(c.device)[c.int()].reshape(*e.shape, GROUP) * _power(e)[:, :, None]
    return v.reshape(c.shape).to(DTYPES[case["out"]])[(st["s2f"] // case["k"]).long()]


def _rows(st):
    return st["x"].float() if st["xs"] is None else _values(st["x"], st["xs"])


def _gemm(st):
    if own:
        import token_dispatch_expert_amd as moe
        moe.moe_grouped_gemm_mxfp4(st["x"], st["offsets"], st["w"], st["ws"], st["y"], x_scales=st["xs"])
        return st["y"]
    x, y = _rows(st), torch.empty_like(st["y"])
    for e, a, b in _experts(st["bounds"]):
        y[a:b] = x[a:b] @ _values(st["w"][e], st["ws"][e]).t()
    return y


def _dgrad(st):
    if own:
        import token_dispatch_expert_amd as moe
        moe.moe_grouped_gemm_mxfp4_dgrad(st["dy"], st["offsets"], st["w"], st["ws"], st["dx"], dy2=st["dy2"],
                                         w2=st["w2"], w2_scales=st["w2s"])
        return st["dx"]
    dx = torch.empty_like(st["dx"])
    for e, a, b in _experts(st["bounds"]):
        dx[a:b] = (st["dy"][a:b].float() @ _values(st["w"][e], st["ws"][e])
                   + st["dy2"][a:b].float() @ _values(st["w2"][e], st["w2s"][e]))
    return dx


def _swiglu(st):
    if own:
        import token_dispatch_expert_amd as moe
        moe.moe_grouped_swiglu_mxfp4(st["x"], st["offsets"], st["w"], st["ws"], st["w2"], st["w2s"], st["y"],
                                     x_scales=st["xs"])
        return st["y"]
    x, h = _rows(st), torch.empty_like(st["y"])
    for e, a, b in _experts(st["bounds"]):
        g = x[a:b] @ _values(st["w"][e], st["ws"][e]).t()
        u = x[a:b] @ _values(st["w2"][e], st["w2s"][e]).t()
        h[a:b] = g / (1 + torch.exp(-g)) * u
    return h


_RUN = dict(quantize=_quantize, gemm=_gemm, dgrad=_dgrad, swiglu=_swiglu)


def run(state):
    return _RUN[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------
def work(case):
    T, k, op = case["T"], case["k"], case["op"]
    R = T * k
    size = dict(bf16=2, f32=4, mxfp4=17 / 32)  # a byte for 32 scaled codes of half a byte
    if op == "quantize":
        d = case["d"]
        held = R * d * size["mxfp4"]
        return dict(bytes=T * d * size[case["x"]] + 2 * held + R * d * size[case["out"]] + 4 * R,
                    flops=4 * T * d + R * d)
    active = sum(c > 0 for c in _counts(case))
    N, K = (case["f"], case["d"]) if op == "swiglu" else (case["N"], case["K"])
    w = active * N * K * size["mxfp4"]
    if op == "gemm":
        return dict(bytes=R * K * size[case["x"]] + w + R * N * size[case["out"]], flops=2 * R * N * K)
    if op == "dgrad":
        return dict(bytes=2 * (R * N * 2 + w) + R * K * size[case["out"]], flops=4 * R * N * K)
    return dict(bytes=R * K * size[case["x"]] + 2 * w + R * N * 2, flops=4 * R * N * K)


# ----------------------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------------------
def _power64(n):
    """2^n as a 64-bit float, from its bits."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _magnitude64(c):
    """What the three low bits of a code stand for: two of exponent (bias 1), one of mantissa."""
    e, m = (c >> 1) & 3, (c & 1).double()
    return torch.where(e == 0, m / 2, (1 + m / 2) * _power64(e - 1))


def _values64(codes, scales):
    rows, half = codes.shape
    out = torch.empty((rows, 2 * half), dtype=torch.float64, device=codes.device)
    for h in range(2):
        c = (codes.int() >> (4 * h)) & 15
        out[:, h::2] = torch.where(c >= 8, -_magnitude64(c), _magnitude64(c))
    for j in range(2 * half // GROUP):  # the group's scale: block j / 8, place j % 8
        out[:, GROUP * j:GROUP * (j + 1)] *= _power64(scales[j // 8, :, j % 8].int() - 127)[:, None]
    return out


def _held64(x):
    """The values of rows in 4 bits, by search among the codes' values; a tie goes to the even code."""
    table = _magnitude64(torch.arange(8, device=x.device))
    g = x.reshape(x.shape[0], -1, GROUP)
    top = g.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 6.0)) / 6.0)).long()
    e = e - ((top <= 6.0 * _power64(e - 1)) & (top > 0)).long()  # log2 may land on either side
    e = (e + (top > 6.0 * _power64(e)).long()).clamp(-MAX_EXP, MAX_EXP)
    v = (g.abs() / _power64(e)).clamp(max=6.0)
    hi = torch.searchsorted(table, v.contiguous()).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    below, above = v - table[lo], table[hi] - v
    pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return (torch.sign(g) * table[pick] * _power64(e)).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    op, k = case["op"], case["k"]
    if op == "quantize":
        return _held64(st["x"].double())[torch.div(st["s2f"], k, rounding_mode="floor").long()]
    offsets = st["offsets"].long()
    owner = torch.bucketize(torch.arange(case["T"] * k, device="cuda"), offsets[1:], right=True)
    res = torch.zeros(st["dx" if op == "dgrad" else "y"].shape, dtype=torch.float64, device="cuda")
    if op != "dgrad":
        x = st["x"].double() if st["xs"] is None else _values64(st["x"], st["xs"])
    for e in torch.unique(owner).tolist():
        mine = torch.nonzero(owner == e).reshape(-1)
        w = _values64(st["w"][e], st["ws"][e])
        if op == "gemm":
            res[mine] = torch.mm(w, x[mine].t()).t()
            continue
        w2 = _values64(st["w2"][e], st["w2s"][e])
        if op == "dgrad":
            both = torch.cat([st["dy"][mine], st["dy2"][mine]], 1).double()
            res[mine] = torch.mm(both, torch.cat([w, w2], 0))
        else:
            gu = torch.mm(torch.cat([w, w2], 0), x[mine].t()).t()
            gate = gu[:, : w.shape[0]]
            res[mine] = gate * torch.sigmoid(gate) * gu[:, w.shape[0]:]
    return res
