"""64-bit references of the training step's operators, and the buffers that its tests use.

Tolerances. u(t) = finfo(t).eps / 2 is the most that one rounding to nearest in format t moves a
value, relative to it. A sum of n products in fp32 is off by at most n * 2^-23 * sum |a||b| (each of
the n additions is off by less than one unit, 2^-23, of a partial sum of at most sum |a||b|, also
where an addition truncates); an output in format t adds u(t) of the value."""
import torch

POISON = float("nan")


def u(dtype):
    return torch.finfo(dtype).eps / 2


def guarded(shape, dtype, dev, fill=POISON, pad=128):
    """An uninitialised-looking tensor inside a larger buffer: everything is `fill`; returns (view, whole)."""
    n = 1
    for s in shape:
        n *= s
    if dtype in (torch.float8_e4m3fn,):
        whole = torch.full((n + 2 * pad,), 0xAB, dtype=torch.uint8, device=dev)
        return whole[pad:pad + n].view(torch.float8_e4m3fn).view(shape), whole
    whole = torch.full((n + 2 * pad,), fill, dtype=dtype, device=dev)
    return whole[pad:pad + n].view(shape), whole


def put(values, dtype, dev):
    """values in a guarded buffer of NaN."""
    t, _ = guarded(tuple(values.shape), dtype, dev)
    t.copy_(values)
    return t


def guards_intact(whole, n, fill=POISON, pad=128):
    ends = torch.cat([whole[:pad], whole[pad + n:]])
    if ends.dtype == torch.uint8:
        return bool((ends == 0xAB).all())
    return bool(torch.isnan(ends).all()) if fill != fill else bool((ends == fill).all())


def offsets_of(counts, dev):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.cumsum(torch.tensor(counts, dtype=torch.int64), 0)
    return o.to(dev)


def spans(counts):
    a = 0
    for e, n in enumerate(counts):
        yield e, a, a + n
        a += n


def forward(x, w, counts):
    y = torch.zeros((sum(counts), w.shape[1]), dtype=torch.float64, device=x.device)
    for e, a, b in spans(counts):
        if b > a:
            y[a:b] = x[a:b].double() @ w[e].double().t()
    return y


def dgrad(dy, w, counts):
    dx = torch.zeros((sum(counts), w.shape[2]), dtype=torch.float64, device=dy.device)
    for e, a, b in spans(counts):
        if b > a:
            dx[a:b] = dy[a:b].double() @ w[e].double()
    return dx


def wgrad(dy, x, counts):
    dw = torch.zeros((len(counts), dy.shape[1], x.shape[1]), dtype=torch.float64, device=dy.device)
    for e, a, b in spans(counts):
        if b > a:
            dw[e] = dy[a:b].double().t() @ x[a:b].double()
    return dw


# ---- rows held in 8 bits --------------------------------------------------------------------
def code_values():
    """The value of each of the 256 e4m3fn codes (sign, 4 exponent bits with bias 7, 3 mantissa bits)."""
    out = torch.empty(256, dtype=torch.float64)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = float("nan") if (c & 127) == 127 else (-v if c & 128 else v)
    return out


def held_scale(group):
    """The documented scale of one group (a list of Python floats), by trying powers of two upwards."""
    top = max((abs(v) for v in group if abs(v) < float("inf")), default=0.0)  # NaN compares false
    if top == 0.0:
        return 1.0
    e = -117
    while 448.0 * 2.0 ** e < top and e < 120:
        e += 1
    return 2.0 ** e


def held(x):
    """What rows held in 8 bits stand for, in 64 bits on the host: (values, scales)."""
    table = code_values()[:127]
    x = x.detach().double().cpu()
    d = x.shape[1]
    vals, scales = torch.empty_like(x), torch.empty((x.shape[0], -(-d // 128)), dtype=torch.float64)
    for g in range(-(-d // 128)):
        part = x[:, g * 128:(g + 1) * 128]
        s = torch.tensor([held_scale(r) for r in part.tolist()], dtype=torch.float64).reshape(-1, 1)
        scales[:, g] = s[:, 0]
        v = part.abs() / s
        fine = torch.isfinite(v)
        v = torch.where(fine, v, torch.zeros_like(v))
        hi = torch.searchsorted(table, v.contiguous()).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        up = (table[hi] - v < v - table[lo]) | ((table[hi] - v == v - table[lo]) & (hi % 2 == 0))
        code = torch.where(up, hi, lo)
        code = torch.where((s == 2.0 ** 120) & (code > 119), torch.full_like(code, 119), code)  # 240
        q = torch.sign(part) * table[code] * s
        vals[:, g * 128:(g + 1) * 128] = torch.where(fine, q, torch.full_like(q, float("nan")))
    return vals, scales


def swiglu(g, u_):
    return g * torch.sigmoid(g) * u_


def swiglu_backward(dh, g, u_):
    """(dg, du, h) in 64 bits."""
    s, r = torch.sigmoid(g), torch.sigmoid(-g)
    return dh * u_ * (s + g * s * r), dh * g * s, g * s * u_
