"""64-bit reference of the MXFP4 format, written from its definition: elements e2m1 (two exponent bits of bias 1, one
mantissa bit), one scale byte b per 32 elements for 2^(b - 127), 255 for NaN; scales in blocks of 256 elements.
Everything runs on the tensors' own device."""
import torch

CODES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def power(n):
    """2^n as a 64-bit float (whole n within the normal numbers)."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def blocked(scales):
    """Scale bytes [.., rows, groups] as the library holds them: [.., ceil(groups/8), rows, 8], 127 past the last."""
    g = scales.shape[-1]
    s = torch.nn.functional.pad(scales, (0, -g % 8), value=127)
    s = s.reshape(*s.shape[:-1], -1, 8)
    return s.transpose(-3, -2).contiguous()


def rows_of(scales, groups):
    """[.., blocks, rows, 8] as [.., rows, groups]."""
    s = scales.view(torch.uint8).transpose(-3, -2)
    return s.reshape(*s.shape[:-2], -1)[..., :groups]


def values(codes, scales):
    """The values [.., rows, d] of codes [.., rows, d/2] and scales [.., ceil(d/256), rows, 8]."""
    c = codes.view(torch.uint8).long()
    c = torch.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)
    v = CODES.to(c.device)[c & 7]
    v = torch.where(c >= 8, -v, v)
    s = rows_of(scales, c.shape[-1] // 32).long()
    f = torch.where(s == 255, torch.full(s.shape, float("nan"), dtype=torch.float64, device=s.device), power(s - 127))
    return (v.reshape(*s.shape, 32) * f[..., None]).reshape(c.shape)


def scale_of(x):
    """The scale bytes [.., rows, groups] of values x [.., rows, d], by trying every power of two."""
    g = x.double().reshape(*x.shape[:-1], -1, 32)
    top = g.abs().amax(-1)
    steps = 6.0 * power(torch.arange(-125, 126, device=x.device))  # the largest value of each scale, ascending
    b = torch.searchsorted(steps, top.contiguous()).clamp(max=250) + 2
    b = torch.where(top == 0, torch.full_like(b, 127), b)
    return torch.where(torch.isfinite(g).all(-1), b, torch.full_like(b, 255)).to(torch.uint8)


def codes_of(x, scales):
    """The codes [.., rows, d/2] of x under scale bytes [.., rows, groups]: the nearest, of two the even code."""
    g = x.double().reshape(*x.shape[:-1], -1, 32)
    bad = (scales == 255)[..., None]
    v = torch.where(bad, torch.zeros_like(g), g / power(scales.long() - 127)[..., None])
    table = CODES.to(x.device)
    a = v.abs().clamp(max=6.0)
    hi = torch.searchsorted(table, a.contiguous()).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    below, above = a - table[lo], table[hi] - a
    c = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    c = (c + 8 * (torch.signbit(v) & ~bad)).reshape(x.shape).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def quantize(x):
    """codes and (blocked) scales of x [.., rows, d]."""
    s = scale_of(x)
    return codes_of(x, s), blocked(s)
