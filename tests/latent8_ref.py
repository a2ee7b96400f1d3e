"""Plain fp64 evaluations of the 8-bit latent cache, for the tests."""
import math

import torch


def _value(code):
    sign, e, m = code >> 7, code >> 3 & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    v = math.ldexp(8 + m, e - 10) if e else math.ldexp(m, -9)
    return -v if sign else v


VALUES = torch.tensor([_value(c) for c in range(256)], dtype=torch.float64)


def values(codes, scales, rope):
    """[pages, page, L+R] in fp64 of a cache's tensors (codes as uint8)"""
    x = VALUES[codes.cpu().view(torch.uint8).long()] * scales.cpu().double()[..., None]
    return x if rope is None else torch.cat([x, rope.cpu().double()], -1)


def quantize(x):
    """(codes, scales) of finite rows x [T, L] in fp64: the scale from exact comparisons, each code the nearest value,
    the even one of two that are as near."""
    top = x.abs().amax(-1)
    scales = torch.empty_like(top)
    for t, a in enumerate(top.tolist()):
        e = -126
        if a > 0:
            e = max(e, math.frexp(a)[1] - 10)
            while a > math.ldexp(448, e):
                e += 1
        scales[t] = math.ldexp(1.0, e)
    y = x / scales[:, None]
    grid = VALUES[:127]                                    # 0 .. 448, ascending: code = index
    a = y.abs()
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code + torch.where(torch.signbit(y), 128, 0)).to(torch.uint8), scales
