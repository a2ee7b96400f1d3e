"""Plain fp64 evaluations of the 8-bit latent cache, for the tests."""
import math

import torch

from tests import latent_ref as ref


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


def decode(cache, table, lengths, q, q_rope, scale):
    """As ref.decode, over rows in fp64; rows that no query sees may hold NaN."""
    return ref.decode(cache, table, lengths, q, q_rope, scale)


def score_error(cache, q, scale):
    """How far the 8-bit products' own sums can put a score off: they keep all but 2^-11 of the largest product
    of 128, for the leading half of the query and for the rest (at most 2^-4 of it)."""
    L = q.shape[-1]
    big = q.double().abs().max().item() * cache[..., :L].nan_to_num(0, 0, 0).abs().max().item()
    return scale * -(-L // 128) * (1 + 2.0 ** -4) * 2.0 ** -11 * big


def check(out, lse, want, delta, name=""):
    """As ref.check, with scores off by at most ``delta`` besides: each weight, and the sum that it is divided by, is off
    by that part of itself, so out by 2 delta sum p |v| and lse by delta.  The bounds of ref.check: out is rounded to
    bf16 (2^-8 of itself), the weights times scales were (2^-8 of sum p |v|), fp32 steps add under 2^-12; lse 1e-4."""
    out_ref, lse_ref, mag = want
    o = out.detach().cpu().double().reshape(out_ref.shape)
    assert torch.isfinite(o).all(), name
    bound = 2.0 ** -8 * out_ref.abs() + (2.0 ** -8 + 2.0 ** -12 + 2 * delta) * mag + 1e-30
    over = ((o - out_ref).abs() / bound).max().item()
    rel = ((o - out_ref).norm() / out_ref.norm().clamp(min=1e-30)).item()
    print("  %s out: worst %.2f of its bound, relative L2 %.2e" % (name, over, rel), flush=True)
    assert over <= 1.0, (name, over)
    if lse is not None:
        s = lse.detach().cpu().double().reshape(lse_ref.shape)
        empty = torch.isinf(lse_ref)
        assert torch.equal(torch.isinf(s) & (s < 0), empty), name
        off = (s - lse_ref)[~empty].abs().max().item() if (~empty).any() else 0.0
        assert off <= 1e-4 + delta, (name, off)
