"""Plain forms for the tests of the 8-bit cache with a factor for each block: 64-bit torch, block after block."""
import math

import torch

LOWEST, HIGHEST = -40, 40


def decoded(bits):
    """e4m3 from its bits."""
    bits = bits.long()
    exponent, fraction = (bits >> 3) & 15, bits & 7
    size = torch.where(exponent == 0, fraction.double() * 2.0 ** -9, (8 + fraction.double()) * torch.exp2(exponent.double() - 10))
    size = torch.where((bits & 127) == 127, math.nan, size)
    return torch.where(bits >= 128, -size, size)


def rounded(y):
    """To the nearest e4m3 value, ties to even, beyond 448 as 448 with its sign; NaN stays."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(2.0 ** -6, 448.0))) - 3)
    return torch.where(torch.isinf(y), y, (y / step).round() * step).clamp(-448.0, 448.0)


def exponent_for(top):
    """The least e in range with top <= 448 * 2^e."""
    e = LOWEST
    while e < HIGHEST and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def store(held, factor, x, at, block):
    """x [new, dim] of one head behind the `at` values that are held: held [tokens, dim] in units of the factors, factor a list
    with one for each block (its old content where there is one).  Both are changed."""
    new = x.shape[0]
    for b in range(at // block, -(-(at + new) // block)):
        p0, p1 = max(at, b * block), min(at + new, (b + 1) * block)
        part = x[p0 - at:p1 - at]
        finite = part[torch.isfinite(part)].abs()
        e = exponent_for(float(finite.max()) if finite.numel() else 0.0)
        if p0 > b * block:
            old = min(max(factor[b], 2.0 ** LOWEST), 2.0 ** HIGHEST) if not math.isnan(factor[b]) else 2.0 ** LOWEST
            before = math.floor(math.log2(old))
            e = max(e, before)
            if e != before:
                held[b * block:p0] = rounded(held[b * block:p0] * 2.0 ** (before - e))
        factor[b] = 2.0 ** e
        held[p0:p1] = rounded(part / 2.0 ** e)
