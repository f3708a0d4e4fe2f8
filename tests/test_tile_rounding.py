"""How the attention of many rows rounds stored keys and values to 16-bit floats, checked in plain arithmetic on the CPU for
every scale and every quant: to 11 bits, or to 2^-17 (Q4_0) or 2^-20 (Q8_0) of the largest value that the largest scale of their 32
neighbouring positions holds, 8 or 127 times that scale.

The kernel takes that scale to [2^10, 2^11) (Q4_0) or [2^14, 2^15) and forms, for unsigned quants u with u 2^-20 (or u 2^-24) exact,
fma(u 2^-20, d, o), o = d * -2^-17 rounded (128 2^-24 and 8 2^-20 are both 2^-17).  Results are below 2^-6 or 2^-2, and 16-bit floats have
no step finer than 2^-24.  Where d is at least 2^3, o is exact and the fma rounds once: 11 bits, or half a step, 2^-25.  Below, o may be off
by 2^-25 too, 2^-24 together.  The largest value is at least 8 2^10 2^-20 = 2^-7, or 127 2^14 2^-24 = 2^-3 (1 - 2^-7): quotients of 2^-17 and
just above 2^-21.

f16 tokens take two terms of each scale of at least 2^3: its first 8 (Q4_0) or 4 bits and the rest.  The first one's products with quants
have 11 bits and are exact; Q4_0's second ones have 6 bits, Q8_0's are rounded to 11 bits of at most 2^-3 of the value: 2^-14."""
import numpy as np
import pytest


def f16(x):
    return np.asarray(x, np.float64).astype(np.float16).astype(np.float64)


def decoded(bits, d, e, terms):
    """The kernel's tile values for every scale of d (in columns: every quant) with largest exponent field e, and the exact ones."""
    x = (25 if bits == 4 else 29) - e
    dn = f16(f16(d * 2.0 ** min(x, 15)) * 2.0 ** (x - min(x, 15)))
    first = (dn.astype(np.float16).view(np.uint16) & (0xfff8 if bits == 4 else 0xff80)).view(np.float16).astype(np.float64)
    first = np.where((dn >= 8) & (terms == 2), first, dn)
    u = np.arange(1 << bits, dtype=np.float64)
    forms = [0, 0] if bits == 4 else [0]                        # (two positions of a nibble)
    for t in (first, dn - first):
        o, t = f16(t * -2.0 ** -17)[:, None], t[:, None]
        if bits == 8:
            forms[0] = forms[0] + f16(u * 2.0 ** -24 * t + o)
        else:
            forms[0], forms[1] = forms[0] + f16(u * 2.0 ** -24 * f16(16 * t) + o), forms[1] + f16(u * 2.0 ** -20 * t + o)
    return forms, (u - (8 if bits == 4 else 128)) * d[:, None] * 2.0 ** (x - (20 if bits == 4 else 24))


@pytest.mark.parametrize("terms", [1, 2])
@pytest.mark.parametrize("bits,bound", [(4, 2.0 ** -17), (8, 2.0 ** -20)])
def test_every_scale_and_quant(bits, bound, terms):
    relative = 2.0 ** -11 if terms == 1 else 0.0 if bits == 4 else 2.0 ** -14
    scales = np.arange(0x7c00, dtype=np.uint16)                 # every finite one; signs change nothing
    for e in (0, 1, 2, 5, 8, 11, 14, 15, 17, 20, 24, 29, 30):
        d = scales[scales >> 10 <= e].view(np.float16).astype(np.float64)
        forms, exact = decoded(bits, d, e, terms)
        # the smallest scale with this exponent field, times what its block holds at most
        least = (2.0 ** (e - 15) if e else 2.0 ** -24) * (8 if bits == 4 else 127) * 2.0 ** (5 - e)
        for got in forms:
            assert np.isfinite(got).all()
            assert (np.abs(got - exact) <= relative * np.abs(exact) + bound * least).all(), (e, bits)
            if bits == 4 and e >= 15:                           # the bound is no looser than twice
                assert (np.abs(got - exact) > relative * np.abs(exact) + bound / 2 * least).any()
