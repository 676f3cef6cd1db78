"""The two terms that scaled_attn_chunk makes of a query (e4m3, and e5m2 of what that leaves), for every bf16 value.

A row's largest value is scaled to [2^7, 2^8).  From 2^-6 on a value has e4m3's four significant bits or more above
2^-9, and the remainder, at most 8 units of bf16's last place, fits three bits.  Below, the first term is a multiple of 2^-9, the
remainder is at most 2^-10 and three bits of it are kept: half a step is 2^-14, 2^-21 of the row's largest."""
import torch


def test_terms_of_every_value():
    bits = torch.arange(1 << 15, dtype=torch.int32)
    x = (bits << 16).view(torch.float32)
    x = x[torch.isfinite(x)].double()
    x = x[(x < 2.0 ** 8) & ((x >= 2.0 ** -100) | (x == 0))]
    for sign in (1, -1):
        v = (sign * x).float()
        first = v.to(torch.float8_e4m3fn).float()
        rest = v - first
        second = rest.to(torch.float8_e5m2).float()
        off = (v.double() - first.double() - second.double()).abs()
        assert bool((off[v.abs() >= 2.0 ** -6] == 0).all())
        assert float(off.max()) <= 2.0 ** -14


def test_rows_too_small_to_be_scaled_to_2_to_the_7th():
    """A row whose largest is below 2^-119 is scaled by 2^126, the most that there is: its elements are multiples of 2^-133, so of 2^-7 then, and the terms keep
    each of them whole."""
    bits = torch.arange(1 << 15, dtype=torch.int32)
    x = (bits << 16).view(torch.float32).double()
    x = x[x < 2.0 ** -119]
    assert float(x[1]) == 2.0 ** -133
    v = (x * 2.0 ** 126).float()
    first = v.to(torch.float8_e4m3fn).float()
    second = (v - first).to(torch.float8_e5m2).float()
    assert bool((v.double() == first.double() + second.double()).all()) and bool((v.double() * 2.0 ** -126 == x).all())
