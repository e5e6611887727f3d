"""The cosines and sines of zm.rotary themselves, as the rotation of (1, 0).

A sine or cosine of half turns is within 4 ulp of its argument's (8 * 2^-24 of itself),
the part of the angle that 32 bits leave out adds one rounding (2^-24), and the 64-bit
angle is off by two roundings of a product and one of 1 / (2 pi): 2^-51 of itself.
The products with 1 and 0 add nothing.  An angle rounded to 32 bits as a part of a turn
would be off by up to 9e-8, which shows where a sine is small: near half a turn."""
import math

import pytest
import torch

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", [0, 1, 2])
@pytest.mark.parametrize("n,pairs,far", [(300, 32, 0), (257, 28, 4000), (100, 5, 1_000_000)])
def test_angles_keep_their_bits(n, pairs, far, layout, inverse):
    print(f"case rotary angles n={n} pairs={pairs} far={far} layout={layout} inverse={inverse}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(n)
    d = 64
    # odd multiples of about pi
    freqs = (math.pi * (1 + 0.02 * (2 * torch.rand(pairs, generator=gen, device="cuda") - 1) / (1 + far))).float()
    pos = 2 * torch.randint(0, 20 + far, (n, 1), generator=gen, device="cuda", dtype=torch.int32) + 1
    pos[::5] //= 2  # and any others
    i = torch.arange(pairs, device="cuda")
    a, b = (2 * i, 2 * i + 1) if layout == 1 else (i, i + pairs)
    q = torch.zeros((n, 1, d), device="cuda")
    q[..., a] = 1.0
    y, _ = zm.rotary(q, None, pos, freqs, (pairs,), layout=layout, inverse=inverse)
    angle = pos.double() * freqs.double() * (-1 if inverse else 1)
    for got, want in ((y[:, 0, a], torch.cos(angle)), (y[:, 0, b], torch.sin(angle))):
        bound = 9 * U * want.abs() + angle.abs() * 2.0 ** -51
        off = (got.double() - want).abs()
        assert (off <= bound).all(), f"{(off / bound).max():.3g} of the bound"
