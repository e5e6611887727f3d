"""Outputs of the gated delta rule where they are what is left of large terms.

A token whose key is a unit vector and whose rate is one replaces what the state holds
for that key: read with the same vector, o = scale v, whatever was there before, as the
difference of scale gam M q and of that within P U.  Of what was there (in units
of 2^-24 of it) the products K M and Q M, the difference, T X and P U each add at
most one rounding and a split of 24 bits (1.25): under 8.  The token's own value
meets two factors of its decays (3.2 each) and three roundings: under 10."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,heads,heads_k,d,strong", [
    (64, 2, 2, 64, False), (40, 1, 1, 64, True), (128, 2, 1, 128, False), (100, 3, 3, 128, True),
])
def test_a_replaced_value_leaves_nothing(n, heads, heads_k, d, strong, dtype):
    print(f"case delta overwrite n={n} heads={heads}/{heads_k} d={d} strong={strong} {dtype}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(n + d)
    k = torch.eye(d, device="cuda")[torch.arange(n, device="cuda") % d][:, None].expand(n, heads_k, d)
    k = k.contiguous().to(dtype)
    v = torch.randn((n, heads, d), generator=gen, device="cuda").to(dtype)
    g = -0.02 * torch.rand((n, heads), generator=gen, device="cuda")
    if strong:  # the chunk is formed with its decays in place
        g[n - 1] = -100.0
    state = 4096 * torch.randn((1, heads, d, d), generator=gen, device="cuda")
    o, _ = zm.delta_rule(k, k, v, g, torch.ones_like(g), state=state, scale=0.5)
    held = torch.stack([state[0, :, :, t % d].double().abs() for t in range(n)])
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    want = 0.5 * v.double()
    bound = 0.5 * 8 * U * held + (1.01 * half + 10 * U) * want.abs()
    off = (o.double() - want).abs()
    assert (off <= bound).all(), f"{(off / bound).max():.3g} of the bound"
