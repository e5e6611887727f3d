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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,heads,d", [(64, 2, 64), (40, 1, 128), (128, 2, 128)])
def test_the_gradient_of_a_replaced_value_leaves_nothing(n, heads, d, dtype):
    # dq_t = scale S_t^T do_t, from M^T do and W K, which cancel where a key was replaced.  Without decays
    # and with one element of do to a token nothing is added up: K M, the difference, T X, U dO^T, its product
    # with K, M^T dO and their sum round once each, and the operands' splits add 0.25 five times: under 10.
    print(f"case delta backward overwrite n={n} heads={heads} d={d} {dtype}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(n + d + 1)
    at = torch.arange(n, device="cuda") % d
    k = torch.eye(d, device="cuda")[at][:, None].expand(n, heads, d).contiguous().to(dtype)
    v = torch.randn((n, heads, d), generator=gen, device="cuda").to(dtype)
    g = torch.zeros((n, heads), device="cuda")
    state = 4096 * torch.randn((1, heads, d, d), generator=gen, device="cuda")
    do = torch.zeros_like(v)
    row = torch.randint(0, d, (n,), generator=gen, device="cuda")
    do[torch.arange(n, device="cuda"), :, row] = torch.randn((n, heads), generator=gen, device="cuda").to(dtype)
    dq = zm.delta_rule_backward(do, k, k, v, g, torch.ones_like(g), state=state, scale=0.5)[0]
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    S = state[0].double().clone()
    for t in range(n):
        S[:, :, at[t]] = v[t].double()
        w = 0.5 * do[t, :, row[t]].double()[:, None]
        want, held = w * S[:, row[t]], (w * state[0, :, row[t]].double()).abs()
        off = (dq[t].double() - want).abs()
        bound = 10 * U * (held + want.abs()) + 1.01 * half * want.abs()
        assert (off <= bound).all(), f"token {t}: {(off / bound).max():.3g} of the bound"
