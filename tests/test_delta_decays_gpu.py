"""Decay factors of the gated delta rule where a running sum of decays is large.

With keys that are distinct unit vectors and rates of one nothing is added up: column
c of the state is the value that was last written there times its decays, so every
factor shows.  In units of u = 2^-24, relative: a factor 2^x of a 64-bit x has its
fraction rounded (|f| <= 1/2: 0.2) and an instruction of 1 ulp (2), and is
multiplied in (1): 3.2.  An fp32 operand goes into a product as three bf16 parts of
24 bits with their signs (0.25) and comes out with one rounding (1).  A value meets
the factor of its token (3.2), products (2 * 1.25) and the factor at the end of its
chunks (3.2): under 9 u.  Each further chunk, segment or change of the running
exponent is one more factor (3.2)."""
import math

import pytest
import torch

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float32]


def basis(n, heads, d, dtype, bits, seed):
    """Keys e_0, e_1, ... again and again; decays that add up to `bits` powers of two in 64 tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.eye(d, device="cuda")[torch.arange(n, device="cuda") % d][:, None].expand(n, heads, d)
    w = torch.rand((n, heads), generator=g, device="cuda") * 2
    return dict(k=k.contiguous().to(dtype), v=torch.randn((n, heads, d), generator=g, device="cuda").to(dtype),
                g=w * (bits * math.log(2) / 64), beta=torch.ones((n, heads), device="cuda"))


def written(x):
    """The state after the last token, from none: [heads, d (v), d (k)]."""
    n, heads, d = x["k"].shape
    after = torch.flip(torch.cumsum(torch.flip(x["g"].double(), (0,)), 0), (0,)) - x["g"].double()
    S = torch.zeros((heads, d, d), dtype=torch.float64, device="cuda")
    for t in range(max(0, n - d), n):
        S[:, :, t % d] = x["v"][t].double() * torch.exp(after[t])[:, None]
    return S


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,heads,d,bits,factors", [
    (64, 2, 64, -57.0, 2), (64, 2, 128, 57.0, 2), (128, 2, 128, -28.0, 3), (128, 4, 128, 28.0, 3),
    (100, 1, 128, -33.0, 3), (1374, 8, 128, -28.0, 5), (2000, 2, 64, -9.0, 4),
])
def test_the_state_has_its_24_bits(n, heads, d, bits, factors, dtype):
    print(f"case delta decays n={n} heads={heads} d={d} bits={bits} {dtype}", flush=True)
    x = basis(n, heads, d, dtype, bits, n + d)
    _, end = zm.delta_rule(x["k"], x["k"], x["v"], x["g"], x["beta"])
    want = written(x)
    off = (end[0].double() - want).norm(dim=1) / want.norm(dim=1).clamp_min(1e-300)
    bound = 3.2 * factors + 2.5
    if n > d:  # what a column held before is taken off it and leaves a rounding
        bound += 1
    assert off.max() <= bound * U, f"{off.max() / U:.3g} of 2^-24"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bits", [-57.0, 57.0])
def test_the_gradient_of_a_state_has_its_24_bits(bits, dtype):
    # columns of the first state that no key meets keep their place and take all the decays
    print(f"case delta backward decays bits={bits} {dtype}", flush=True)
    n, heads, d = 64, 2, 128
    x = basis(n, heads, d, dtype, bits, 5)
    dstate = torch.randn((1, heads, d, d), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    grads = zm.delta_rule_backward(torch.zeros_like(x["v"]), x["k"], x["k"], x["v"], x["g"], x["beta"], dstate=dstate)
    total = torch.exp(x["g"].double().sum(0))[:, None, None]
    want = dstate[0, :, :, n:].double() * total
    assert ((grads[5][0, :, :, n:].double() - want).abs() <= 3.2 * 1.01 * U * want.abs()).all()
    # dv of a token: its column of the gradient times the decays after it
    after = torch.flip(torch.cumsum(torch.flip(x["g"].double(), (0,)), 0), (0,)) - x["g"].double()
    dv = dstate[0, :, :, :n].double().permute(2, 0, 1) * torch.exp(after)[..., None]
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert ((grads[2].double() - dv).abs() <= (1.01 * half + (3.2 + 2.5) * U) * dv.abs()).all()
