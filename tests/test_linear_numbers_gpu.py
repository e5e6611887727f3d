"""What numbers linear attention holds on the way: outputs of bf16 tokens whose terms cancel.

Tolerances.  Operands of 24 bits are exact (three parts of 8), so are their products with +1 and -1, and
what the matrix instructions' sums round is named at each test; on top comes the output's own
rounding, half a step of 2^-7."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.gpu
B = torch.bfloat16
HALF = 2.0 ** -8 * 1.01


def seeded(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("d", [64, 128])
def test_columns_of_the_state_that_cancel(d):
    """o = S[:, 0] - S[:, 1], two columns that differ in their last 10 bits.  Three instructions (one a
    part) add to it: each rounds once to 2^-24 of what it adds up, at most 4."""
    h, gen = 8, seeded(d)
    state = torch.rand((1, h, d, d), generator=gen, device="cuda") + 1.0
    state[..., 1] = state[..., 0] + (torch.rand((1, h, d), generator=gen, device="cuda") - 0.5) * 2.0 ** -13
    q = torch.zeros((5, h, d), dtype=B, device="cuda")
    q[..., 0], q[..., 1] = 1.0, -1.0
    k = torch.randn((5, h, d), generator=gen, device="cuda").to(B)
    o, end = zm.linear_attention(q, k, torch.zeros_like(k), state=state, scale=1.0)
    want = (state[0, ..., 0].double() - state[0, ..., 1].double()).expand(5, h, d)
    off = (o.double() - want).abs() - HALF * want.abs()
    assert off.max() <= 3 * 4 * 2.0 ** -24, f"{off.max().item():.3g}"
    assert torch.equal(end, state)


@pytest.mark.parametrize("d", [64, 128])
def test_products_of_tokens_that_cancel(d):
    """The last of three tokens reads T_0 - T_1, T_j = q.k_j of 24 bits, equal but for the last 8.  T's own
    sum rounds once to 2^-24 of 2 for each of the two, and three instructions once to 2^-24 of at most 4."""
    h, gen = 64, seeded(d)

    def eight_bits(*shape):  # in [1, 1.9]
        return (1.0 + torch.randint(0, 116, shape, generator=gen, device="cuda") / 128.0).to(B)

    q, k, v = (torch.zeros((3, h, d), dtype=B, device="cuda") for _ in range(3))
    q[2, :, 0], q[2, :, 1], q[2, :, 2] = 1.0, 2.0 ** -8, 2.0 ** -16
    k[:2] = eight_bits(h, d)  # the same for both ..
    k[:2, :, 2] = eight_bits(2, h)  # .. but here
    v[0], v[1] = 1.0, -1.0
    o, _ = zm.linear_attention(q, k, v, scale=1.0)
    want = (2.0 ** -16 * (k[0, :, 2].double() - k[1, :, 2].double()))[:, None].expand(h, d)
    off = (o[2].double() - want).abs() - HALF * want.abs()
    assert off.max() <= (2 * 2 + 3 * 4) * 2.0 ** -24, f"{off.max().item():.3g}"
    assert not o[:2].any()
