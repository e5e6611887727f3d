"""What numbers linear attention holds on the way: outputs of bf16 tokens whose terms cancel, and
the gradient where decays, lengths and values make the held states large.

Tolerances.  Where terms cancel: operands of 24 bits are exact (three parts of 8), so are their products
with +1 and -1, and what the matrix instructions' sums round is named at each test; on top comes
the output's own rounding, half a step of 2^-7.  Otherwise those of linear_reference.py."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm
import test_linear_attention_gpu as forwards
import test_linear_backward_gpu as backwards
from linear_reference import check, chunks, inputs

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


def whole(q, k, v, do, g, scale):
    """dq, dk, dv and dg of one sequence of one head from zero states, in 64 bits, from
    o_i = scale sum_{j <= i} exp(g_{j+1} + .. + g_i) (q_i.k_j) v_j as it stands:
    dg_t is the sum of X_ij = G_ij (q_i.k_j) (do_i.v_j) over i >= t > j."""
    q, k, v, do, g = (x.double() for x in (q, k, v, do, g))
    c = torch.cumsum(g, 0)
    n = len(c)
    low = torch.ones((n, n), dtype=torch.bool, device=q.device).tril()
    G = scale * torch.exp(torch.where(low, c[:, None] - c[None], -torch.inf))
    A, P = q @ k.T.contiguous(), do @ v.T.contiguous()
    X = G * A * P
    before = torch.cumsum(X, 1)  # [i, t - 1]: j < t
    upto = torch.flip(torch.cumsum(torch.flip(before, (0,)), 0), (0,))  # [t, t' - 1]: i >= t
    dg = torch.cat([torch.zeros(1, dtype=torch.float64, device=q.device), torch.diagonal(upto, -1)])
    return (G * P) @ k, (G * P).T.contiguous() @ q, (G * A).T.contiguous() @ do, dg


# Sequences of 34 chunks in one segment each: in the middle one the states are held less 2^55
# from either side, as a decay of 2^-3.3 a chunk makes them.
@pytest.mark.parametrize("kind", ["mean", "loss scale"])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("d,dtype", [(64, B), (128, B), (64, torch.float32), (128, torch.float32)])
def test_dg_in_long_segments(d, dtype, decay, kind):
    h, n_seq, ch = 16, 32, 32 if dtype == torch.float32 else 64
    length = 34 * ch
    n = n_seq * length
    print(f"case linear long segments d={d} {dtype} {decay} {kind}", flush=True)
    gen = seeded(d + n)

    def tokens(mean, size):
        x = torch.empty((n, h, d), dtype=dtype, device="cuda")
        for i in range(h):
            x[:, i] = ((torch.randn((n, d), generator=gen, device="cuda") + mean) * size).to(dtype)
        return x

    if kind == "mean":
        q, k, v, do = tokens(1.0, 1.0), tokens(1.0, 1.0), tokens(1.0, 8.0), tokens(1.0, 8.0)
    else:
        q, k, v, do = tokens(0.0, 1.0), tokens(0.0, 1.0), tokens(0.0, 1.0), tokens(0.0, 65536.0)
    rate = -3.3 * 0.6931471805599453 / ch
    head = torch.full((h,), rate, device="cuda")
    head[1::2] *= 1.02
    g = head if decay == "head" else (head * (0.5 + torch.rand((n, h), generator=gen, device="cuda")))
    offsets = torch.arange(0, n + 1, length, dtype=torch.int32, device="cuda")
    got = dict(zip(("dq", "dk", "dv", "dg"), zm.linear_attention_backward(do, q, k, v, g, offsets=offsets)))
    for i in (0, 9):
        of_head = 0.0, 0.0
        for b in (0, 17, 31) if decay == "token" else range(n_seq):
            at = slice(b * length, (b + 1) * length)
            x = [t[at, i] for t in (q, k, v, do)]
            gi = g[at, i] if decay == "token" else g[i].expand(length)
            want, size = whole(*x, gi, d ** -0.5), whole(*(t.abs() for t in x), gi, d ** -0.5)
            steps = 2 * chunks(length, dtype) + 2
            for name, w, s in zip(("dq", "dk", "dv"), want, size):
                check(name, got[name][at, i], w, s, steps)
            if decay == "token":
                check("dg", got["dg"][at, i], want[3], size[3], steps)
            of_head = of_head[0] + want[3].sum(), of_head[1] + size[3].sum()
        if decay == "head":
            check("dg", got["dg"][i], *of_head, steps)


# Values near the largest that the operator takes: 2^11 and states of 2^22, with |q|.|k| up to 2^29, (|q|.|k|)
# (|do|.|v|) up to 2^58, (|S| |q|).|do| up to 2^57 and <|S|, |dS|> of 2^56, below 2^60 all of them; a decay of 0.63 a token
# takes the powers beside them to 2^58 within a chunk of 64.
@pytest.mark.parametrize("decay", [0.63, 0.3, 0.02, 0.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [B, torch.float32])
def test_large_values(dtype, d, decay):
    n, h, size = 200, 2, 2.0 ** (11 if d == 64 else 10.5)
    print(f"case linear large values d={d} {dtype} decay {decay}", flush=True)
    x = inputs(n, h, 1, d, dtype, 3, decay=decay)
    for name in "qkv":
        x[name] = (x[name].float() * size).to(dtype)
    x["g"] = torch.full_like(x["g"], -decay)
    x["state"] *= size * size
    do, dstate = backwards.grads_in(x, 4)
    do, dstate = (do.float() * size).to(dtype), dstate * (size * size)
    forwards.compare(x, forwards.run(x))
    backwards.compare(backwards.run(do, dstate, x), do, dstate, x)


@pytest.mark.parametrize("dtype", [B, torch.float32])
def test_growing_states(dtype):
    """77 tokens of a = exp(0.5), 2^55 in all, down again and up once more."""
    n = 240
    x = inputs(n, 2, 2, 64, dtype, 5)
    x["g"][:] = -0.5
    x["g"][20:97] = 0.5
    x["g"][180:] = 0.5
    do, dstate = backwards.grads_in(x, 6)
    forwards.compare(x, forwards.run(x))
    backwards.compare(backwards.run(do, dstate, x), do, dstate, x)
