"""zm.linear_attention_backward against the recurrence's gradient in 64 bits (autograd,
tests/linear_reference.py, with the tolerances) and against differences of the forward."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm
from linear_reference import check, chunks, gradient, inputs

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
NAMES = ("dq", "dk", "dv", "dg", "dstate")


def grads_in(x, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(x["v"].shape, generator=g, device="cuda").to(x["v"].dtype),
            torch.randn(x["state"].shape, generator=g, device="cuda"))


def args(x):
    return [x[name] for name in ("q", "k", "v", "g")]


def run(do, dstate, x, offsets=None, **kw):
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    return zm.linear_attention_backward(do, *args(x), state=x["state"], dstate=dstate, offsets=off, **kw)


def compare(got, do, dstate, x, offsets=None, scale=None):
    n = x["q"].shape[0]
    size = lambda t: None if t is None else t.abs()  # noqa: E731
    want = gradient(do, *args(x), x["state"], dstate, offsets, scale)
    sizes = gradient(do.abs(), *[size(t) for t in args(x)[:3]], x["g"], size(x["state"]), size(dstate), offsets, scale)
    longest = max([b - a for a, b in zip(offsets, offsets[1:])] + [0]) if offsets else n
    # twice: a gradient's term passes through the states before and behind its token; a sum over all
    # tokens (one decay to a head) has its own rounding for each, far below
    steps = 2 * chunks(longest, do.dtype) + 2
    a, e = (offsets[0], offsets[-1]) if offsets else (0, n)
    for name, y, w, s in zip(NAMES, got, want, sizes):
        if y is None:
            assert w is None and name == "dg"
        elif name == "dstate" or (name == "dg" and y.dim() == 1):
            check(name, y, w, s, steps)
        else:
            check(name, y[a:e], w[a:e], s[a:e], steps)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 31, 33, 63, 64, 65, 130])
def test_one_sequence(n, d, dtype):
    print(f"case linear backward n={n} d={d} {dtype}", flush=True)
    x = inputs(n, 2, 2, d, dtype, n + d)
    do, dstate = grads_in(x, n)
    compare(run(do, dstate, x), do, dstate, x)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,heads_k,d", [(1, 1, 64), (3, 1, 128), (8, 2, 64), (6, 3, 128)])
def test_shared_key_heads(heads, heads_k, d, dtype):
    print(f"case linear backward heads={heads}/{heads_k} d={d} {dtype}", flush=True)
    x = inputs(90, heads, heads_k, d, dtype, heads)
    do, dstate = grads_in(x, 1)
    compare(run(do, dstate, x, scale=0.7), do, dstate, x, scale=0.7)


@pytest.mark.parametrize("decay", ["head", "none"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [100, 700])
def test_one_decay_to_a_head_and_none(decay, dtype, n):
    print(f"case linear backward decay {decay} {dtype}", flush=True)
    x = inputs(n, 4, 2, 128, dtype, 8, n_seq=2)
    x["g"] = torch.tensor([-0.5, 0.0, -1e-3, -3.0], device="cuda") if decay == "head" else None
    do, dstate = grads_in(x, 2)
    offsets = [3, 70, n - 9]
    compare(run(do, dstate, x, offsets), do, dstate, x, offsets)


@pytest.mark.parametrize("dtype", DTYPES)
def test_packed_sequences(dtype):
    lengths = [5, 0, 64, 1, 130, 0, 0, 65, 3]
    offsets = [7]
    for c in lengths:
        offsets.append(offsets[-1] + c)
    n = offsets[-1] + 13
    print(f"case linear backward packed {dtype}", flush=True)
    x = inputs(n, 4, 2, 64, dtype, 5, n_seq=len(lengths))
    do, dstate = grads_in(x, 3)
    like = lambda *shape, t=torch.float32: torch.full(shape, 7.0, dtype=t, device="cuda")  # noqa: E731
    out = (like(n, 2, 64, t=dtype), like(n, 2, 64, t=dtype), like(n, 4, 64, t=dtype), like(n, 4), like(9, 4, 64, 64))
    got = run(do, dstate, x, offsets, out=out)
    compare(got, do, dstate, x, offsets)
    for y in got[:4]:
        assert (y[:7] == 7).all() and (y[offsets[-1]:] == 7).all()
    empty = [b for b, c in enumerate(lengths) if c == 0]
    assert torch.equal(got[4][empty], dstate[empty])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,n_seq,heads,d", [(1374, 1, 2, 128), (900, 2, 3, 64)])
def test_segments(n, n_seq, heads, d, dtype):
    print(f"case linear backward segments n={n} n_seq={n_seq} {dtype}", flush=True)
    offsets = [n * b // n_seq for b in range(n_seq)] + [n]
    x = inputs(n, heads, heads, d, dtype, n, n_seq=n_seq, decay=0.01)
    do, dstate = grads_in(x, 4)
    compare(run(do, dstate, x, offsets), do, dstate, x, offsets)
    # the gradient of the first states in the place of that of the last ones
    base = run(do, dstate, x, offsets)
    out = tuple(torch.empty_like(y) for y in base[:4]) + (dstate.clone(),)
    again = run(do, out[4], x, offsets, out=out)
    for name, a, b in zip(NAMES, again, base):
        assert torch.equal(a, b), name


@pytest.mark.parametrize("dtype", DTYPES)
def test_strong_decays_and_resets(dtype):
    n = 200
    x = inputs(n, 2, 2, 64, dtype, 12, decay=2.0)
    x["g"][20] = float("-inf")
    x["g"][70, 0] = -60.0
    x["g"][100:130] = 0.0
    x["g"][150] = -14.0  # one strong decay among weak ones: its gradient is small and has to be as exact
    do, dstate = grads_in(x, 5)
    got = run(do, dstate, x)
    y = dict(x, g=x["g"].clamp(min=-1e4))  # exp(-inf) has the gradient 0 times inf in autograd's eyes
    compare(got, do, dstate, y)
    assert (got[3][20] == 0).all()


def test_no_states():
    x = inputs(100, 2, 2, 64, torch.float32, 13)
    x["state"] = None
    do = torch.randn((100, 2, 64), device="cuda")
    compare(run(do, None, x), do, None, x)


def test_differences():
    """The forward is linear in each of q, k, v and the first state alone, so a difference over a whole
    step in one of them is its gradient times the step; in g it is taken over a small one, off by
    a 24th of its third power times the third derivative (|dg| sums of decays of up to n tokens)."""
    n, d = 77, 64
    x = inputs(n, 2, 1, d, torch.float32, 14)
    do, dstate = grads_in(x, 6)
    got = dict(zip(("q", "k", "v", "g", "state"), run(do, dstate, x)))
    gen = torch.Generator(device="cuda").manual_seed(7)

    def loss(y):
        o, end = zm.linear_attention(*args(y), state=y["state"])
        return float((o.double() * do.double()).sum() + (end.double() * dstate.double()).sum())

    # what the loss's rounding can be: 64 steps for each of the chunks and two more of the sum of sizes
    size = dict(x, **{k: x[k].abs() for k in ("q", "k", "v", "state")})
    o, end = zm.linear_attention(*args(size), state=size["state"])
    rounding = 64 * (chunks(n, torch.float32) + 2) * 2.0 ** -24 * float(
        (o.double() * do.abs().double()).sum() + (end.double() * dstate.abs().double()).sum())
    for name in ("q", "k", "v", "state"):
        u = torch.randn(x[name].shape, generator=gen, device="cuda")
        dif = loss(dict(x, **{name: x[name] + u})) - loss(x)
        want = float((got[name].double() * u.double()).sum())
        # x + u is rounded, and the sizes are those of x + u: at most thrice those of x here
        assert abs(dif - want) <= 4 * rounding, name
    h = 2.0 ** -6
    for t in (0, 40, 76):
        u = torch.zeros_like(x["g"])
        u[t, 1] = h
        dif = (loss(dict(x, g=x["g"] + u)) - loss(dict(x, g=x["g"] - u))) / (2 * h)
        # moving one g moves one factor a_t: sinh(h) / h off by h^2 / 6, so h^2 / 5 of the gradient's own size
        assert abs(dif - float(got["g"][t, 1])) <= rounding / h + h * h / 5 * abs(dif)


def test_workspaces_full_of_nan_and_the_same_bits_again():
    x = inputs(1000, 3, 1, 128, torch.bfloat16, 22, n_seq=2)
    do, dstate = grads_in(x, 8)
    base = run(do, dstate, x, [0, 700, 1000])
    desc = zm.LinearDesc(3, 1, 128, zm.BF16, 2, 1.0, 128, 128, 384, 384, 3)
    need = zm.linear_attention_backward_workspace_size(desc, 1000)
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    for name, a, b in zip(NAMES, run(do, dstate, x, [0, 700, 1000], workspace=ws), base):
        assert torch.equal(a, b), name


def test_a_captured_call():
    x = inputs(700, 2, 1, 64, torch.bfloat16, 23, n_seq=3)
    do, dstate = grads_in(x, 9)
    off = torch.tensor([0, 500, 540, 700], dtype=torch.int32, device="cuda")
    base = run(do, dstate, x, off.tolist())
    out = tuple(torch.empty_like(y) for y in base)
    desc = zm.LinearDesc(2, 1, 64, zm.BF16, 3, 1.0, 64, 64, 128, 128, 2)
    ws = torch.empty(zm.linear_attention_backward_workspace_size(desc, 700), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        zm.linear_attention_backward(do, *args(x), state=x["state"], dstate=dstate, offsets=off, out=out, workspace=ws)
    for _ in range(3):
        for y in out:
            y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name, a, b in zip(NAMES, out, base):
            assert torch.equal(a, b), name
        run(do, dstate, x, off.tolist())
