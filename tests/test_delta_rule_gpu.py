"""zm.delta_rule and zm.delta_rule_step against the recurrence token by token in 64
bits (tests/delta_reference.py).

Tolerance.  A chunk of 64 tokens is five products in a row (K K^T, T, K M, T X,
K^T U).  Each adds at most 128 terms in fp32, at most 24 roundings of a partial
sum, and leaves out part products under 3 * 2^-24: at most 32 * 2^-24 of the
norms of its factors; unit keys and rates in (0, 1) keep T's norm near 1 (2
allowed).  So a chunk adds at most 320 * 2^-24 of the largest state to the state's error, and since the
recurrence does not expand (beta |k|^2 <= 1, decays <= 1) the errors of chunks add up.
An output reads the state with |q| scale = scale; with bf16 io its own products
have two parts (2^-16 for each factor) and it is rounded by 2^-8 of itself."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm
from delta_reference import forward, inputs

pytestmark = pytest.mark.gpu

EPS = 320 * 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float32]


def check(x, got_o, got_s, offsets=None, scale=None, state="own"):
    n, _, d = x["q"].shape
    scale = d ** -0.5 if scale is None else scale
    args = [x[name] for name in ("q", "k", "v", "g", "beta")]
    o, end, top = forward(*args, x["state"] if state == "own" else state, offsets, scale)
    offsets = [0, n] if offsets is None else offsets
    for b in range(len(offsets) - 1):
        a, e = offsets[b], offsets[b + 1]
        chunks = max(1, -(-(e - a) // 64))
        vmax = x["v"][a:e].double().norm(dim=-1).amax(0) if e > a else torch.zeros_like(top[b])
        size = top[b] + vmax
        assert ((got_s[b].double() - end[b]).norm(dim=(1, 2)) <= EPS * chunks * size).all(), f"state of sequence {b}"
        bf16 = got_o.dtype == torch.bfloat16
        fp = (EPS * chunks + (2.0 ** -13 if bf16 else 0)) * size * abs(scale)
        tol = fp[None, :, None] + (2.0 ** -8 if bf16 else 2.0 ** -24) * 1.01 * o[a:e].abs()
        off = (got_o[a:e].double() - o[a:e]).abs()
        assert (off <= tol).all(), f"outputs of sequence {b}: {(off / tol).max().item():.3g} of the tolerance"


def run(x, offsets=None, **kw):
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    return zm.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], state=kw.pop("state", x["state"]), offsets=off, **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 17, 63, 64, 65, 127, 200])
def test_one_sequence(n, d, dtype):
    print(f"case delta n={n} d={d} {dtype}", flush=True)
    x = inputs(n, 2, 2, d, dtype, n + d)
    check(x, *run(x))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,heads_k,d", [(1, 1, 64), (3, 1, 128), (8, 2, 64), (6, 3, 128), (64, 64, 64)])
def test_heads(heads, heads_k, d, dtype):
    print(f"case delta heads={heads}/{heads_k} d={d} {dtype}", flush=True)
    x = inputs(90, heads, heads_k, d, dtype, heads)
    check(x, *run(x))


@pytest.mark.parametrize("dtype", DTYPES)
def test_packed_sequences(dtype):
    lengths = [5, 0, 64, 1, 130, 0, 0, 65, 3]
    offsets = [0]
    for c in lengths:
        offsets.append(offsets[-1] + c)
    offsets = [c + 7 for c in offsets]   # tokens before the first and behind the last sequence
    n = offsets[-1] + 13
    print(f"case delta packed {dtype}", flush=True)
    x = inputs(n, 4, 2, 128, dtype, 5, n_seq=len(lengths))
    out = torch.full((n, 4, 128), 7.0, dtype=dtype, device="cuda")
    o, end = run(x, offsets, out=out)
    check(x, o, end, offsets)
    assert (o[:7] == 7).all() and (o[offsets[-1]:] == 7).all()
    empty = [b for b, c in enumerate(lengths) if c == 0]
    assert torch.equal(end[empty], x["state"][empty])


def test_more_sequences_than_a_block_has_threads():
    n_seq = 2500
    g = torch.Generator().manual_seed(1)
    lengths = torch.randint(0, 5, (n_seq,), generator=g).tolist()
    offsets = [0]
    for c in lengths:
        offsets.append(offsets[-1] + c)
    print("case delta 2500 sequences", flush=True)
    x = inputs(offsets[-1], 1, 1, 64, torch.bfloat16, 3, n_seq=n_seq)
    o, end = run(x, offsets)
    for b in list(range(0, 40)) + [1023, 1024, 1025, 2047, 2048, n_seq - 1]:
        part = {k: (t[b:b + 1] if k == "state" else t[offsets[b]:offsets[b + 1]]) for k, t in x.items()}
        check(part, o[offsets[b]:offsets[b + 1]], end[b:b + 1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,n_seq,heads", [(1374, 1, 2), (2100, 1, 1), (3000, 3, 1)])
def test_segments(n, n_seq, heads, dtype):
    # long enough for several segments to a sequence
    print(f"case delta segments n={n} n_seq={n_seq} {dtype}", flush=True)
    offsets = [n * b // n_seq + (b % 2) * 5 for b in range(n_seq)] + [n]
    x = inputs(n, heads, heads, 64 if n == 2100 else 128, dtype, n, n_seq=n_seq, decay=0.01)
    check(x, *run(x, offsets), offsets)
    # the same from rows of one sequence without offsets
    if n_seq == 1:
        o1, s1 = run(x)
        o2, s2 = run(x, offsets)
        assert torch.equal(o1, o2) and torch.equal(s1, s2)


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_state_in_strides_scale_and_in_place(dtype):
    n = 150
    x = inputs(n, 4, 2, 64, dtype, 9)
    o, end = run(x, state=None, scale=0.5)
    check(x, o, end, scale=0.5, state=None)
    row = torch.zeros((n, 2 * 2 * 64 + 4 * 64 + 8), dtype=dtype, device="cuda")
    y = dict(x, q=row[:, :128].unflatten(1, (2, 64)), k=row[:, 128:256].unflatten(1, (2, 64)),
             v=row[:, 256:512].unflatten(1, (4, 64)))
    for name in ("q", "k", "v"):
        y[name].copy_(x[name])
    out = torch.zeros((n, 320), dtype=dtype, device="cuda")[:, :256].unflatten(1, (4, 64))
    base = run(x)
    state = x["state"].clone()
    o, end = run(y, state=state, state_out=state, out=out)
    assert end is state and torch.equal(o, base[0]) and torch.equal(state, base[1])


def test_frames_carry_the_state():
    # three frames one by one are the whole sequence up to rounding; the same call twice gives the same bits
    x = inputs(3 * 137, 2, 2, 128, torch.float32, 4)
    state = x["state"].clone()
    outs = []
    for f in range(3):
        part = {k: t[137 * f:137 * (f + 1)] for k, t in x.items() if k != "state"}
        o, _ = zm.delta_rule(*(part[k] for k in ("q", "k", "v", "g", "beta")), state=state, state_out=state)
        outs.append(o)
    check(x, torch.cat(outs), state)
    a, b = run(x), run(x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", DTYPES)
def test_resets_zero_rates_and_repeated_keys(dtype):
    n = 140
    x = inputs(n, 2, 2, 64, dtype, 12, decay=2.0)
    x["g"][20] = float("-inf")       # the state starts anew
    x["g"][70, 0] = -1e30
    x["beta"][30:40] = 0.0           # tokens that only read
    x["beta"][100:120] = 1.0
    x["k"][90:130] = x["k"][90]      # one key again and again
    x["g"][100:130] = 0.0
    check(x, *run(x))
    # what was before a reset does not matter after it
    y = dict(x, v=x["v"].clone(), state=x["state"] * 3)
    y["v"][:20] = -y["v"][:20]
    a, b = run(x), run(y)
    assert (a[0][20:].double() - b[0][20:].double()).abs().max() <= 1e-6


def test_growing_and_strong_decays():
    x = inputs(200, 2, 2, 64, torch.float32, 13)
    x["g"][:] = -60.0 * torch.rand(200, 2, device="cuda")
    check(x, *run(x))
    x["g"][:] = 0.0
    check(x, *run(x))


def test_a_nan_token_stays_in_its_sequence_and_head():
    x = inputs(260, 2, 2, 64, torch.bfloat16, 14, n_seq=2)
    x["v"][100, 1, 3] = float("nan")
    o, end = run(x, [0, 130, 260])
    assert o[100:130, 1, 3].isnan().all() and not o[:64].isnan().any() and not o[:, 0].isnan().any()
    assert not o[130:].isnan().any() and not end[1].isnan().any()


def test_offsets_out_of_range_are_clamped():
    n = 120
    x = inputs(n, 1, 1, 64, torch.float32, 15, n_seq=3)
    good, bad = [0, 50, 50, 120], [-9, 50, 20, 4_000_000]
    a, b = run(x, good), run(x, bad)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    one = dict(x, state=x["state"][:1])
    a, b = run(one, [0, 120]), run(one, [-1, 2 ** 31 - 1])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    o, end = run(one, [90, 10], out=torch.full((n, 1, 64), 3.0, device="cuda"))
    assert (o == 3).all() and torch.equal(end, one["state"])


def test_no_tokens_and_no_sequences():
    x = inputs(0, 2, 1, 64, torch.bfloat16, 16, n_seq=3)
    o, end = run(x, [0, 0, 0, 0])
    assert o.shape == (0, 2, 64) and torch.equal(end, x["state"])
    o, end = run(x, [0, 0, 0, 0], state=None)
    assert not end.any()
    o, end = run(dict(x, state=x["state"][:0]), [0])
    assert end.shape == (0, 2, 64, 64)
    assert zm.delta_rule_step(x["q"], x["k"], x["v"], x["g"], x["beta"], x["state"][:0]).shape == (0, 2, 64)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,heads,heads_k,d", [(1, 1, 1, 64), (1, 8, 8, 128), (5, 6, 2, 128), (67, 3, 3, 64)])
def test_steps(n, heads, heads_k, d, dtype):
    print(f"case delta step n={n} heads={heads}/{heads_k} d={d} {dtype}", flush=True)
    x = inputs(n, heads, heads_k, d, dtype, 3 * n + heads, n_seq=n, decay=0.5)
    x["g"][0, 0] = float("-inf")
    want_o, want_s, top = forward(*(x[k] for k in ("q", "k", "v", "g", "beta", "state")), list(range(n + 1)))
    state = x["state"].clone()
    o = zm.delta_rule_step(x["q"], x["k"], x["v"], x["g"], x["beta"], state)
    # dots of d fp32 terms (at most 8 + 4 roundings in a row) and three more operations
    size = (top + x["v"].double().norm(dim=-1))[..., None]
    assert ((state.double() - want_s).abs() <= 24 * 2.0 ** -24 * size[..., None]).all()
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    assert ((o.double() - want_o).abs() <= 40 * 2.0 ** -24 * size * d ** -0.5 + 1.01 * half * want_o.abs()).all()


def test_steps_continue_a_sequence():
    x = inputs(80, 2, 2, 128, torch.float32, 21)
    first = {k: t[:70] for k, t in x.items()if k != "state"}
    _, state = zm.delta_rule(*(first[k] for k in ("q", "k", "v", "g", "beta")), state=x["state"])
    outs = [zm.delta_rule_step(*(x[k][t:t + 1] for k in ("q", "k", "v", "g", "beta")), state) for t in range(70, 80)]
    o, end, top = forward(*(x[k] for k in ("q", "k", "v", "g", "beta", "state")))
    tol = 4 * EPS * (top[0].max() + 20)
    assert (torch.cat(outs).double() - o[70:]).abs().max() <= tol * 128 ** -0.5
    assert (state.double() - end).abs().max() <= tol


def test_another_stream_and_graph_replays():
    x = inputs(1000, 2, 1, 128, torch.bfloat16, 30, n_seq=2)
    off = torch.tensor([0, 400, 1000], dtype=torch.int32, device="cuda")
    args = [x[k] for k in ("q", "k", "v", "g", "beta")]
    out, end = torch.empty((1000, 2, 128), dtype=torch.bfloat16, device="cuda"), torch.empty_like(x["state"])
    step_state = x["state"].clone()
    one = [t[:2] for t in args]
    desc = zm.DeltaDesc(2, 1, 128, zm.BF16, 2, 1.0, 128, 128, 256, 256)
    ws = torch.empty(zm.delta_rule_workspace_size(desc, 1000), dtype=torch.uint8, device="cuda")

    def call():
        zm.delta_rule(*args, state=x["state"], offsets=off, out=out, state_out=end, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        zm.delta_rule_step(*one, step_state)
    torch.cuda.current_stream().wait_stream(side)
    want = [t.clone() for t in (out, end)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for r in range(3):
        off.copy_(torch.tensor([0, 400 - 70 * r, 1000], dtype=torch.int32))
        ws.random_(0, 255)
        graph.replay()
        got = [t.clone() for t in (out, end)]
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, (out, end)))
        if r == 0:
            assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_offsets_past_32_bits():
    # token rows 2^24 elements apart: the last ones start past 2^31 elements
    n, ld = 135, 1 << 24
    x = inputs(n, 2, 2, 64, torch.bfloat16, 31)
    base = run(x)
    buf = torch.empty(n * ld, dtype=torch.bfloat16, device="cuda")
    far = {k: buf[512 * i:].as_strided((n, 2, 64), (ld, 64, 1)) for i, k in enumerate(("q", "k", "v"))}
    for k, t in far.items():
        t.copy_(x[k])
    out = buf[2048:].as_strided((n, 2, 64), (ld, 64, 1))
    o, end = run(dict(x, **far), out=out)
    assert torch.equal(o, base[0]) and torch.equal(end, base[1])
