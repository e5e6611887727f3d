"""zm.linear_attention and zm.linear_attention_step against the recurrence token by token
in 64 bits (tests/linear_reference.py, with the tolerances)."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm
from linear_reference import ROUGH, check, chunks, forward, inputs

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


def args(x):
    return [x[name] for name in ("q", "k", "v", "g")]


def absolute(x):
    return [y if y is None or name == "g" else y.abs() for name, y in zip(("q", "k", "v", "g"), args(x))]


def compare(x, got, offsets=None, scale=None):
    n = x["q"].shape[0]
    want = forward(*args(x), x["state"], offsets, scale)
    state = None if x["state"] is None else x["state"].abs()
    size = forward(*absolute(x), state, offsets, None if scale is None else abs(scale))
    longest = max([b - a for a, b in zip(offsets, offsets[1:])] + [0]) if offsets else n
    steps = chunks(longest, x["q"].dtype) + 2
    a, e = (offsets[0], offsets[-1]) if offsets else (0, n)
    check("o", got[0][a:e], want[0][a:e], size[0][a:e], steps, ROUGH[got[0].dtype])
    check("state", got[1], want[1], size[1], steps)


def run(x, offsets=None, **kw):
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    return zm.linear_attention(*args(x), state=kw.pop("state", x["state"]), offsets=off, **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 17, 31, 32, 33, 63, 64, 65, 127, 200])
def test_one_sequence(n, d, dtype):
    print(f"case linear n={n} d={d} {dtype}", flush=True)
    x = inputs(n, 2, 2, d, dtype, n + d)
    compare(x, run(x))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,heads_k,d", [(1, 1, 64), (3, 1, 128), (8, 2, 64), (6, 3, 128), (64, 64, 64)])
def test_heads(heads, heads_k, d, dtype):
    print(f"case linear heads={heads}/{heads_k} d={d} {dtype}", flush=True)
    x = inputs(90, heads, heads_k, d, dtype, heads)
    compare(x, run(x))


@pytest.mark.parametrize("decay", ["token", "head", "none", "strided"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_kinds_of_decay(decay, dtype):
    print(f"case linear decay {decay} {dtype}", flush=True)
    x = inputs(150, 4, 2, 128, dtype, 8)
    if decay == "head":
        x["g"] = torch.tensor([-0.5, 0.0, -1e-3, -3.0], device="cuda")
    elif decay == "none":
        x["g"] = None
    elif decay == "strided":
        wide = torch.full((150, 11), float("nan"), device="cuda")
        wide[:, 3:7] = x["g"]
        x["g"] = wide[:, 3:7]
    compare(x, run(x))


@pytest.mark.parametrize("dtype", DTYPES)
def test_packed_sequences(dtype):
    lengths = [5, 0, 64, 1, 130, 0, 0, 65, 3]
    offsets = [7]
    for c in lengths:
        offsets.append(offsets[-1] + c)  # tokens before the first and behind the last sequence
    n = offsets[-1] + 13
    print(f"case linear packed {dtype}", flush=True)
    x = inputs(n, 4, 2, 128, dtype, 5, n_seq=len(lengths))
    for name in ("q", "k", "v"):  # what lies outside the sequences is not looked at
        x[name][:7] = float("nan")
        x[name][offsets[-1]:] = float("inf")
    out = torch.full((n, 4, 128), 7.0, dtype=dtype, device="cuda")
    o, end = run(x, offsets, out=out)
    compare(x, (o, end), offsets)
    assert (o[:7] == 7).all() and (o[offsets[-1]:] == 7).all()
    empty = [b for b, c in enumerate(lengths) if c == 0]
    assert torch.equal(end[empty], x["state"][empty])


def test_more_sequences_than_a_block_has_threads():
    n_seq = 2500
    g = torch.Generator().manual_seed(1)
    lengths = torch.randint(0, 5, (n_seq,), generator=g).tolist()
    lengths[1500] = 900  # among the short ones one that is cut
    offsets = [0]
    for c in lengths:
        offsets.append(offsets[-1] + c)
    print("case linear 2500 sequences", flush=True)
    x = inputs(offsets[-1], 1, 1, 64, torch.bfloat16, 3, n_seq=n_seq)
    o, end = run(x, offsets)
    for b in list(range(0, 30)) + [1023, 1024, 1025, 1499, 1500, 1501, 2047, 2048, n_seq - 1]:
        part = {k: (t[b:b + 1] if k == "state" else t[offsets[b]:offsets[b + 1]]) for k, t in x.items()}
        compare(part, (o[offsets[b]:offsets[b + 1]], end[b:b + 1]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,n_seq,heads", [(1374, 1, 2), (2100, 1, 1), (3000, 3, 1), (1500, 2, 40)])
def test_segments(n, n_seq, heads, dtype):
    # long enough for several segments to a sequence
    print(f"case linear segments n={n} n_seq={n_seq} {dtype}", flush=True)
    offsets = [n * b // n_seq + (b % 2) * 5 for b in range(n_seq)] + [n]
    x = inputs(n, heads, heads, 64 if n in (1500, 2100) else 128, dtype, n, n_seq=n_seq, decay=0.01)
    compare(x, run(x, offsets), offsets)
    # the same from rows of one sequence without offsets
    if n_seq == 1:
        o1, s1 = run(x)
        o2, s2 = run(x, offsets)
        assert torch.equal(o1, o2) and torch.equal(s1, s2)


@pytest.mark.parametrize("n", [150, 2000])
@pytest.mark.parametrize("dtype", DTYPES)
def test_no_state_in_strides_scale_and_in_place(dtype, n):
    print(f"case linear strides n={n} {dtype}", flush=True)
    x = inputs(n, 4, 2, 64, dtype, 9)
    compare(dict(x, state=None), run(x, state=None, scale=-0.5), scale=-0.5)
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
    # three frames one by one are the whole sequence; the same call twice gives the same bits
    x = inputs(3 * 137, 2, 2, 128, torch.float32, 4)
    state = x["state"].clone()
    outs = []
    for f in range(3):
        part = {k: t[137 * f:137 * (f + 1)] for k, t in x.items() if k != "state"}
        outs.append(zm.linear_attention(*args(part), state=state, state_out=state)[0])
    compare(x, (torch.cat(outs), state))
    a, b = run(x), run(x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", DTYPES)
def test_resets_strong_and_growing_decays(dtype):
    n = 140
    x = inputs(n, 2, 2, 64, dtype, 12, decay=2.0)
    x["g"][20] = float("-inf")       # the state starts anew
    x["g"][70, 0] = -1e30
    x["g"][100:120] = 0.0
    compare(x, run(x))
    # what was before a reset does not matter after it
    y = dict(x, v=x["v"].clone(), state=x["state"] * 3)
    y["v"][:20] = -y["v"][:20]
    assert torch.equal(run(x)[0][20:], run(y)[0][20:])
    x["g"][:] = -60.0 * torch.rand(n, 2, device="cuda")
    compare(x, run(x))
    x["g"][:] = 0.3 * torch.rand(n, 2, device="cuda")
    compare(x, run(x))
    x["g"][:] = torch.tensor([-20.0, 20.0], device="cuda").repeat(n // 2)[:, None]  # up and down
    compare(x, run(x))


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
    assert not run(x, [0, 0, 0, 0], state=None)[1].any()
    assert run(dict(x, state=x["state"][:0]), [0])[1].shape == (0, 2, 64, 64)
    assert zm.linear_attention_step(*args(x), x["state"][:0]).shape == (0, 2, 64)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,heads,heads_k,d,decay", [(1, 8, 8, 128, "token"), (37, 3, 1, 64, "token"),
                                                     (5, 4, 2, 128, "head"), (300, 2, 2, 64, "none")])
def test_step(n, heads, heads_k, d, decay, dtype):
    print(f"case linear step n={n} {heads}/{heads_k} d={d} {decay} {dtype}", flush=True)
    x = inputs(n, heads, heads_k, d, dtype, n + d, n_seq=n)
    if decay != "token":
        x["g"] = x["g"][0].contiguous() if decay == "head" else None
    state = x["state"].clone()
    o = zm.linear_attention_step(*args(x), state)
    compare(x, (o, state), list(range(n + 1)))


def test_step_by_step_is_the_whole_sequence():
    x = inputs(70, 2, 1, 64, torch.float32, 21)
    state = x["state"].clone()
    o = [zm.linear_attention_step(x["q"][t:t + 1], x["k"][t:t + 1], x["v"][t:t + 1], x["g"][t:t + 1], state)
         for t in range(70)]
    compare(x, (torch.cat(o), state))


def test_workspaces_full_of_nan():
    x = inputs(1000, 3, 3, 128, torch.bfloat16, 22, n_seq=2)
    base = run(x, [0, 700, 1000])
    desc = zm.LinearDesc(3, 3, 128, zm.BF16, 2, 1.0, 384, 384, 384, 384, 3)
    ws = torch.full((zm.linear_attention_workspace_size(desc, 1000) // 4,), float("nan"), device="cuda")
    o, end = run(x, [0, 700, 1000], workspace=ws)
    assert torch.equal(o, base[0]) and torch.equal(end, base[1])


def test_a_captured_call_on_a_stream_of_its_own():
    x = inputs(900, 2, 2, 128, torch.bfloat16, 23, n_seq=3)
    off = torch.tensor([0, 600, 640, 900], dtype=torch.int32, device="cuda")
    base = run(x, off.tolist())
    state, out = x["state"].clone(), torch.empty_like(base[0])
    desc = zm.LinearDesc(2, 2, 128, zm.BF16, 3, 1.0, 256, 256, 256, 256, 2)
    ws = torch.empty(zm.linear_attention_workspace_size(desc, 900), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        zm.linear_attention(*args(x), state=state, state_out=state, offsets=off, out=out, workspace=ws)
        side.synchronize()
        state.copy_(x["state"])
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            zm.linear_attention(*args(x), state=state, state_out=state, offsets=off, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        state.copy_(x["state"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, base[0]) and torch.equal(state, base[1])
        run(x, off.tolist())  # the program's own work between replays
