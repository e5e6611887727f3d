"""The gated delta rule where one order, one unit or 32 bits do not reach: many
ragged sequences (the longest start first), decays of every size over a long
sequence, growing states, token rows more than 2^32 bytes apart, two streams at
once.  Tolerances as in tests/test_delta_rule_gpu.py; where only the way differs, equal bits."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm
from delta_reference import inputs
from test_delta_rule_gpu import DTYPES, check, run

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "g", "beta")


def ragged(n_seq, seed, longest=200):
    g = torch.Generator().manual_seed(seed)
    offsets = [0]
    for c in torch.randint(0, longest, (n_seq,), generator=g).tolist():
        offsets.append(offsets[-1] + c)
    return offsets


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_seq,heads", [(150, 2), (1024, 1), (1100, 1)])
def test_many_ragged_sequences_are_what_each_is_alone(n_seq, heads, dtype):
    print(f"case delta ragged {n_seq} x {heads} {dtype}", flush=True)
    offsets = ragged(n_seq, n_seq)
    x = inputs(offsets[-1], heads, heads, 64, dtype, 3, n_seq=n_seq)
    o, end = run(x, offsets)
    do = torch.randn_like(x["v"], dtype=torch.float32).to(dtype)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    grads = zm.delta_rule_backward(do, *(x[k] for k in NAMES), state=x["state"], offsets=off)
    for b in list(range(0, n_seq, n_seq // 16)) + [n_seq - 1]:
        rows, own = slice(offsets[b], offsets[b + 1]), slice(b, b + 1)
        one = {k: x[k][rows] for k in NAMES}
        o1, end1 = zm.delta_rule(*one.values(), state=x["state"][own])
        assert torch.equal(o1, o[rows]) and torch.equal(end1, end[own]), f"sequence {b}"
        g1 = zm.delta_rule_backward(do[rows], *one.values(), state=x["state"][own])
        assert all(torch.equal(a, t[rows]) for a, t in zip(g1[:5], grads[:5])), f"gradients of sequence {b}"
        assert torch.equal(g1[5], grads[5][own]), f"gradient of state {b}"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_decays_of_every_size(d, dtype):
    # a chunk's decays add up to anything from nothing to a reset, chunk after chunk
    n = 900
    print(f"case delta decays d={d} {dtype}", flush=True)
    x = inputs(n, 2, 2, d, dtype, 50)
    g = torch.Generator(device="cuda").manual_seed(51)
    size = torch.tensor([0.0, 1e-3, 0.02, 0.3, 0.8, 1.5, 5.0, 40.0, 1e-4], device="cuda")
    pick = torch.randint(0, len(size), (-(-n // 32), 2), generator=g, device="cuda")
    x["g"] = -size[pick].repeat_interleave(32, 0)[:n].contiguous() * torch.rand((n, 2), generator=g, device="cuda")
    x["g"][500, 0] = float("-inf")
    x["g"][501:505, 1] = -300.0
    check(x, *run(x))


@pytest.mark.parametrize("dtype", DTYPES)
def test_growing_states(dtype):
    # g above 0: the state grows by a factor of up to 2 a token for 40 tokens, then shrinks
    x = inputs(260, 2, 2, 128, dtype, 60)
    x["g"][:] = 0.0
    x["g"][70:110, 0] = 0.69
    x["g"][120:200, 0] = -0.5
    x["g"][:, 1] = 0.05
    check(x, *run(x))


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_past_32_bits(dtype):
    # 200 rows of 2^24 elements: the last begins 3.3e9 elements after the first
    n, ld = 200, 1 << 24
    x = inputs(n, 4, 2, 64, dtype, 70)
    far = torch.empty((n, ld), dtype=dtype, device="cuda")
    cut = {"q": (0, 2), "k": (4096, 2), "v": (ld // 2, 4), "o": (ld - 256, 4)}
    view = {name: far[:, c:c + 64 * h].unflatten(1, (h, 64)) for name, (c, h) in cut.items()}
    for name in ("q", "k", "v"):
        view[name].copy_(x[name])
    do = torch.randn_like(x["v"], dtype=torch.float32).to(dtype)
    want, end = run(x)
    _, end2 = zm.delta_rule(view["q"], view["k"], view["v"], x["g"], x["beta"], state=x["state"], out=view["o"])
    assert torch.equal(view["o"], want) and torch.equal(end, end2)
    grads = zm.delta_rule_backward(do, *(x[k] for k in NAMES), state=x["state"])
    view["o"].copy_(do)
    out = [far[:, c:c + 64 * h].unflatten(1, (h, 64)) for c, h in ((8192, 2), (1 << 20, 2), (ld - 1024, 4))]
    out += [torch.empty_like(t) for t in grads[3:]]
    zm.delta_rule_backward(view["o"], view["q"], view["k"], view["v"], x["g"], x["beta"], state=x["state"], out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, grads))


def test_two_streams_at_once():
    a, b = inputs(1374, 8, 8, 128, torch.bfloat16, 80), inputs(1000, 2, 1, 64, torch.float32, 81)
    want = [run(a), run(b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(x))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w[0], o) and torch.equal(w[1], s) for o, s in g)


def test_one_tensor_for_several_arguments():
    # reading only: q, k and v may be one tensor, and the state may be replaced
    x = inputs(100, 2, 2, 64, torch.float32, 90)
    t = x["k"]
    want = zm.delta_rule(t.clone(), t.clone(), t.clone(), x["g"], x["beta"], state=x["state"])
    state = x["state"].clone()
    got = zm.delta_rule(t, t, t, x["g"], x["beta"], state=state, state_out=state)
    assert torch.equal(got[0], want[0]) and torch.equal(state, want[1])
    d = torch.randn_like(state)
    g1 = zm.delta_rule_backward(t, t, t, t, x["g"], x["beta"], state=x["state"], dstate=d)
    out = [torch.empty_like(y) for y in g1[:5]] + [d]
    zm.delta_rule_backward(t, t, t, t, x["g"], x["beta"], state=x["state"], dstate=d, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, g1))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,offsets,heads,heads_k", [(1000, None, 2, 1), (700, [3, 3, 90, 650, 650], 4, 4),
                                                     (1500, [0, 1100, 1110, 1490], 3, 1)])
def test_workspaces_hold_anything(n, offsets, heads, heads_k, dtype):
    # every byte 255 is NaN as fp32 and bf16: nothing is read that the call has not written
    n_seq = len(offsets) - 1 if offsets else 1
    print(f"case delta workspace n={n} {dtype}", flush=True)
    x = inputs(n, heads, heads_k, 64, dtype, n, n_seq=n_seq)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    args, kw = [x[k] for k in NAMES], dict(state=x["state"], offsets=off)
    do = torch.randn_like(x["v"], dtype=torch.float32).to(dtype)
    dstate = torch.randn_like(x["state"])
    desc = zm.DeltaDesc(heads, heads_k, 64, zm.BF16 if dtype == torch.bfloat16 else zm.F32, n_seq, 1.0, 64 * heads_k,
                        64 * heads_k, 64 * heads, 64 * heads)

    def full(size):
        return torch.full((max(size, 256),), 255, dtype=torch.uint8, device="cuda")

    live = slice(offsets[0], offsets[-1]) if offsets else slice(0, n)
    o, end = zm.delta_rule(*args, **kw, workspace=full(zm.delta_rule_workspace_size(desc, n)))
    o2, end2 = zm.delta_rule(*args, **kw)
    assert torch.equal(o[live], o2[live]) and torch.equal(end, end2) and not end.isnan().any()
    a = zm.delta_rule_backward(do, *args, **kw, dstate=dstate,
                               workspace=full(zm.delta_rule_backward_workspace_size(desc, n)))
    b = zm.delta_rule_backward(do, *args, **kw, dstate=dstate)
    assert all(torch.equal(s[live], t[live]) and not s[live].isnan().any() for s, t in zip(a[:5], b[:5]))
    assert torch.equal(a[5], b[5]) and not a[5].isnan().any()


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_token_that_is_not_finite(name, dtype):
    # token 200 of the first sequence (its chunk begins at 192), long enough for segments
    offsets = [0, 700, 800]
    x = inputs(800, 4, 2, 64, dtype, 95, n_seq=2)
    good = run(x, offsets)
    do = torch.randn_like(x["v"], dtype=torch.float32).to(dtype)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    good_g = zm.delta_rule_backward(do, *(x[k] for k in NAMES), state=x["state"], offsets=off)
    x[name][200, 0] = float("nan") if name != "q" else float("inf")
    heads = slice(0, 2) if name in ("q", "k") else slice(0, 1)   # value heads that read it
    rest = slice(heads.stop, 4)
    o, end = run(x, offsets)
    assert not o[200, heads].isfinite().any()
    assert torch.equal(o[:192], good[0][:192]) and torch.equal(o[700:], good[0][700:])
    assert torch.equal(o[:, rest], good[0][:, rest])
    assert torch.equal(end[1], good[1][1]) and torch.equal(end[:, rest], good[1][:, rest])
    g = zm.delta_rule_backward(do, *(x[k] for k in NAMES), state=x["state"], offsets=off)
    assert all(torch.equal(a[700:], b[700:]) for a, b in zip(g[:5], good_g[:5])) and torch.equal(g[5][1], good_g[5][1])
    assert all(torch.equal(a[:, rest], b[:, rest]) for a, b in zip(g[2:5], good_g[2:5]))
