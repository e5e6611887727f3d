"""zm.delta_rule_backward against autograd of the recurrence token by token in 64 bits
(tests/delta_reference.py), and against differences.

Tolerance.  As for the forward (tests/test_delta_rule_gpu.py) every product adds at
most 32 * 2^-24 of its factors' norms; a chunk goes through the forward's five products, the
reverse's five and, for dq, dk, dg and dbeta, three more, so 13 * 64 * 2^-24 =
832 * 2^-24 a chunk (T's norm taken as 2 again) and over all chunks their number
times that, of the sizes of what the products work on: the gradient of the state
(at most ||dstate|| + sum |do| scale, and per token |do| scale enters), the state
(||S||) and the tokens.  Per tensor the 2-norm of the error is compared with that
bound times the product of those sizes.  Rounded to bf16, results are off by
2^-8 of themselves, and the two-part products of dq and dk by 2^-16 of their
sizes."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm
from delta_reference import forward, gradient, inputs

pytestmark = pytest.mark.gpu

EPS = 832 * 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float32]
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dstate")


def case(n, heads, heads_k, d, dtype, seed, n_seq=1, decay=0.1):
    x = inputs(n, heads, heads_k, d, dtype, seed, n_seq, decay)
    g = torch.Generator(device="cuda").manual_seed(seed + 1000)
    x["do"] = torch.randn((n, heads, d), generator=g, device="cuda").to(dtype)
    x["dstate"] = torch.randn((n_seq, heads, d, d), generator=g, device="cuda") * d ** -0.5
    return x


def run(x, offsets=None, **kw):
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    return zm.delta_rule_backward(x["do"], x["q"], x["k"], x["v"], x["g"], x["beta"], state=x["state"],
                                  dstate=x["dstate"], offsets=off, **kw)


def check(x, got, offsets=None, scale=None):
    args = [x[k] for k in ("q", "k", "v", "g", "beta")]
    want = gradient(x["do"], *args, x["state"], x["dstate"], offsets, scale)
    n, _, d = x["q"].shape
    scale = d ** -0.5 if scale is None else scale
    offs = [0, n] if offsets is None else offsets
    chunks = sum(max(1, -(-(e - a) // 64)) for a, e in zip(offs, offs[1:]))
    _, _, top = forward(*args, x["state"], offsets, scale)
    S = top.max().item() if top.numel() else 0.0
    S += x["v"].double().norm(dim=-1).max().item() if n else 0.0
    # the largest gradient of a state: what comes in at the end and with every output
    D = (x["dstate"].double().norm(dim=(2, 3)).max().item() if x["dstate"] is not None and len(offs) > 1 else 0.0)
    D += abs(scale) * (x["do"].double().norm(dim=-1).sum(0).max().item() if n else 0.0)
    rep = x["v"].shape[1] // x["k"].shape[1]
    for name, a, b in zip(NAMES, got, want):
        err = (a.double() - b).norm().item()
        rows = max(1, b.numel() // (d * d if name == "dstate" else 1 if name in ("dg", "dbeta") else d)) ** 0.5
        size = {"dq": abs(scale) * S * x["do"].double().norm(dim=-1).max().item() if n else 0, "dk": S * D,
                "dv": D, "dg": S * D, "dbeta": S * D, "dstate": D}[name]
        tol = EPS * chunks * size * rows * rep
        if a.dtype == torch.bfloat16:
            tol += 2.0 ** -8 * 1.01 * b.norm().item() + 4 * 2.0 ** -16 * size * rows * rep
        assert err <= tol, f"{name}: {err:.3g}, {err / tol:.3g} of the tolerance"
        # the bounds above are for the worst case; a wrong term is far over this
        if b.norm() > 0:
            assert err <= (0.004 if a.dtype == torch.bfloat16 else 2e-4) * b.norm().item() + 1e-9, f"{name}: {err / b.norm():.3g}"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 17, 64, 65, 150])
def test_one_sequence(n, d, dtype):
    print(f"case delta backward n={n} d={d} {dtype}", flush=True)
    x = case(n, 2, 2, d, dtype, n + d)
    check(x, run(x))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,heads_k,d", [(1, 1, 64), (3, 1, 128), (8, 2, 64), (6, 3, 128)])
def test_shared_heads(heads, heads_k, d, dtype):
    print(f"case delta backward heads={heads}/{heads_k} d={d} {dtype}", flush=True)
    x = case(90, heads, heads_k, d, dtype, heads)
    check(x, run(x))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads_k", [1, 2])
def test_packed_sequences(heads_k, dtype):
    lengths = [5, 0, 64, 1, 100, 0]
    offsets = [3]
    for c in lengths:
        offsets.append(offsets[-1] + c)
    n = offsets[-1] + 9
    print(f"case delta backward packed {dtype}", flush=True)
    x = case(n, 2, heads_k, 64, dtype, 5, n_seq=len(lengths))
    out = [torch.full(t, 7.0, dtype=dt, device="cuda") for t, dt in
           (((n, heads_k, 64), dtype), ((n, heads_k, 64), dtype), ((n, 2, 64), dtype), ((n, 2), torch.float32),
            ((n, 2), torch.float32), ((6, 2, 64, 64), torch.float32))]
    got = run(x, offsets, out=out)
    for t in got[:5]:
        assert (t[:3] == 7).all() and (t[offsets[-1]:] == 7).all()
        t[:3] = 0
        t[offsets[-1]:] = 0
    check(x, got, offsets)
    assert torch.equal(got[5][[1, 5]], x["dstate"][[1, 5]])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,n_seq,d", [(1200, 1, 64), (1300, 2, 128)])
def test_segments(n, n_seq, d, dtype):
    print(f"case delta backward segments n={n} n_seq={n_seq} {dtype}", flush=True)
    offsets = [n * b // n_seq + (b % 2) * 5 for b in range(n_seq)] + [n]
    x = case(n, 1, 1, d, dtype, n, n_seq=n_seq, decay=0.01)
    check(x, run(x, offsets), offsets)


def test_resets_zero_rates_and_repeated_keys():
    n = 140
    x = case(n, 2, 2, 64, torch.float32, 12, decay=1.0)
    x["g"][70, 0] = -1e30
    x["g"][20] = -200.0
    x["beta"][30:40] = 0.0
    x["k"][90:130] = x["k"][90]
    got = run(x)
    check(x, got)
    # nothing of the first tokens reaches what is after the reset
    y = dict(x, do=x["do"].clone())
    y["do"][:20] = 0
    assert torch.equal(run(y)[5], torch.zeros_like(got[5]))
    inf = dict(x, g=x["g"].clone())
    inf["g"][20] = float("-inf")
    assert all(torch.equal(a, b) for a, b in zip(run(inf), got))


def test_none_for_states_strides_scale_and_repeats():
    n = 100
    x = case(n, 4, 2, 64, torch.bfloat16, 9)
    x["state"] = x["dstate"] = None
    got = run(x, scale=0.7)
    zero = torch.zeros((1, 4, 64, 64), device="cuda")
    check(dict(x, state=zero, dstate=zero), got, scale=0.7)
    assert all(torch.equal(a, b) for a, b in zip(got, run(x, scale=0.7)))
    buf = torch.zeros((n, 2 * 128 + 256 + 16), dtype=torch.bfloat16, device="cuda")
    out = (buf[:, :128].unflatten(1, (2, 64)), buf[:, 128:256].unflatten(1, (2, 64)), buf[:, 256:512].unflatten(1, (4, 64)),
           got[3].clone(), got[4].clone(), got[5].clone())
    do = torch.zeros((n, 264), dtype=torch.bfloat16, device="cuda")[:, :256].unflatten(1, (4, 64))
    do.copy_(x["do"])
    assert all(torch.equal(a, b) for a, b in zip(got, run(dict(x, do=do), scale=0.7, out=out)))
    assert not buf[:, 512:].any()


def test_against_differences():
    # <o, do> + <S, dstate> by central differences in 64 bits along random directions
    x = case(70, 2, 1, 64, torch.float32, 40)
    got = run(x)
    g = torch.Generator(device="cuda").manual_seed(2)
    for name, grad in zip(("q", "k", "v", "g", "beta", "state"), got):
        way = torch.randn(x[name].shape, generator=g, device="cuda", dtype=torch.float64)
        vals = []
        for s in (1e-5, -1e-5):
            y = {k: t.double() for k, t in x.items()}
            y[name] = y[name] + s * way
            o, end, _ = forward(*(y[k] for k in ("q", "k", "v", "g", "beta", "state")))
            vals.append((o * y["do"]).sum() + (end * y["dstate"]).sum())
        diff = (vals[0] - vals[1]) / 2e-5
        want = (grad.double() * way).sum()
        # the kernel's own error is under 1e-4 of the gradient's norm (test above), a
        # direction picks up at most |way| / sqrt(size) of it; the differences' is 1e-10
        assert abs((diff - want).item()) <= 2e-4 * grad.double().norm().item() + 1e-6, name


def test_no_tokens():
    x = case(0, 2, 1, 64, torch.bfloat16, 16, n_seq=2)
    got = run(x, [0, 0, 0])
    assert torch.equal(got[5], x["dstate"]) and got[0].shape == (0, 1, 64)
    got = run(dict(x, state=x["state"][:0], dstate=x["dstate"][:0]), [0])
    assert got[5].shape == (0, 2, 64, 64)


def test_graph_replays_on_another_stream():
    x = case(700, 2, 1, 128, torch.bfloat16, 30, n_seq=2)
    off = torch.tensor([0, 300, 700], dtype=torch.int32, device="cuda")
    args = [x[k] for k in ("do", "q", "k", "v", "g", "beta")]
    kw = dict(state=x["state"], dstate=x["dstate"], offsets=off)
    out = zm.delta_rule_backward(*args, **kw)
    want = [t.clone() for t in out]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        zm.delta_rule_backward(*args, **kw, out=out)
    for r in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        zm.delta_rule_backward(*args, **kw)
