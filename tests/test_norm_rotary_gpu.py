"""zm.norm_rotary and its gradient against the formulas in 64 bits, the gradient by autograd
and against differences.

Tolerance.  A row's sums have at most 256 terms, added by lanes and then by exchanges: under 32
roundings.  x - mu is off by a rounding of x and by mu's error, r by the same relative to its
rows' own spread: with A the row's largest |x|, (|x| + A) r (1 + |xh|) |gamma| + |beta| bounds what
is rounded, and 64 steps of 2^-24 of it are allowed before the rotation (whose cosine and sine are
good to 2 steps), which adds two such values.  The gradient's dx has the sizes of its three
terms in that place.  Sums over tokens and heads: 256 steps (at most 100 terms to a lane here,
then exchanges, waves and slots).  On top comes half a step of the result itself."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
STEP = 2.0 ** -24
LAYOUTS = [zm.ROTARY_HALVES, zm.ROTARY_PAIRS, zm.ROTARY_AXIS_HALVES]


def dims(sections, layout):
    """The two dims of each pair and its axis."""
    P, first, out = sum(sections), 0, []
    for a, s in enumerate(sections):
        for p in range(first, first + s):
            out.append({0: (p, p + P), 1: (2 * p, 2 * p + 1), 2: (p + first, p + first + s)}[layout] + (a,))
        first += s
    return (torch.tensor(x, device="cuda", dtype=torch.long) for x in zip(*out))


def turn(x, pos, freqs, sections, layout, absolute=False):
    i, j, axis = dims(sections, layout)
    angle = pos.double()[:, axis] * freqs.double()
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = x[..., i], x[..., j]
    if absolute:
        return x.index_copy(2, i, a + b).index_copy(2, j, a + b)
    return x.index_copy(2, i, a * c - b * s).index_copy(2, j, a * s + b * c)


def reference(x, gamma, beta, eps, norm, *rot):
    mu = x.mean(-1, keepdim=True) if norm == zm.NORM_LAYER else 0.0
    xh = (x - mu) / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    y = xh if gamma is None else xh * gamma
    return turn(y if beta is None else y + beta, *rot)


def spread(x, eps, norm):
    """(|x| + A) r (1 + |xh|), xh, r."""
    mu = x.mean(-1, keepdim=True) if norm == zm.NORM_LAYER else 0.0
    r = 1 / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    xh, top = (x - mu) * r, x.abs().amax(-1, keepdim=True)
    return (x.abs() + top) * r * (1 + xh.abs()), xh, r, 1 + top * r


def inputs(n, hq, hk, d, dtype, sections, seed, affine=True, far=False, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = {"q": (rand(n, hq, d) * 1.5 + shift).to(dtype), "k": (rand(n, hk, d) * 1.5 + shift).to(dtype) if hk else None,
         "pos": torch.randint(0, 40, (n, len(sections)), generator=g, device="cuda", dtype=torch.int32),
         "freqs": torch.rand(sum(sections), generator=g, device="cuda")}
    if far:
        x["pos"] = x["pos"].float() * 12345.678
    for p in ("q", "k"):
        x[p + "_gamma"] = rand(d) * 0.2 + 1 if affine else None
        x[p + "_beta"] = rand(d) * 0.1 if affine else None
    return x


def run(x, sections, layout, norm, **kw):
    return zm.norm_rotary(x["q"], x["k"], x["pos"], x["freqs"], sections, q_gamma=x["q_gamma"], k_gamma=x["k_gamma"],
                          q_beta=x["q_beta"], k_beta=x["k_beta"], norm=norm, layout=layout, **kw)


def check(x, got, sections, layout, norm, eps=1e-6):
    rot = (x["pos"], x["freqs"], sections, layout)
    for p, y in zip(("q", "k"), got):
        if y is None:
            continue
        xd = x[p].double()
        want = reference(xd, x[p + "_gamma"], x[p + "_beta"], eps, norm, *rot)
        size = spread(xd, eps, norm)[0]
        if x[p + "_gamma"] is not None:
            size = size * x[p + "_gamma"].abs() + x[p + "_beta"].abs()
        tol = 64 * STEP * turn(size, *rot, absolute=True) + 1.01 * HALF[y.dtype] * want.abs()
        off = (y.double() - want).abs()
        assert (off <= tol).all(), f"{p}: {(off / tol).max().item():.3g} of the tolerance"


SHAPES = [(128, (16, 24, 24)), (64, (8, 12, 8)), (128, (5, 7, 11)), (64, (32,)), (8, (1, 2)), (256, (40, 41, 3, 2)),
          (256, (128,)), (24, (4, 8)), (16, (0, 8)), (200, (33, 1))]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("norm", [zm.NORM_RMS, zm.NORM_LAYER])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("d,sections", SHAPES)
def test_forward(d, sections, layout, norm, dtype):
    print(f"case norm_rotary d={d} {sections} layout={layout} norm={norm} {dtype}", flush=True)
    for n, hq, hk, affine in ((1, 1, 0, False), (37, 3, 1, True), (130, 2, 5, True)):
        x = inputs(n, hq, hk, d, dtype, sections, d + n, affine=affine, far=n == 130)
        check(x, run(x, sections, layout, norm), sections, layout, norm)


@pytest.mark.parametrize("norm", [zm.NORM_RMS, zm.NORM_LAYER])
def test_many_tokens_slices_and_in_place(norm):
    n, sections = 5000, (16, 24, 24)
    print("case norm_rotary 5000 tokens", flush=True)
    x = inputs(n, 8, 2, 128, torch.bfloat16, sections, 3)
    base = run(x, sections, 0, norm)
    check(x, base, sections, 0, norm)
    y = torch.zeros((n, 12 * 128 + 16), dtype=torch.bfloat16, device="cuda")
    s = dict(x, q=y[:, :1024].unflatten(1, (8, 128)), k=y[:, 1024:1280].unflatten(1, (2, 128)))
    s["q"].copy_(x["q"])
    s["k"].copy_(x["k"])
    got = run(s, sections, 0, norm, q_out=s["q"], k_out=s["k"])
    assert got[0] is s["q"] and torch.equal(got[0], base[0]) and torch.equal(got[1], base[1])
    assert not y[:, 1280:].any()


def test_rows_of_zeros_and_equal_elements_and_far_from_zero():
    x = inputs(50, 2, 2, 64, torch.float32, (32,), 4)
    x["q"][3] = 0.0
    x["q"][4] = 2.5
    for norm in (zm.NORM_RMS, zm.NORM_LAYER):
        check(x, run(x, (32,), 0, norm), (32,), 0, norm)
    x = inputs(50, 2, 2, 64, torch.float32, (32,), 5, shift=300.0)
    check(x, run(x, (32,), 0, zm.NORM_LAYER), (32,), 0, zm.NORM_LAYER)


def test_a_nan_stays_in_its_head_and_no_tokens():
    x = inputs(20, 2, 2, 64, torch.bfloat16, (32,), 6)
    base = run(x, (32,), 0, zm.NORM_LAYER)
    x["q"][7, 1, 5] = float("nan")
    q, k = run(x, (32,), 0, zm.NORM_LAYER)
    assert q[7, 1].isnan().all() and torch.equal(k, base[1])
    q[7, 1] = base[0][7, 1]
    assert torch.equal(q, base[0])
    x = inputs(0, 2, 2, 64, torch.bfloat16, (32,), 7)
    assert run(x, (32,), 0, zm.NORM_RMS)[0].shape == (0, 2, 64)
    got = zm.norm_rotary_backward(x["q"], x["k"], x["q"], x["k"], x["pos"], x["freqs"], (32,))
    assert not any(t.any() for t in got)


def backward(x, dq, dk, sections, layout, norm, **kw):
    return zm.norm_rotary_backward(dq, dk, x["q"], x["k"], x["pos"], x["freqs"], sections, q_gamma=x["q_gamma"],
                                   k_gamma=x["k_gamma"], norm=norm, layout=layout, **kw)


def check_backward(x, dys, got, sections, layout, norm, eps=1e-6):
    rot = (x["pos"], x["freqs"], sections, layout)
    for p, dy, dx, dg, db in zip(("q", "k"), dys, got[:2], got[2:4], got[4:]):
        if dy is None:
            assert dx is None and dg is None and db is None
            continue
        d = dy.shape[2]
        one = torch.ones(d, dtype=torch.float64, device="cuda")
        leaves = [x[p].double(), one.clone() if x[p + "_gamma"] is None else x[p + "_gamma"].double(), one * 0]
        for t in leaves:
            t.requires_grad_()
        want = torch.autograd.grad(reference(*leaves, eps, norm, *rot), leaves, dy.double())
        size, xh, r, wide = spread(x[p].double(), eps, norm)
        u = turn(dy.double().abs(), *rot, absolute=True)
        a = u * leaves[1].detach().abs()
        three = r * (a + a.mean(-1, keepdim=True) + xh.abs() * (a * xh.abs()).mean(-1, keepdim=True)) * wide * (1 + xh.abs())
        for name, y, w, s, steps in (("dx", dx, want[0], three, 96), ("dgamma", dg, want[1], (u * size).sum((0, 1)), 256),
                                     ("dbeta", db, want[2], u.sum((0, 1)), 256)):
            tol = steps * STEP * s + 1.01 * HALF[y.dtype] * w.abs()
            off = (y.double() - w).abs()
            assert (off <= tol).all(), f"{name} of {p}: {(off / tol).max().item():.3g} of the tolerance"


def grads(x, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [None if x[p] is None else torch.randn(x[p].shape, generator=g, device="cuda").to(x[p].dtype) for p in "qk"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("norm", [zm.NORM_RMS, zm.NORM_LAYER])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("d,sections", SHAPES)
def test_backward(d, sections, layout, norm, dtype):
    print(f"case norm_rotary backward d={d} {sections} layout={layout} norm={norm} {dtype}", flush=True)
    for n, hq, hk, affine in ((1, 1, 0, False), (37, 3, 1, True), (130, 2, 5, True)):
        x = inputs(n, hq, hk, d, dtype, sections, d + n, affine=affine, far=n == 130)
        dys = grads(x, n)
        check_backward(x, dys, backward(x, *dys, sections, layout, norm), sections, layout, norm)


@pytest.mark.parametrize("norm", [zm.NORM_RMS, zm.NORM_LAYER])
def test_backward_of_many_tokens_in_place_and_the_same_bits(norm):
    n, sections = 5000, (16, 24, 24)
    print("case norm_rotary backward 5000 tokens", flush=True)
    x = inputs(n, 8, 2, 128, torch.bfloat16, sections, 8)
    dys = grads(x, 9)
    base = backward(x, *dys, sections, 0, norm)
    check_backward(x, dys, base, sections, 0, norm)
    out = (dys[0].clone(), x["k"].clone()) + tuple(torch.empty_like(t) for t in base[2:])
    ws = torch.full((1024 * 4 * 128,), float("nan"), device="cuda")
    got = backward(dict(x, k=out[1]), out[0], dys[1], sections, 0, norm, out=out, workspace=ws)
    for a, b in zip(got, base):
        assert torch.equal(a, b)
    got = backward(x, *dys, sections, 0, norm, out=out[:2] + (None, out[3], None, None))
    assert torch.equal(got[0], base[0]) and torch.equal(got[3], base[3])


def test_differences():
    """A central difference of sum(y dy) over a small step: off by the step's square times the third
    derivative (|u| <= 3 steps: (r |u|)^3 times a few of the loss's size) and by the loss's rounding over it."""
    n, sections = 9, (8, 12, 8)
    x = inputs(n, 2, 1, 64, torch.float32, sections, 10)
    dys = grads(x, 11)
    got = dict(zip(("q", "k", "q_gamma", "k_gamma", "q_beta", "k_beta"), backward(x, *dys, sections, 2, zm.NORM_LAYER)))
    g = torch.Generator(device="cuda").manual_seed(12)

    def loss(y):
        return sum(float((o.double() * dy.double()).sum()) for o, dy in zip(run(y, sections, 2, zm.NORM_LAYER), dys))

    out = run(x, sections, 2, zm.NORM_LAYER)
    total = sum(float((o.double().abs() * dy.double().abs()).sum()) for o, dy in zip(out, dys))
    for name, grad in got.items():
        u, h = torch.randn(x[name].shape, generator=g, device="cuda"), 2.0 ** -7
        dif = (loss(dict(x, **{name: x[name] + h * u})) - loss(dict(x, **{name: x[name] - h * u}))) / (2 * h)
        want = float((grad.double() * u.double()).sum())
        # 16 steps of 2^-24 of each term over h; h^2 times 27 times the terms (r is about 1 / 1.5, |u| under 4)
        assert abs(dif - want) <= total * (16 * STEP / h + 27 * h * h / 6), name


def test_a_captured_call():
    sections = (16, 24, 24)
    x = inputs(300, 4, 2, 128, torch.bfloat16, sections, 13)
    dys = grads(x, 14)
    base = run(x, sections, 0, 0) + backward(x, *dys, sections, 0, 0)
    out = [torch.empty_like(t) for t in base]
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        run(x, sections, 0, 0, q_out=out[0], k_out=out[1])
        backward(x, *dys, sections, 0, 0, out=out[2:], workspace=ws)
    for _ in range(3):
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, base):
            assert torch.equal(a, b)
        run(x, sections, 0, 0)
