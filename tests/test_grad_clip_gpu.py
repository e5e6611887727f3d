"""zm.grad_norm and zm.clip_grads against sums in 64 bits.

Tolerance.  Squares and their sums are in 64 bits, so the norm has its own rounding to 32 bits
(2^-24) and 2^-30 for all else.  A clipped element is a 64-bit product rounded to fp32 (half a step,
or of the smallest step where it is subnormal) and, for bf16, from there to bf16."""
import math

import pytest
import torch

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.gpu
B, F = torch.bfloat16, torch.float32
HALF = {B: 2.0 ** -8 + 2.0 ** -24, F: 2.0 ** -24}
TINY = {B: 2.0 ** -134, F: 2.0 ** -150}


def tensors(sizes, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=g, device="cuda") * scale * 10.0 ** -(i % 4)).to(t) for i, (s, t) in enumerate(sizes)]


def norm_of(xs):
    return math.sqrt(math.fsum(float(x.double().square().sum()) for x in xs))


def check(xs, ys, norm, max_norm):
    want = norm_of(xs)
    assert abs(float(norm) - want) <= want * (2.0 ** -24 + 2.0 ** -30)
    c = min(1.0, max_norm / (want + 1e-6))
    for i, (x, y) in enumerate(zip(xs, ys)):
        w = x.double() * c
        off, tol = (y.double() - w).abs(), w.abs() * (HALF[x.dtype] + 2.0 ** -30) + TINY[x.dtype] * 1.01
        assert (off <= tol).all(), f"tensor {i}: {(off - tol).max().item():.3g} over"


SIZES = [
    [(1, F)], [(1, B)], [(7, B), (3, F)], [(8, B)], [(9, B), (4, F), (5, F), (0, F), (17, B)],
    [(8192, F), (16384, B)], [(8193, F), (16385, B)], [(8191, F), (16383, B), (1, F)],
    [(300_001, B), (123_457, F)], [(0, F), (0, B), (5, F), (0, F)],
    [(100 + 37 * i, B if i % 3 else F) for i in range(128)], [(1 + 11 * i, B if i % 2 else F) for i in range(129)],
    [(i % 5, F if i % 2 else B) for i in range(700)], [(40_000_003, B)],
]


@pytest.mark.parametrize("max_norm", [0.5, 1e9, 0.0])
@pytest.mark.parametrize("which", range(len(SIZES)))
def test_in_place_and_apart(which, max_norm):
    print(f"case clip {which} max {max_norm}", flush=True)
    xs = tensors(SIZES[which], which)
    ys = [torch.full_like(x, 3.0) for x in xs]
    norm = zm.clip_grads(xs, max_norm, out=ys)
    check(xs, ys, norm, max_norm)
    assert float(zm.grad_norm(xs)) == float(norm)
    zs = [x.clone() for x in xs]
    again = zm.clip_grads(zm.TensorList(zs), max_norm, norm=torch.empty(1, device="cuda"))
    assert float(again) == float(norm)
    for y, z in zip(ys, zs):
        assert torch.equal(y, z)


def test_pieces_of_a_bucket_at_any_element():
    sizes = [5, 1, 33_000, 7, 64, 100_001, 2, 9, 0, 17]
    for t in (F, B):
        print(f"case clip bucket {t}", flush=True)
        flat = tensors([(sum(sizes) + 3, t)], 40)[0]
        xs = list(torch.split(flat[3:], sizes))
        out = torch.full((sum(sizes) + 8,), 9.0, dtype=t, device="cuda")
        for skip in (0, 1, 3):  # the outputs lie as the inputs do to 16 bytes, or not
            ys = list(torch.split(out[skip:skip + sum(sizes)], sizes))
            check(xs, ys, zm.clip_grads(xs, 0.25, out=ys), 0.25)
            assert (out[skip + sum(sizes):] == 9).all()
        want = [x.clone() for x in xs]
        zm.clip_grads(want, 0.25)
        head = flat[:3].clone()
        zm.clip_grads(xs, 0.25)
        assert torch.equal(torch.cat(want), torch.cat(xs)) and torch.equal(flat[:3], head)


def test_large_small_and_values_that_are_not_finite():
    big = [torch.full((1000,), 2e38, device="cuda"), torch.full((9,), -3e38, dtype=B, device="cuda")]
    ys = [torch.empty_like(x) for x in big]
    norm = zm.clip_grads(big, 1.0, out=ys)
    assert float(norm) == math.inf  # over fp32's range, but the factor is not: it is formed in 64 bits
    c = 1.0 / norm_of(big)
    for x, y in zip(big, ys):
        assert ((y.double() - x.double() * c).abs() <= (x.double() * c).abs() * 2 * HALF[x.dtype]).all()
    small = [torch.full((1000,), 1e-30, device="cuda"), torch.full((8,), 1e-40, device="cuda")]
    ys = [torch.empty_like(x) for x in small]
    check(small, ys, zm.clip_grads(small, 1e-36, out=ys), 1e-36)
    x = tensors([(100, F), (50, B)], 41)
    x[0][3] = math.inf
    y = [t.clone() for t in x]
    assert float(zm.clip_grads(y, 1.0)) == math.inf
    assert y[0][3].isnan() and not y[0][:3].any() and not y[0][4:].any() and not y[1].any()
    x[0][3] = math.nan
    y = [t.clone() for t in x]
    assert math.isnan(float(zm.clip_grads(y, 1.0))) and all(t.isnan().all() for t in y)


def test_no_tensors_and_the_norm_s_place():
    norm = torch.full((), 5.0, device="cuda")
    assert float(zm.clip_grads([], 1.0, norm=norm)) == 0.0
    assert float(zm.grad_norm([], norm=norm)) == 0.0
    with pytest.raises(zm.ZmError, match="no tensors"):
        zm.grad_norm([])
    x = torch.randn(64, device="cuda")
    for bad in (lambda: zm.clip_grads([x, x], 1.0), lambda: zm.clip_grads([x], 1.0, out=[x.view(-1)[:32]]),
                lambda: zm.clip_grads([x[:32]], 1.0, out=[x[16:48]]), lambda: zm.clip_grads([x], 1.0, norm=x[3]),
                lambda: zm.clip_grads([x], float("nan")), lambda: zm.clip_grads([x], -1.0),
                lambda: zm.clip_grads([x.view(8, 8).T], 1.0), lambda: zm.clip_grads([x.half()], 1.0),
                lambda: zm.clip_grads([x], 1.0, norm=torch.empty(2, device="cuda")),
                lambda: zm.clip_grads([x, x.cpu()], 1.0), lambda: zm.clip_grads(zm.TensorList([x]), 1.0, out=[x]),
                lambda: zm.clip_grads([x], 1.0, workspace=torch.empty(64, device="cuda"))):
        with pytest.raises(zm.ZmError):
            bad()
    assert not torch.equal(x, torch.zeros_like(x))


def test_a_captured_call_and_the_same_bits():
    sizes = [(1000 + i, B if i % 2 else F) for i in range(200)]
    xs = tensors(sizes, 42)
    keep = [x.clone() for x in xs]
    ys = [x.clone() for x in xs]
    base = float(zm.clip_grads(ys, 0.5))
    grads, norm = zm.TensorList(xs), torch.empty((), device="cuda")
    ws = torch.full((zm.grad_norm_workspace_size(200) // 4,), float("nan"), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        zm.clip_grads(grads, 0.5, norm=norm, workspace=ws)
    for _ in range(3):
        for x, k in zip(xs, keep):
            x.copy_(k)
        norm.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert float(norm) == base and all(torch.equal(x, y) for x, y in zip(xs, ys))
        zm.grad_norm(keep)
