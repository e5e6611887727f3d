"""zm.rotary against a plain fp64 rotation.

Tolerance: cos and sin come from an angle reduced in 64 bits and rounded to 32
(an error of at most pi 2^-24 where the reduced angle is largest) and are
themselves off by under 2 ulp, so each is off by less than 8 * 2^-24; two
products and a sum add 2^-24 each: 12 * 2^-24 (|x| + |y|), and the rounding to
bf16 2^-8 of the result."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def pair_dims(sections, layout):
    P, out, f = sum(sections), [], 0
    for a, s in enumerate(sections):
        for j in range(s):
            p = f + j
            out.append((a, p, *((p, p + P), (2 * p, 2 * p + 1), (2 * f + j, 2 * f + s + j))[layout]))
        f += s
    return out


def reference(x, pos, freqs, sections, layout, inverse):
    y = x.double().clone()
    tol = torch.zeros_like(y)
    for a, p, i, j in pair_dims(sections, layout):
        ang = pos[:, a].double() * freqs[p].double() * (-1.0 if inverse else 1.0)
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        u, v = x[..., i].double(), x[..., j].double()
        y[..., i], y[..., j] = u * c - v * s, u * s + v * c
        tol[..., i] = tol[..., j] = 12 * U * (u.abs() + v.abs())
    return y, tol + HALF[x.dtype] * y.abs() * 1.01 + 1e-37


def make(n, hq, hk, d, dtype, axes, seed, far=0, fractional=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    y = torch.randn((n, (hq + hk) * d + 24), generator=g, device="cuda").to(dtype)
    q, k = y[:, :hq * d].unflatten(1, (hq, d)), y[:, hq * d:(hq + hk) * d].unflatten(1, (max(hk, 1), -1))
    pos = torch.randint(-far if far else 0, far + 40, (n, axes), generator=g, device="cuda", dtype=torch.int32)
    if fractional:
        pos = pos.float() + torch.rand((n, axes), generator=g, device="cuda")
    return y, q, (k if hk else None), pos


CASES = [
    # n, hq, hk, d, sections
    (1, 1, 1, 64, (8, 12, 12)), (1374, 8, 8, 128, (16, 24, 24)), (33, 16, 4, 64, (8, 12, 8)),
    (7, 3, 1, 128, (5, 7, 11)), (129, 2, 0, 64, (32,)), (50, 4, 2, 8, (1, 1, 1, 1)), (40, 2, 2, 256, (64, 64)),
    (21, 1, 3, 96, (0, 16, 0)), (65, 64, 64, 16, (4, 0, 2)),
]


@pytest.mark.parametrize("layout", [0, 1, 2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_rotation(case, dtype, layout):
    n, hq, hk, d, sec = case
    print(f"case rotary {case} {dtype} layout={layout}", flush=True)
    for inverse, far, frac in ((False, 0, False), (True, 3_000_000, False), (False, 1000, True)):
        buf, q, k, pos = make(n, hq, hk, d, dtype, len(sec), 7 * n + d, far, frac)
        freqs = torch.rand(sum(sec), device="cuda") + 0.01
        whole = buf.clone()
        qo, ko = zm.rotary(q, k, pos, freqs, sec, layout=layout, inverse=inverse)
        assert torch.equal(buf, whole)
        for x, y in ((q, qo), (k, ko)):
            if x is None:
                assert y is None
                continue
            ref, tol = reference(x, pos, freqs, sec, layout, inverse)
            worst = ((y.double() - ref).abs() / tol).max().item()
            assert worst <= 1.0, f"{worst:.3g} of the tolerance"
            free = torch.ones(d, dtype=torch.bool, device="cuda")
            for _, _, i, j in pair_dims(sec, layout):
                free[i] = free[j] = False
            assert torch.equal(y[..., free], x[..., free])
        # in place on the projection's rows: the same bits, nothing beside them
        zm.rotary(q, k, pos, freqs, sec, layout=layout, inverse=inverse, q_out=q, k_out=k)
        assert torch.equal(q, qo) and (k is None or torch.equal(k, ko))
        assert torch.equal(buf[:, (hq + hk) * d:], whole[:, (hq + hk) * d:])


def test_special_tokens_are_unchanged_and_bad_positions_stay_in_their_axis():
    _, q, k, pos = make(12, 4, 4, 128, torch.bfloat16, 3, 5, fractional=True)
    pos[::2] = 0
    pos[1, 1] = float("inf")
    freqs = torch.rand(64, device="cuda")
    qo, ko = zm.rotary(q, k, pos, freqs, (16, 24, 24))
    assert torch.equal(qo[::2], q[::2]) and torch.equal(ko[::2], k[::2])
    bad = qo[1].isnan()
    want = torch.zeros(128, dtype=torch.bool, device="cuda")
    want[16:40] = want[80:104] = True
    assert torch.equal(bad, want.expand(4, 128))


def test_the_inverse_is_the_gradient():
    # <R x, w> has the gradient R^T w by x: the inverse rotation of w
    _, q, _, pos = make(40, 3, 0, 64, torch.float32, 3, 6)
    w = torch.randn_like(q.contiguous())
    freqs = torch.rand(28, device="cuda")
    for layout in (0, 1, 2):
        x = q.double().contiguous().requires_grad_()
        y = x.clone()
        for a, p, i, j in pair_dims((8, 12, 8), layout):
            ang = pos[:, a].double() * freqs[p].double()
            c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
            cols = torch.zeros_like(y)
            cols[..., i], cols[..., j] = 1, 1
            y = y * (1 - cols) + torch.nn.functional.one_hot(torch.tensor(i, device="cuda"), 64) * (
                x[..., i:i + 1] * c[..., None] - x[..., j:j + 1] * s[..., None]) + torch.nn.functional.one_hot(
                torch.tensor(j, device="cuda"), 64) * (x[..., i:i + 1] * s[..., None] + x[..., j:j + 1] * c[..., None])
        (y * w.double()).sum().backward()
        got, _ = zm.rotary(w, None, pos, freqs, (8, 12, 8), layout=layout, inverse=True)
        assert (got.double() - x.grad).abs().max() < 14 * U * 2 * w.abs().max()


def test_offsets_past_32_bits():
    # rows 2^24 elements apart: the last ones start past 2^31 elements
    n, ld = 140, 1 << 24
    buf = torch.empty(n * ld, dtype=torch.bfloat16, device="cuda")
    q = buf.as_strided((n, 2, 64), (ld, 64, 1))
    src = torch.randn(n, 2, 64, device="cuda").to(torch.bfloat16)
    q.copy_(src)
    pos = torch.arange(n, device="cuda", dtype=torch.int32)[:, None].contiguous()
    freqs = torch.rand(32, device="cuda")
    zm.rotary(q, None, pos, freqs, (32,), q_out=q)
    want, _ = zm.rotary(src, None, pos, freqs, (32,))
    assert torch.equal(q, want)


def test_no_tokens_and_graph_replays():
    empty = torch.empty((0, 2, 64), device="cuda")
    pos = torch.empty((0, 1), dtype=torch.int32, device="cuda")
    freqs = torch.rand(32, device="cuda")
    assert zm.rotary(empty, empty, pos, freqs, (32,))[0].shape == (0, 2, 64)
    q, k = torch.randn(300, 2, 64, device="cuda"), torch.randn(300, 2, 64, device="cuda")
    pos = torch.randint(0, 99, (300, 1), device="cuda", dtype=torch.int32)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    zm.rotary(q, k, pos, freqs, (32,), q_out=qo, k_out=ko)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        zm.rotary(q, k, pos, freqs, (32,), q_out=qo, k_out=ko)
    for _ in range(3):
        pos.random_(0, 1000)
        graph.replay()
        a, b = zm.rotary(q, k, pos, freqs, (32,))
        torch.cuda.synchronize()
        assert torch.equal(a, qo) and torch.equal(b, ko)
