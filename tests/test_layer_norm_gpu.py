"""zm.layer_norm and its backward against a plain fp64 form.

Tolerances.  A result rounded to bf16 is off by at most 2^-8 of its value
(fp32: 2^-24); what the kernel computes before that, in fp32, adds the error of
its sums.  A sum over a row is a chain of at most 32 adds in a lane, 6 across
the wave and 3 across waves, each off by 2^-24 of what it has, so mu is off by
at most 41 * 2^-24 mean|x| and r by half as much of itself plus the rounding of
its root and quotient: 64 * 2^-24 (r mean|x| + |xh| + 1) covers xh, and gamma
scales it.  The parameter gradients add n terms in chains of
ceil(n / slots / rows) + 3 and then ceil(slots / 16) + 16, each term off as
above: (chain + 64) * 2^-24 times the sum of the terms' sizes."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rows(n, width, ld, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, ld), generator=g, device="cuda") * scale + shift
    return x.to(dtype)[:, :width]


def params(width, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1 + 0.2 * torch.randn(width, generator=g, device="cuda"),
            0.3 * torch.randn(width, generator=g, device="cuda"))


def reference(x, eps):
    x = x.double()
    mu = x.mean(1, keepdim=True)
    r = 1 / torch.sqrt(((x - mu) ** 2).mean(1, keepdim=True) + eps)
    return mu, r, (x - mu) * r


def close(got, ref, tol, what):
    off = (got.double() - ref).abs()
    worst = (off / tol).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the tolerance"


SHAPES = [(1, 8), (3, 64), (5, 520), (1374, 1024), (7, 1032), (130, 2048), (9, 2056), (33, 4096), (5, 4104),
          (6, 8192), (2, 8184)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,width", SHAPES)
@pytest.mark.parametrize("affine", ["both", "gamma", "beta", "none"])
def test_forward(n, width, dtype, affine):
    print(f"case layer norm forward n={n} width={width} {dtype} {affine}", flush=True)
    x = rows(n, width, width + 8 * (n % 3), dtype, 11 * n + width, 2.0, 0.7)
    gamma, beta = params(width, 5)
    gamma = gamma if affine in ("both", "gamma") else None
    beta = beta if affine in ("both", "beta") else None
    stats = torch.full((2, n), float("nan"), device="cuda")
    y = zm.layer_norm(x, gamma, beta, eps=1e-5, stats=stats)
    mu, r, xh = reference(x, 1e-5)
    gd = gamma.double() if gamma is not None else 1.0
    ref = xh * gd + (beta.double() if beta is not None else 0.0)
    size = x.double().abs().mean(1, keepdim=True) * r
    fp32 = 64 * U * ((size + xh.abs() + 1) * (abs(gd) if gamma is None else gd.abs())
                     + (beta.double().abs() if beta is not None else 0.0))
    close(y, ref, fp32 + HALF[dtype] * ref.abs() * 1.01, "y")
    close(stats[0], mu[:, 0], 64 * U * x.double().abs().mean(1) + 1e-30, "mean")
    close(stats[1], r[:, 0], 64 * U * r[:, 0] * (1 + size[:, 0]), "rstd")
    again = zm.layer_norm(x, gamma, beta, eps=1e-5)
    assert torch.equal(again, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,width", SHAPES + [(20_011, 256)])
def test_backward(n, width, dtype):
    print(f"case layer norm backward n={n} width={width} {dtype}", flush=True)
    x = rows(n, width, width + 16, dtype, 3 * n + width, 1.5, -0.4)
    dy = rows(n, width, width + 8, dtype, 3 * n + width + 1)
    gamma, _ = params(width, 6)
    mu, r, _ = reference(x, 1e-6)
    stats = torch.cat([mu, r], 1).T.float().contiguous()
    dx, dgamma, dbeta = zm.layer_norm_backward(dy, x, stats, gamma)
    m, r = stats.double()[0][:, None], stats.double()[1][:, None]
    xh, d = (x.double() - m) * r, dy.double()
    a = d * gamma.double()
    ma, mx = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    ref = r * (a - ma - xh * mx)
    fp32 = 64 * U * r * (a.abs() + a.abs().mean(1, keepdim=True)
                         + (xh.abs() + 1) * (a * xh).abs().mean(1, keepdim=True))
    close(dx, ref, fp32 + HALF[dtype] * ref.abs() * 1.01, "dx")
    chain = n / 64 + 96
    close(dgamma, (d * xh).sum(0), (chain + 64) * U * ((d * xh).abs().sum(0) + (r * m.abs() * d.abs()).sum(0)), "dgamma")
    close(dbeta, d.sum(0), chain * U * d.abs().sum(0) + 1e-30, "dbeta")
    # the same bits again, and in place of dy and of x
    for target in (dy.clone(), x.clone()):
        t2 = target if target.stride(1) == 1 else target.contiguous()
        other = zm.layer_norm_backward(t2, x, stats, gamma, out=t2) if torch.equal(t2, dy) else \
            zm.layer_norm_backward(dy, t2, stats, gamma, out=t2)
        assert all(torch.equal(p, q) for p, q in zip(other, (dx, dgamma, dbeta)))


def test_backward_against_differences():
    x = rows(3, 24, 24, torch.float32, 1).double()
    gamma, beta = params(24, 2)
    w = rows(3, 24, 24, torch.float32, 3)

    def loss(x, gamma, beta):
        _, _, xh = reference(x, 1e-6)
        return ((xh * gamma + beta) * w.double()).sum()

    stats = torch.empty(2, 3, device="cuda")
    zm.layer_norm(x.float(), gamma, beta, stats=stats)
    dx, dgamma, dbeta = zm.layer_norm_backward(w, x.float(), stats, gamma)
    x, h = x.float().double(), 1e-6
    for t, grad in ((x, dx), (gamma.double(), dgamma), (beta.double(), dbeta)):
        flat = t.reshape(-1)
        for i in range(0, flat.numel(), 5):
            vals = []
            for s in (h, -h):
                p = flat.clone()
                p[i] += s
                p = p.view_as(t)
                vals.append(loss(p if t is x else x, p if grad is dgamma else gamma.double(),
                                 p if grad is dbeta else beta.double()))
            # central differences of step h: third derivatives times h^2 and 2^-52 / h
            # of the loss (about 30) are both under 1e-7
            assert abs(((vals[0] - vals[1]) / (2 * h) - grad.reshape(-1)[i].double()).item()) < 2e-5


def test_in_place_and_padding_is_left_alone():
    buf = torch.randn(37, 1104, device="cuda").to(torch.bfloat16)
    whole = buf.clone()
    x = buf[:, :1032]
    y = zm.layer_norm(x.clone())
    zm.layer_norm(x, out=x)
    assert torch.equal(x, y) and torch.equal(buf[:, 1032:], whole[:, 1032:])


def test_constant_rows_and_non_finite_rows():
    x = torch.full((4, 512), 3.0, device="cuda")
    x[1, 7] = float("nan")
    x[2, 3] = float("inf")
    y = zm.layer_norm(x)
    assert torch.equal(y[0], torch.zeros(512, device="cuda")) and torch.equal(y[3], y[0])
    assert y[1].isnan().all() and y[2].isnan().all()
    # a mean far from zero: the distances to it decide
    far = 4096.0 + torch.randn(8, 1024, device="cuda")
    y, (_, _, xh) = zm.layer_norm(far), reference(far, 1e-6)
    close(y, xh, 64 * U * (4100.0 + xh.abs()), "far mean")


def test_no_rows():
    x = torch.empty((0, 64), device="cuda")
    stats = torch.empty((2, 0), device="cuda")
    assert zm.layer_norm(x, stats=stats).shape == (0, 64)
    dx, dgamma, dbeta = zm.layer_norm_backward(x, x, stats)
    assert dx.shape == (0, 64) and not dgamma.any() and not dbeta.any()


def test_side_stream_and_graph_replays():
    x = rows(700, 1024, 1024, torch.bfloat16, 8)
    dy = rows(700, 1024, 1024, torch.bfloat16, 9)
    gamma, beta = params(1024, 10)
    stats = torch.empty((2, 700), device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dg, db = torch.empty(1024, device="cuda"), torch.empty(1024, device="cuda")
    ws = torch.empty(zm.layer_norm_backward_workspace_size(700, 1024), dtype=torch.uint8, device="cuda")

    def both():
        zm.layer_norm(x, gamma, beta, out=y, stats=stats)
        zm.layer_norm_backward(dy, x, stats, gamma, out=dx, dgamma=dg, dbeta=db, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in range(3):
        x.copy_(rows(700, 1024, 1024, torch.bfloat16, 20 + seed))
        graph.replay()
        got = [t.clone() for t in (y, stats, dx, dg, db)]
        both()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, (y, stats, dx, dg, db)))
