"""The sequence operators together, as a layer uses them: layer norm of the tokens, one
projection to q, k, v (torch), the rotation of q and k where the projection left
them, the gated delta rule in frames with the state carried along and then by single
tokens; and the gradient back to the tokens, the norm's parameters and the
projection.  Compared with the same in 64 bits and its autograd.

Tolerance, of a tensor's 2-norm.  fp32: the norm adds at most 16 roundings of 2^-24,
the projection of 128 terms 128, the rotation 4: under 2^-16 on q, k and v.  The rule
reads q and v once and k twice, does not expand, and remembers for a few tokens only
(decays about 0.93, rates about 0.5: under 16), so an output moves by at most
4 * 16 * 2^-16 = 2^-10; the rule's own error is far below that.  A gradient goes
through the same again: 2^-9.  bf16: the norm's rows, the projection, the rotated
q and k and the outputs are rounded by at most 2^-8 each (2^-9 on average), 4 reads
of them: 4 * 4 * 2^-9 = 2^-5; the gradient rounds as many again: 2^-4."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm
from delta_reference import forward

pytestmark = pytest.mark.gpu

N, H, HK, D, W = 150, 4, 2, 64, 128
SECTIONS = (8, 12, 12)
CUTS = [0, 64, 101, 145]  # frames, then single tokens


def make(dtype):
    g = torch.Generator(device="cuda").manual_seed(77)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    pos = torch.randint(0, 50, (N, 3), generator=g, device="cuda", dtype=torch.int32)
    pos[::30] = 0  # special tokens
    return dict(x=(2 * normal(N, W) + 1).to(dtype), gamma=1 + 0.1 * normal(W), beta=0.1 * normal(W),
                proj=(normal((2 * HK + H) * D, W) * (W * D) ** -0.5).to(dtype), pos=pos,
                freqs=10.0 ** (-torch.arange(32, device="cuda") / 16.0), g=-0.1 * torch.nn.functional.softplus(normal(N, H)),
                rate=torch.sigmoid(normal(N, H)), do=normal(N, H, D).to(dtype), dend=normal(1, H, D, D) * D ** -0.5,
                state=normal(1, H, D, D) * D ** -0.5)


def split(rows):
    q, k, v = rows[:, :HK * D], rows[:, HK * D:2 * HK * D], rows[:, 2 * HK * D:]
    return q.unflatten(1, (HK, D)), k.unflatten(1, (HK, D)), v.unflatten(1, (H, D))


def run(p):
    stats = torch.empty((2, N), device="cuda")
    y = zm.layer_norm(p["x"], p["gamma"], p["beta"], stats=stats)
    rows = y @ p["proj"].t()
    q0, k0, v = split(rows)
    q, k = zm.rotary(q0, k0, p["pos"], p["freqs"], SECTIONS)
    state, outs = p["state"].clone(), []
    for a, e in zip(CUTS, CUTS[1:]):
        o, state = zm.delta_rule(q[a:e], k[a:e], v[a:e], p["g"][a:e], p["rate"][a:e], state=state, state_out=state)
        outs.append(o)
    for t in range(CUTS[-1], N):
        outs.append(zm.delta_rule_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], p["g"][t:t + 1], p["rate"][t:t + 1], state))
    return torch.cat(outs), state, (stats, y, q, k, v)


def run_backward(p, saved):
    stats, y, q, k, v = saved
    rows = torch.empty((N, (2 * HK + H) * D), dtype=p["x"].dtype, device="cuda")
    dq, dk, dv = split(rows)
    dg, drate = torch.empty_like(p["g"]), torch.empty_like(p["rate"])
    dstate = torch.empty_like(p["state"])
    zm.delta_rule_backward(p["do"], q, k, v, p["g"], p["rate"], state=p["state"], dstate=p["dend"],
                           out=(dq, dk, dv, dg, drate, dstate))
    zm.rotary(dq, dk, p["pos"], p["freqs"], SECTIONS, inverse=True, q_out=dq, k_out=dk)
    dproj = rows.t().contiguous() @ y
    dx, dgamma, dbeta = zm.layer_norm_backward(rows @ p["proj"], p["x"], stats, p["gamma"])
    return dict(x=dx, gamma=dgamma, beta=dbeta, proj=dproj, g=dg, rate=drate, state=dstate)


def reference(p):
    leaves = {k: p[k].double().requires_grad_() for k in ("x", "gamma", "beta", "proj", "g", "rate", "state")}
    x = leaves["x"]
    c = x - x.mean(1, keepdim=True)
    y = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-6) * leaves["gamma"] + leaves["beta"]
    q, k, v = split(y @ leaves["proj"].t())
    axis = torch.tensor([i for i, s in enumerate(SECTIONS) for _ in range(s)], device="cuda")
    ang = (p["pos"].double()[:, axis] * p["freqs"].double())[:, None]

    def turn(z):
        a, b = z[..., :32], z[..., 32:]
        return torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1)

    o, end, _ = forward(turn(q), turn(k), v, leaves["g"], leaves["rate"], leaves["state"])
    loss = (o * p["do"].double()).sum() + (end * p["dend"].double()).sum()
    names = list(leaves)
    return o.detach(), end.detach(), dict(zip(names, torch.autograd.grad(loss, [leaves[n] for n in names])))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_operators_together(dtype):
    print(f"case sequence block {dtype}", flush=True)
    p = make(dtype)
    o, state, saved = run(p)
    want_o, want_end, want = reference(p)
    tol = 2.0 ** -10 if dtype == torch.float32 else 2.0 ** -5
    for name, a, b in (("outputs", o, want_o), ("state", state, want_end)):
        err = (a.double() - b).norm() / b.norm()
        assert err <= tol, f"{name}: {err:.3g}"
    got = run_backward(p, saved)
    for name, b in want.items():
        err = (got[name].double() - b).norm() / b.norm()
        assert err <= 2 * tol, f"gradient of {name}: {err:.3g}"


def test_the_operators_together_in_a_graph():
    # one frame captured: the state moves on with every replay
    p = make(torch.bfloat16)
    off = slice(0, 101)
    stats = torch.empty((2, 101), device="cuda")
    y = torch.empty((101, W), dtype=torch.bfloat16, device="cuda")
    rows = torch.empty((101, (2 * HK + H) * D), dtype=torch.bfloat16, device="cuda")
    state = p["state"].clone()
    out = torch.empty((101, H, D), dtype=torch.bfloat16, device="cuda")

    def frame():
        zm.layer_norm(p["x"][off], p["gamma"], p["beta"], out=y, stats=stats)
        torch.mm(y, p["proj"].t(), out=rows)
        q, k, v = split(rows)
        zm.rotary(q, k, p["pos"][off], p["freqs"], SECTIONS, q_out=q, k_out=k)
        zm.delta_rule(q, k, v, p["g"][off], p["rate"][off], state=state, state_out=state, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        frame()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        frame()
    want = []
    state.copy_(p["state"])
    for _ in range(3):
        frame()
        want.append((out.clone(), state.clone()))
    state.copy_(p["state"])
    for a, b in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a) and torch.equal(state, b)
