"""The gated delta rule and its gradient token by token in 64 bits, without the
chunks: what the kernels' tests compare with."""
import torch


def inputs(n, heads, heads_k, d, dtype, seed, n_seq=1, decay=0.1, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=device)

    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    return dict(q=unit(normal(n, heads_k, d)).to(dtype), k=unit(normal(n, heads_k, d)).to(dtype),
                v=normal(n, heads, d).to(dtype), g=-decay * torch.nn.functional.softplus(normal(n, heads)),
                beta=torch.sigmoid(normal(n, heads)), state=normal(n_seq, heads, d, d) * d ** -0.5)


def forward(q, k, v, g, beta, state, offsets=None, scale=None):
    """(o, end states, the largest Frobenius norm each state had), fp64."""
    n, hk, d = q.shape
    h, rep = v.shape[1], v.shape[1] // hk
    scale = d ** -0.5 if scale is None else scale
    offsets = [0, n] if offsets is None else offsets
    q, k = (x.double().repeat_interleave(rep, 1) for x in (q, k))
    v, a, beta = v.double(), torch.exp(g.double()), beta.double()
    o, ends, tops = torch.zeros_like(v), [], []
    for b in range(len(offsets) - 1):
        S = state[b].double().clone() if state is not None else torch.zeros(h, d, d, dtype=torch.float64,
                                                                           device=q.device)
        top = S.norm(dim=(1, 2))
        for t in range(offsets[b], offsets[b + 1]):
            S = S * a[t][:, None, None]
            u = beta[t][:, None] * (v[t] - (S * k[t][:, None]).sum(-1))
            S = S + u[..., None] * k[t][:, None]
            o[t] = scale * (S * q[t][:, None]).sum(-1)
            top = torch.maximum(top, S.norm(dim=(1, 2)))
        ends.append(S)
        tops.append(top)
    empty = torch.zeros((0, h, d, d), dtype=torch.float64, device=q.device)
    return o, torch.stack(ends) if ends else empty, torch.stack(tops) if tops else empty[..., 0, 0]


def gradient(do, q, k, v, g, beta, state, dstate, offsets=None, scale=None):
    """Gradients by q, k, v, g, beta and the first states, by autograd of the recurrence."""
    leaves = [x.double().requires_grad_() for x in (q, k, v, g, beta)]
    n, hk, d = q.shape
    h, rep = v.shape[1], v.shape[1] // hk
    scale = d ** -0.5 if scale is None else scale
    offsets = [0, n] if offsets is None else offsets
    first = (state.double() if state is not None else
             torch.zeros(len(offsets) - 1, h, d, d, dtype=torch.float64, device=q.device)).requires_grad_()
    qd, kd = (x.repeat_interleave(rep, 1) for x in leaves[:2])
    vd, ad, bd = leaves[2], torch.exp(leaves[3]), leaves[4]
    loss = 0.0
    for b in range(len(offsets) - 1):
        S = first[b]
        for t in range(offsets[b], offsets[b + 1]):
            S = S * ad[t][:, None, None]
            u = bd[t][:, None] * (vd[t] - (S * kd[t][:, None]).sum(-1))
            S = S + u[..., None] * kd[t][:, None]
            loss = loss + (scale * (S * qd[t][:, None]).sum(-1) * do[t].double()).sum()
        if dstate is not None:
            loss = loss + (S * dstate[b].double()).sum()
    got = torch.autograd.grad(loss, leaves + [first], allow_unused=True)
    return [x if x is not None else torch.zeros_like(l) for x, l in zip(got, leaves + [first])]
