"""Linear attention with decays and its gradient token by token in 64 bits, without the
chunks: what the kernels' tests compare with.

Tolerances.  Every result is a sum of products of tokens, states, decays and the scale.  The
same call on absolute values gives the sum of its terms' sizes, A.  A product of three-part
operands leaves out parts under 2^-24, a decay factor is off by a few 2^-24 (exp2 of the rest
after the whole part, twice, and their product), and a sum of a chunk (at most 18 matrix
instructions of 32 products, their own rounding about three steps each) by at most 54: 64 steps
of 2^-24 of A allowed, for each chunk that a term passes through and two more (the chunk's
own products and the join of segments).  On top comes the output's rounding, half a step of itself.
Outputs o in bf16 take states and triangles in two parts, each rounded to the nearest.  x = hi + r
with |r| <= 2^-8 |x|, r = lo + e with |e| <= 2^-8 |r|: a term is off by at most 2^-16 of its size, so the
sum by at most 2^-16 of A (ROUGH)."""
import torch

STEP = 2.0 ** -24
ROUGH = {torch.bfloat16: 2.0 ** -16, torch.float32: 0.0}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def inputs(n, heads, heads_k, d, dtype, seed, n_seq=1, decay=0.1, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=device)

    return dict(q=normal(n, heads_k, d).to(dtype), k=normal(n, heads_k, d).to(dtype), v=normal(n, heads, d).to(dtype),
                g=-decay * torch.nn.functional.softplus(normal(n, heads)), state=normal(n_seq, heads, d, d))


def forward(q, k, v, g, state, offsets=None, scale=None):
    """(o, end states), fp64."""
    n, hk, d = q.shape
    h, rep = v.shape[1], v.shape[1] // hk
    scale = d ** -0.5 if scale is None else scale
    offsets = [0, n] if offsets is None else offsets
    q, k = (x.double().repeat_interleave(rep, 1) for x in (q, k))
    v = v.double()
    a = torch.ones((n, h), dtype=torch.float64, device=q.device) if g is None else torch.exp(g.double()).expand(n, h)
    o, ends = [torch.zeros_like(v[:offsets[0]])], []
    for b in range(len(offsets) - 1):
        S = state[b].double() if state is not None else torch.zeros(h, d, d, dtype=torch.float64, device=q.device)
        for t in range(offsets[b], offsets[b + 1]):
            S = S * a[t][:, None, None] + v[t][..., None] * k[t][:, None]
            o.append(scale * (S * q[t][:, None]).sum(-1)[None])
        ends.append(S)
    o.append(torch.zeros_like(v[offsets[-1]:]))
    return torch.cat(o), torch.stack(ends) if ends else torch.zeros((0, h, d, d), dtype=torch.float64, device=q.device)


def gradient(do, q, k, v, g, state, dstate, offsets=None, scale=None):
    """Gradients by q, k, v, g (None without) and the first states, by autograd of the recurrence."""
    n, hk, d = q.shape
    n_seq = 1 if offsets is None else len(offsets) - 1
    first = state if state is not None else torch.zeros(n_seq, v.shape[1], d, d, device=q.device)
    leaves = [None if x is None else x.double().requires_grad_() for x in (q, k, v, g, first)]
    o, ends = forward(*leaves, offsets, scale)
    loss = (o * do.double()).sum()
    if dstate is not None:
        loss = loss + (ends * dstate.double()).sum()
    got = iter(torch.autograd.grad(loss, [x for x in leaves if x is not None], allow_unused=True))
    out = []
    for x in leaves:
        y = None if x is None else next(got)
        out.append(torch.zeros_like(x) if x is not None and y is None else y)
    return out


def sizes(x, names):
    """The inputs with absolute values in the place of `names`."""
    return [None if x[name] is None else x[name].abs() if name in names else x[name] for name in x]


def chunks(n, dtype):
    return -(-n // (32 if dtype == torch.float32 else 64))


def check(name, got, want, size, steps, rough=0.0):
    """|got - want| within steps * 2^-24 of size (and `rough` of it) and the output's own rounding."""
    tol = (64 * steps * STEP + rough) * size + HALF[got.dtype] * 1.01 * want.abs() + 1e-300
    off = (got.double() - want).abs()
    assert (off <= tol).all(), f"{name}: {(off / tol).max().item():.3g} of the tolerance"
