"""Timing cases of the layer norm, the multi-axis rotary rotation and the gated delta rule.

Each case runs one operator in its plain form (own = False: elementary torch
operations in 32 bits, angles in 64) or through the package (own = True).
Frames have 37 * 37 + 5 = 1374 tokens and the model width is 1024 = 8 heads of
128, as in workloads.py.
"""
import math

import torch

own = False

FRAME = 1374
CHUNK = 64
HALVES, PAIRS, AXIS_HALVES = 0, 1, 2


def listed():
    norm = dict(op="norm", n=FRAME, width=1024, dtype="bf16", ld=1024, backward=False)
    rot = dict(op="rotary", n=FRAME, heads=8, heads_k=8, d=128, dtype="bf16", s0=16, s1=24, s2=24,
               layout=HALVES, inverse=False, far=0, fused=True)
    delta = dict(op="delta", n=FRAME, n_seq=1, heads=8, heads_k=8, d=128, dtype="bf16", mode="forward")
    return [
        # the tokens of one streamed frame, normalised before the projections
        dict(norm, name="norm_frame"),
        # fp32 tokens in padded rows, an odd count of them
        dict(norm, name="norm_f32_rows", n=40_001, width=2048, ld=2056, dtype="f32"),
        # the gradient over the tokens of 100 frames
        dict(norm, name="norm_backward_100_frames", n=100 * FRAME, backward=True),
        # q and k of one frame, rotated where the fused projection left them
        dict(rot, name="rotary_frame"),
        # the gradient's rotation of 40 frames of fp32 tokens, grouped heads, far and fractional positions
        dict(rot, name="rotary_inverse_f32", n=40 * FRAME, heads=16, heads_k=4, d=64, dtype="f32", s0=8, s1=12,
             s2=8, layout=PAIRS, inverse=True, far=1_000_000, fused=False),
        # one token of one sequence: what a serving step waits for
        dict(delta, name="delta_step_1", n=1, n_seq=1, mode="step"),
        # one token of each of 256 sequences: bound by the states' memory traffic
        dict(delta, name="delta_step_256", n=256, n_seq=256, mode="step"),
        # 4 short fp32 sequences of one narrow head (frames of 70 x 70 pixels)
        dict(delta, name="delta_tiny_f32", n=120, n_seq=4, heads=1, heads_k=1, d=64, dtype="f32"),
        # one streamed frame with the state carried along
        dict(delta, name="delta_frame"),
        # a packed batch of ragged sequences, query/key heads shared by four value heads
        dict(delta, name="delta_packed", n=54_321, n_seq=61, heads=16, heads_k=4),
        # 100 frames as one long sequence: few heads, a long axis
        dict(delta, name="delta_100_frames", n=100 * FRAME),
        # the gradient of 8 sequences of about a frame each
        dict(delta, name="delta_backward_8_frames", n=8 * FRAME, n_seq=8, mode="backward"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rotary", "step", "delta", "delta", "backward"])
    dtype = "f32" if rng.random() < 0.3 else "bf16"
    if op == "norm":
        width = 8 * _log(rng, 8, 512)
        n = _log(rng, 1, max(2, 100 * FRAME * 1024 // (width * (2 if dtype == "f32" else 1))))
        return dict(op="norm", n=n, width=width, dtype=dtype, ld=width + 8 * rng.randrange(3),
                    backward=rng.random() < 0.5)
    d = rng.choice([64, 128])
    if op == "rotary":
        layout = rng.choice([HALVES, PAIRS, AXIS_HALVES])
        s = [rng.randrange(0, d // 6) + 1 for _ in range(3)]
        if rng.random() < 0.5:  # a whole rotation of 8-pair sections
            s = [d // 8, 3 * d // 16, 3 * d // 16]
        group = rng.choice([1, 1, 2, 4])
        heads_k = rng.choice([1, 2, 4])
        n = _log(rng, 1, 60 * FRAME * 8 * 128 // (heads_k * group * d * (2 if dtype == "f32" else 1)))
        return dict(op="rotary", n=min(n, 100 * FRAME), heads=heads_k * group, heads_k=heads_k, d=d, dtype=dtype,
                    s0=s[0], s1=s[1], s2=s[2], layout=layout, inverse=rng.random() < 0.5,
                    far=rng.choice([0, 0, 1_000_000]), fused=rng.random() < 0.5)
    heads_k = rng.choice([1, 2, 4, 8])
    heads = heads_k * rng.choice([1, 1, 2, 3])
    case = dict(op="delta", n=0, n_seq=0, heads=heads, heads_k=heads_k, d=d, dtype=dtype, mode=op)
    if op == "step":
        case["n"] = case["n_seq"] = _log(rng, 1, 4096 // heads)
        return case
    case["mode"] = "forward" if op == "delta" else "backward"
    case["n_seq"] = _log(rng, 1, 64)
    most = (60 if op == "delta" else 8) * FRAME * 8 * 128 // (heads * d * (2 if dtype == "f32" else 1))
    case["n"] = _log(rng, 1, max(2, min(most, 60 * FRAME)))
    return case


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _rows(n, width, ld, dtype, gen, scale=1.0, shift=0.0):
    """[n, width] normal values in rows of stride ld."""
    x = torch.randn((n, ld), generator=gen, device="cuda").mul_(scale).add_(shift)
    return x.to(dtype)[:, :width]


def _lengths(case, seed):
    """n tokens cut into n_seq ragged sequences (some may be empty), none over four times the mean."""
    n, b = case["n"], case["n_seq"]
    if case["mode"] == "step":
        return [1] * b
    g = torch.Generator().manual_seed(seed + 1)
    w = torch.rand(b, generator=g).add_(0.35)
    ends = (torch.cumsum(w, 0) / w.sum() * n).round().long().tolist()
    ends[-1] = n
    return [b - a for a, b in zip([0] + ends[:-1], ends)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, n = _dtype(case), case["n"]
    s = {"case": dict(case)}
    if case["op"] == "norm":
        w = case["width"]
        s["x"] = _rows(n, w, case["ld"], dtype, gen, 1.5, 0.3)
        s["gamma"] = torch.randn(w, generator=gen, device="cuda").mul_(0.1).add_(1.0)
        s["beta"] = torch.randn(w, generator=gen, device="cuda").mul_(0.1)
        s["eps"] = 1e-6
        if case["backward"]:
            s["dy"] = _rows(n, w, case["ld"], dtype, gen)
            xf = s["x"].double()
            mean = xf.mean(1)
            s["stats"] = torch.stack([mean, 1 / torch.sqrt(xf.var(1, unbiased=False) + s["eps"])]).float()
        return s
    H, HK, d = case["heads"], case["heads_k"], case["d"]
    if case["op"] == "rotary":
        if case["fused"]:  # q and k where the projection of [q | k | v | rate] left them
            y = _rows(n, (H + HK) * d, (H + 2 * HK) * d + H + (-H) % 8, dtype, gen)
            s["q"], s["k"] = y[:, :H * d].unflatten(1, (H, d)), y[:, H * d:].unflatten(1, (HK, d))
        else:
            s["q"] = torch.randn((n, H, d), generator=gen, device="cuda").to(dtype)
            s["k"] = torch.randn((n, HK, d), generator=gen, device="cuda").to(dtype)
        i = torch.arange(n, device="cuda")
        t, p = i // FRAME, i % FRAME - 5
        grid = [t, torch.where(p < 0, 0, p // 37 + 1), torch.where(p < 0, 0, p % 37 + 1)]
        pos = torch.stack(grid, 1).to(torch.int32)
        if case["far"]:
            pos = (pos + torch.rand((n, 3), generator=gen, device="cuda") * case["far"]).float()
        s["pos"] = pos.contiguous()
        s["sections"] = (case["s0"], case["s1"], case["s2"])
        s["freqs"] = torch.cat([100.0 ** (-torch.arange(c, dtype=torch.float64) / c) for c in s["sections"]]
                               ).float().cuda()
        return s
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    s["q"] = unit(torch.randn((n, HK, d), generator=gen, device="cuda")).to(dtype)
    s["k"] = unit(torch.randn((n, HK, d), generator=gen, device="cuda")).to(dtype)
    s["v"] = torch.randn((n, H, d), generator=gen, device="cuda").to(dtype)
    # decays from a few tokens to some thousand, by head
    rate = torch.exp(torch.empty(H, device="cuda").uniform_(math.log(1e-3), 0.0, generator=gen))
    z = torch.randn((n, H), generator=gen, device="cuda")
    s["g"] = -rate * torch.log1p(torch.exp(z - 1.0))
    s["beta"] = torch.sigmoid(torch.randn((n, H), generator=gen, device="cuda"))
    s["state"] = torch.randn((case["n_seq"], H, d, d), generator=gen, device="cuda").mul_(d ** -0.5)
    s["scale"] = d ** -0.5
    lens = _lengths(case, seed)
    at = [0]
    for c in lens:
        at.append(at[-1] + c)
    s["offsets"] = torch.tensor(at, dtype=torch.int32, device="cuda")
    # the padded form's plan: sequence b's token j, or n where it has none
    L = max(max(lens), 1)
    L = L if case["mode"] == "step" else -(-L // CHUNK) * CHUNK
    j = torch.arange(L, device="cuda")[None]
    lens, start = torch.tensor(lens, device="cuda")[:, None], s["offsets"][:-1, None].long()
    s["index"] = torch.where(j < lens, start + j, n)
    if case["mode"] == "backward":
        s["do"] = torch.randn((n, H, d), generator=gen, device="cuda").to(dtype)
        s["dstate"] = torch.randn((case["n_seq"], H, d, d), generator=gen, device="cuda").mul_(d ** -0.5)
    return s


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "norm":
        return _norm_backward(state) if case["backward"] else _norm(state)
    if case["op"] == "rotary":
        return _rotary(state, case)
    if case["mode"] == "step":
        return _delta_step(state, case)
    return _delta_backward(state, case) if case["mode"] == "backward" else _delta(state, case)


def _run_own(s, case):
    import reconstruction_lact_chunk_amd as zm

    if case["op"] == "norm":
        if case["backward"]:
            dx, dgamma, dbeta = zm.layer_norm_backward(s["dy"], s["x"], s["stats"], s["gamma"])
            return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
        stats = torch.empty((2, s["x"].shape[0]), device="cuda")
        y = zm.layer_norm(s["x"], s["gamma"], s["beta"], eps=s["eps"], stats=stats)
        return {"y": y, "stats": stats}
    if case["op"] == "rotary":
        q, k = zm.rotary(s["q"], s["k"], s["pos"], s["freqs"], s["sections"], layout=case["layout"],
                         inverse=case["inverse"])
        return {"q": q, "k": k}
    a = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    if case["mode"] == "step":
        o = zm.delta_rule_step(*a, s["state"], scale=s["scale"])
        return {"o": o, "state": s["state"]}
    if case["mode"] == "backward":
        dq, dk, dv, dg, dbeta, dstate = zm.delta_rule_backward(s["do"], *a, state=s["state"], dstate=s["dstate"],
                                                               offsets=s["offsets"], scale=s["scale"])
        return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta, "dstate": dstate}
    o, end = zm.delta_rule(*a, state=s["state"], offsets=s["offsets"], scale=s["scale"])
    return {"o": o, "state": end}


# ---- plain forms ------------------------------------------------------------
def _norm(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / torch.sqrt(c.square().mean(1) + s["eps"])
    y = c * rstd[:, None] * s["gamma"] + s["beta"]
    return {"y": y.to(s["x"].dtype), "stats": torch.stack([mean, rstd])}


def _norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    xh = (x - s["stats"][0][:, None]) * s["stats"][1][:, None]
    a = dy * s["gamma"]
    dx = (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True)) * s["stats"][1][:, None]
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}


def _pair_dims(case):
    """The two dims of each pair."""
    sec = (case["s0"], case["s1"], case["s2"])
    P = sum(sec)
    p = torch.arange(P, device="cuda")
    if case["layout"] == HALVES:
        return p, p + P
    if case["layout"] == PAIRS:
        return 2 * p, 2 * p + 1
    off = torch.tensor([0, sec[0], sec[0] + sec[1]], device="cuda")
    size = torch.tensor(sec, device="cuda")
    ax = (p >= sec[0]).long() + (p >= sec[0] + sec[1]).long()
    first = p + off[ax]
    return first, first + size[ax]


def _rotary(s, case):
    sec = s["sections"]
    ax = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(sec, device="cuda"),
                                 output_size=sum(sec))
    angle = s["pos"].double()[:, ax] * s["freqs"].double()
    c, sn = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if case["inverse"]:
        sn = -sn
    i, j = _pair_dims(case)

    def turn(x):
        xf = x.float()
        a, b = xf[..., i], xf[..., j]
        y = xf.clone()
        y[..., i] = a * c - b * sn
        y[..., j] = a * sn + b * c
        return y.to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _delta_step(s, case):
    rep = case["heads"] // case["heads_k"]
    q, k = (s[x].float().repeat_interleave(rep, 1)[:, :, None] for x in ("q", "k"))
    v = s["v"].float()
    S = s["state"].mul_(torch.exp(s["g"])[:, :, None, None])
    u = s["beta"][..., None] * (v - (S * k).sum(-1))
    S.add_(u[..., None] * k)
    return {"o": ((S * q).sum(-1) * s["scale"]).to(s["v"].dtype), "state": S}


def _padded(x, index):
    """x [n, H, ...] as [b, H, chunks, CHUNK, ...] in 32 bits, zeros where a sequence has no token."""
    x = torch.cat([x.float(), x.new_zeros((1,) + x.shape[1:]).float()])[index]
    return x.transpose(1, 2).unflatten(2, (-1, CHUNK)).contiguous()


def _back(x, s, dtype):
    """The inverse of _padded."""
    y = x.new_zeros((s["v"].shape[0] + 1, x.shape[1]) + x.shape[4:])
    y[s["index"]] = x.flatten(2, 3).transpose(1, 2)
    return y[:-1].to(dtype)


def _t(x):
    return x.transpose(-1, -2).contiguous()


def _chunk_parts(s, case):
    """What a chunk's equations need that does not depend on the state."""
    rep = case["heads"] // case["heads_k"]
    f = {x: _padded(s[x], s["index"]) for x in ("q", "k", "v", "g", "beta")}
    q, k = (f[x].repeat_interleave(rep, 1) for x in ("q", "k"))
    q = q * s["scale"]
    c = torch.cumsum(f["g"].double(), -1)
    low = torch.ones(CHUNK, CHUNK, device="cuda", dtype=torch.bool).tril()
    G = torch.exp((c[..., :, None] - c[..., None, :]).masked_fill(~low, -math.inf)).float()
    kk = torch.matmul(k, _t(k)) * G
    A = (kk * f["beta"][..., None]).tril(-1)
    T = torch.zeros_like(A)
    T[..., 0, 0] = 1
    for i in range(1, CHUNK):
        T[..., i, :i] = -torch.matmul(A[..., i:i + 1, :i], T[..., :i, :i])[..., 0, :]
        T[..., i, i] = 1
    gam, dec = torch.exp(c).float()[..., None], torch.exp(c[..., -1:] - c).float()[..., None]
    P = torch.matmul(q, _t(k)) * G
    return dict(q=q, k=k, v=f["v"], beta=f["beta"][..., None], G=G, kk=kk, T=T, P=P, gam=gam, dec=dec,
                kd=_t(k * dec), last=gam[..., -1:, :])


def _scan(p, M):
    """The chunks in order; the outputs, each chunk's U and first state, and the last state."""
    o, us, ms = [], [], []
    for c in range(p["k"].shape[2]):
        ms.append(M)
        R = p["v"][:, :, c] - p["gam"][:, :, c] * torch.matmul(p["k"][:, :, c], M)
        U = torch.matmul(p["T"][:, :, c], p["beta"][:, :, c] * R)
        o.append(p["gam"][:, :, c] * torch.matmul(p["q"][:, :, c], M) + torch.matmul(p["P"][:, :, c], U))
        M = p["last"][:, :, c] * M + torch.matmul(p["kd"][:, :, c], U)
        us.append(U)
    return torch.stack(o, 2), torch.stack(us, 2), ms, M


def _delta(s, case):
    o, _, _, M = _scan(_chunk_parts(s, case), _t(s["state"]))
    return {"o": _back(o, s, s["v"].dtype), "state": _t(M)}


def _delta_backward(s, case):
    p = _chunk_parts(s, case)
    _, U, ms, _ = _scan(p, _t(s["state"]))
    do = _padded(s["do"], s["index"])
    D = _t(s["dstate"])
    Pt, Tt, qt, kt = _t(p["P"]), _t(p["T"]), _t(p["q"]), _t(p["k"])
    dX, ds = [], []
    for c in reversed(range(len(ms))):
        ds.append(D)
        dU = torch.matmul(Pt[:, :, c], do[:, :, c]) + p["dec"][:, :, c] * torch.matmul(p["k"][:, :, c], D)
        dX.append(torch.matmul(Tt[:, :, c], dU))
        g = p["gam"][:, :, c]
        D = (p["last"][:, :, c] * D + torch.matmul(qt[:, :, c], g * do[:, :, c])
             - torch.matmul(kt[:, :, c], g * p["beta"][:, :, c] * dX[-1]))
    dX, D1, M0 = torch.stack(dX[::-1], 2), torch.stack(ds[::-1], 2), torch.stack(ms, 2)
    dR = p["beta"] * dX
    Ut, Mt = _t(U), _t(M0)
    doM, dXM = p["gam"] * torch.matmul(do, Mt), p["gam"] * torch.matmul(dX, Mt)
    UD = p["dec"] * torch.matmul(U, _t(D1))
    dP, XU = torch.matmul(do, Ut), torch.matmul(dX, Ut)
    W = dP * p["G"]
    E = -(XU * p["G"] * p["beta"]).tril(-1)
    dq = doM + torch.matmul(W, p["k"])
    dk = -p["beta"] * dXM + torch.matmul(_t(W), p["q"]) + UD + torch.matmul(E, p["k"]) + torch.matmul(_t(E), p["k"])
    dbeta = (dX * p["v"]).sum(-1) - (dXM * p["k"]).sum(-1) - (XU * p["kk"]).tril(-1).sum(-1)
    # derivatives by the decay's running sum
    pp, ee = dP * p["P"], (E * torch.matmul(p["k"], kt))
    dec = (UD * p["k"]).sum(-1)
    dc = ((doM * p["q"]).sum(-1) - (p["beta"] * dXM * p["k"]).sum(-1) + pp.sum(-1) - pp.sum(-2)
          + ee.sum(-1) - ee.sum(-2) - dec)
    dc[..., -1] += dec.sum(-1) + p["last"][..., 0, 0] * (M0 * D1).sum((-1, -2))
    dg = torch.flip(torch.cumsum(torch.flip(dc, (-1,)), -1), (-1,))
    dq = dq * s["scale"]
    rep, HK = case["heads"] // case["heads_k"], case["heads_k"]
    dq, dk = (x.unflatten(1, (HK, rep)).sum(2) for x in (dq, dk))
    t = s["v"].dtype
    return {"dq": _back(dq, s, t), "dk": _back(dk, s, t), "dv": _back(dR, s, t), "dg": _back(dg, s, torch.float32),
            "dbeta": _back(dbeta, s, torch.float32), "dstate": _t(D)}


# ---- what one pass cannot do without ---------------------------------------
def work(case):
    size, n = 2 if case["dtype"] == "bf16" else 4, case["n"]
    if case["op"] == "norm":
        e = n * case["width"]
        return {"bytes": e * size * (3 if case["backward"] else 2) + 8 * n + 8 * case["width"],
                "flops": e * (14 if case["backward"] else 8)}
    H, HK, d = case["heads"], case["heads_k"], case["d"]
    if case["op"] == "rotary":
        pairs = case["s0"] + case["s1"] + case["s2"]
        return {"bytes": 2 * n * (H + HK) * d * size + 12 * n, "flops": 6 * n * (H + HK) * pairs}
    states = case["n_seq"] * H * d * d * 4
    tokens = n * d * size
    if case["mode"] == "backward":
        return {"bytes": tokens * (4 * HK + 3 * H) + 16 * n * H + 3 * states, "flops": 16 * n * H * d * d}
    return {"bytes": tokens * (2 * HK + 2 * H) + 8 * n * H + 2 * states, "flops": 6 * n * H * d * d}


# ---- the definitions in 64 bits -----------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    if case["op"] == "rotary":
        return _exact_rotary(s, case)
    return _exact_delta(s, case)


def _exact_norm(s, case):
    x = s["x"].double()
    mu = x.sum(1, keepdim=True) / case["width"]
    if not case["backward"]:
        var = ((x - mu) ** 2).sum(1, keepdim=True) / case["width"]
        r = (var + s["eps"]) ** -0.5
        return {"y": (x - mu) * r * s["gamma"].double() + s["beta"].double(), "stats": torch.cat([mu, r], 1).T}
    mu, r = s["stats"].double()[0][:, None], s["stats"].double()[1][:, None]
    dy, w = s["dy"].double(), case["width"]
    h = (x - mu) * r
    a = dy * s["gamma"].double()
    dot, total = (a * h).sum(1, keepdim=True), a.sum(1, keepdim=True)
    return {"dx": r / w * (w * a - total - h * dot), "dgamma": torch.einsum("nw,nw->w", dy, h), "dbeta": dy.sum(0)}


def _exact_rotary(s, case):
    sign = -1.0 if case["inverse"] else 1.0
    P = sum(s["sections"])
    ends = [case["s0"], case["s0"] + case["s1"], P]
    out = {x: s[x].double() for x in ("q", "k")}
    for p in range(P):
        a = 0 if p < ends[0] else 1 if p < ends[1] else 2
        begin = ends[a] - s["sections"][a]
        i, j = ((p, p + P), (2 * p, 2 * p + 1), (begin + p, begin + p + s["sections"][a]))[case["layout"]]
        z = torch.polar(torch.ones(case["n"], 1, dtype=torch.float64, device="cuda"),
                        sign * s["pos"][:, a:a + 1].double() * s["freqs"][p].double())
        for x in ("q", "k"):
            y = torch.complex(s[x][..., i].double(), s[x][..., j].double()) * z
            out[x][..., i], out[x][..., j] = y.real, y.imag
    return out


def _exact_delta(s, case):
    """The recurrence token by token, all sequences side by side."""
    B, H, d, rep = case["n_seq"], case["heads"], case["d"], case["heads"] // case["heads_k"]
    index, scale = s["index"], s["scale"]
    steps = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    if steps * (30 if case["mode"] == "backward" else 8) > 1_500_000:
        return None

    def rows(x, group=1):  # [steps, B H, d, 1] or [steps, B H, 1, 1]
        x = torch.cat([x.double(), torch.zeros((1,) + x.shape[1:], dtype=torch.float64, device="cuda")])
        x = x.repeat_interleave(group, 1)[index[:, :steps]].transpose(0, 1)
        return x.reshape(steps, B * H, -1, 1).contiguous()

    def cols(x, heads):  # back to [n, heads, ...]
        y = torch.zeros((case["n"] + 1, H) + x.shape[2:3], dtype=torch.float64, device="cuda")
        y[index[:, :steps]] = x.reshape((steps, B, H) + x.shape[2:3]).transpose(0, 1)
        return y[:-1] if heads == H else y[:-1].unflatten(1, (heads, H // heads)).sum(2)

    q, k, v = rows(s["q"], rep), rows(s["k"], rep), rows(s["v"])
    al, be = torch.exp(rows(s["g"])), rows(s["beta"])
    S = s["state"].double().reshape(B * H, d, d).clone()

    def step(S, t, o=None):
        S.mul_(al[t])
        u = be[t] * torch.baddbmm(v[t], S, k[t], alpha=-1)
        S.baddbmm_(u, k[t].transpose(1, 2))
        if o is not None:
            torch.bmm(S, q[t], out=o[t])
        return u

    if case["mode"] != "backward":
        o = torch.empty((steps, B * H, d, 1), dtype=torch.float64, device="cuda")
        for t in range(steps):
            step(S, t, o)
        return {"o": cols(o[..., 0] * scale, H), "state": S.reshape(B, H, d, d)}
    marks = []
    for t in range(steps):
        if t % 64 == 0:
            marks.append(S.clone())
        step(S, t)
    do = rows(s["do"])
    D = s["dstate"].double().reshape(B * H, d, d).clone()
    dq, dk, dv = (torch.empty_like(v) for _ in range(3))
    dg, db = torch.empty_like(al), torch.empty_like(al)
    for m in reversed(range(len(marks))):
        S, past, us = marks[m], [], []
        for t in range(64 * m, min(steps, 64 * m + 64)):
            past.append(S.clone())
            us.append(step(S, t))
        for t in reversed(range(64 * m, min(steps, 64 * m + 64))):
            prev, u = past.pop(), us.pop()
            held = prev * al[t]
            kt = k[t].transpose(1, 2)
            D.baddbmm_(do[t], q[t].transpose(1, 2), alpha=scale)
            dq[t] = scale * ((held + u * kt).transpose(1, 2).contiguous() @ do[t])
            du = D @ k[t]
            db[t] = (du * (v[t] - held @ k[t])).sum(1, keepdim=True)
            dv[t] = be[t] * du
            dk[t] = D.transpose(1, 2).contiguous() @ u - held.transpose(1, 2).contiguous() @ dv[t]
            D.baddbmm_(dv[t], kt, alpha=-1)
            dg[t] = (D * held).sum((1, 2))[:, None, None]
            D.mul_(al[t])
    one = lambda x: cols(x, H)[..., 0]  # noqa: E731
    HK = case["heads_k"]
    return {"dq": cols(dq[..., 0], HK), "dk": cols(dk[..., 0], HK), "dv": cols(dv[..., 0], H),
            "dg": one(dg[..., 0]), "dbeta": one(db[..., 0]), "dstate": D.reshape(B, H, d, d)}
