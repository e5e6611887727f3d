"""Timing cases of linear attention with decays, the normed rotation of queries and keys,
and the clipping of gradients by their global norm.

Each case runs one operator in its plain form (own = False: elementary torch
operations in 32 bits, angles and sums of decays in 64) or through the package
(own = True).  Frames have 37 * 37 + 5 = 1374 tokens and the model width is
1024 = 8 heads of 128, as in workloads.py.
"""
import math

import torch

own = False

FRAME = 1374
CHUNK = 64
HALVES, PAIRS, AXIS_HALVES = 0, 1, 2


def listed():
    lin = dict(op="linear", mode="forward", n=FRAME, n_seq=1, heads=8, heads_k=8, d=128, dtype="bf16", decay="token")
    rot = dict(op="rotary", n=FRAME, heads=8, heads_k=8, d=128, dtype="bf16", s0=16, s1=24, s2=24, layout=HALVES,
               norm="rms", affine=False, far=0, fused=True, backward=False)
    clip = dict(op="clip", dtype="f32", layers=0, count=3, n=3 * 8 * 256 * 128, flat=False, shapes=0, max_norm=1.0)
    return [
        # one token of one sequence: what a serving step waits for
        dict(lin, name="linear_step_1", mode="step", n=1),
        # one token of each of 256 sequences: bound by the states' memory traffic
        dict(lin, name="linear_step_256", mode="step", n=256, n_seq=256),
        # one streamed frame with the state carried along
        dict(lin, name="linear_frame"),
        # a packed batch of ragged sequences, query/key heads shared by four value heads
        dict(lin, name="linear_packed", n=54_321, n_seq=61, heads=16, heads_k=4),
        # 100 frames as one long sequence, one decay to a head: few heads, a long axis
        dict(lin, name="linear_100_frames", n=100 * FRAME, decay="head"),
        # the gradient of 8 sequences of about a frame each
        dict(lin, name="linear_backward_8_frames", mode="backward", n=8 * FRAME, n_seq=8),
        # the gradient of fp32 tokens of narrow heads, shared keys, one decay to a head, an odd count
        dict(lin, name="linear_backward_f32", mode="backward", n=4_123, n_seq=3, heads=6, heads_k=2, d=64,
             dtype="f32", decay="head"),
        # q and k of one frame, where the fused projection left them
        dict(rot, name="norm_rotary_frame"),
        # fp32 tokens of grouped heads, layer norm with its parameters, far and fractional positions
        dict(rot, name="norm_rotary_f32", n=40 * FRAME, heads=16, heads_k=4, d=64, dtype="f32", s0=8, s1=12, s2=8,
             layout=PAIRS, norm="layer", affine=True, far=1_000_000, fused=False),
        # the gradient over the tokens of 100 frames
        dict(rot, name="norm_rotary_backward_100_frames", n=100 * FRAME, affine=True, backward=True),
        # the gradients of one layer's fast weights: three small tensors
        dict(clip, name="clip_fast_weights"),
        # the gradients of 24 layers: projections, gates, norms and fast weights, bf16 and fp32
        dict(clip, name="clip_24_layers", dtype="mixed", layers=24, count=0, n=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "forward", "forward", "backward", "rotary", "rotary", "clip"])
    dtype = "f32" if rng.random() < 0.3 else "bf16"
    if op == "clip":
        count = _log(rng, 1, 600)
        return dict(op="clip", dtype=rng.choice(["bf16", "f32", "mixed"]), layers=0, count=count,
                    n=_log(rng, 4 * count, 100_000_000), flat=rng.random() < 0.5, shapes=rng.randrange(1 << 30),
                    max_norm=rng.choice([0.25, 1.0, 1.0, 1e6]))
    d = rng.choice([64, 128])
    if op == "rotary":
        s = [rng.randrange(0, d // 6) + 1 for _ in range(3)]
        if rng.random() < 0.6:  # a whole rotation of 8-pair sections
            s = [d // 8, 3 * d // 16, 3 * d // 16]
        group, heads_k = rng.choice([1, 1, 2, 4]), rng.choice([1, 2, 4])
        most = 60 * FRAME * 8 * 128 // (heads_k * group * d * (2 if dtype == "f32" else 1))
        return dict(op="rotary", n=_log(rng, 1, min(most, 100 * FRAME)), heads=heads_k * group, heads_k=heads_k, d=d,
                    dtype=dtype, s0=s[0], s1=s[1], s2=s[2], layout=rng.choice([HALVES, PAIRS, AXIS_HALVES]),
                    norm=rng.choice(["rms", "layer"]), affine=rng.random() < 0.7, far=rng.choice([0, 0, 1_000_000]),
                    fused=rng.random() < 0.5, backward=rng.random() < 0.5)
    heads_k = rng.choice([1, 2, 4, 8])
    heads = heads_k * rng.choice([1, 1, 2, 3])
    case = dict(op="linear", mode=op, n=0, n_seq=0, heads=heads, heads_k=heads_k, d=d, dtype=dtype,
                decay=rng.choice(["token", "token", "head", "none"]))
    if op == "step":
        case["n"] = case["n_seq"] = _log(rng, 1, 4096 // heads)
        return case
    case["n_seq"] = _log(rng, 1, 64)
    most = (60 if op == "forward" else 16) * FRAME * 8 * 128 // (heads * d * (2 if dtype == "f32" else 1))
    case["n"] = _log(rng, 1, max(2, min(most, 60 * FRAME)))
    return case


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


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


def _shapes(case):
    """Element counts of the gradient tensors and whether each is bf16."""
    if case["layers"]:
        # a layer's norm, input projection [q | k | v | rate], gate, output scale and fast weights
        layer = [(1024, 0), (1024, 0), (3080 * 1024, 1), (1024 * 1024, 1), (1024, 0)] + [(8 * 256 * 128, 0)] * 3
        return layer * case["layers"]
    if case["shapes"] == 0:
        return [(case["n"] // case["count"], 0)] * case["count"]
    g = torch.Generator().manual_seed(case["shapes"])
    w = torch.exp(3.0 * torch.randn(case["count"], generator=g)).double()
    sizes = (w / w.sum() * case["n"]).long().clamp_(min=1).tolist()
    kinds = torch.randint(0, 2, (case["count"],), generator=g).tolist()
    fixed = {"bf16": 1, "f32": 0}.get(case["dtype"])
    return [(s, k if fixed is None else fixed) for s, k in zip(sizes, kinds)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(case)}
    if case["op"] == "clip":
        return _prepare_clip(s, case, gen)
    dtype, n = _dtype(case), case["n"]
    H, HK, d = case["heads"], case["heads_k"], case["d"]

    def tokens(heads, scale=1.0):
        return torch.randn((n, heads, d), generator=gen, device="cuda").mul_(scale).to(dtype)

    if case["op"] == "rotary":
        if case["fused"]:  # q and k where the projection of [q | k | v | rate] left them
            y = torch.randn((n, (H + 2 * HK) * d + H + (-H) % 8), generator=gen, device="cuda").mul_(1.5).to(dtype)
            s["q"], s["k"] = y[:, :H * d].unflatten(1, (H, d)), y[:, H * d:(H + HK) * d].unflatten(1, (HK, d))
        else:
            s["q"], s["k"] = tokens(H, 1.5), tokens(HK, 1.5)
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
        for x in ("q", "k"):
            s[x + "_gamma"] = s[x + "_beta"] = None
            if case["affine"]:
                s[x + "_gamma"] = torch.randn(d, generator=gen, device="cuda").mul_(0.2).add_(1.0)
                s[x + "_beta"] = torch.randn(d, generator=gen, device="cuda").mul_(0.1)
        s["eps"] = 1e-6
        if case["backward"]:
            s["dq"], s["dk"] = tokens(H), tokens(HK)
        return s
    s["q"], s["k"], s["v"] = tokens(HK), tokens(HK), tokens(H)
    # decays from a few tokens to some thousand, by head
    rate = torch.exp(torch.empty(H, device="cuda").uniform_(math.log(1e-3), 0.0, generator=gen))
    z = torch.randn((n, H), generator=gen, device="cuda")
    s["g"] = {"token": -rate * torch.log1p(torch.exp(z - 1.0)), "head": -rate, "none": None}[case["decay"]]
    s["state"] = torch.randn((case["n_seq"], H, d, d), generator=gen, device="cuda")
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
        s["do"] = tokens(H)
        s["dstate"] = torch.randn((case["n_seq"], H, d, d), generator=gen, device="cuda").mul_(d ** -0.5)
    return s


def _buckets(case):
    """For each type its tensors' first elements and counts in one buffer: one behind the other (flat),
    or each from a multiple of 64 on with zeros between them."""
    out = {}
    for i, (c, k) in enumerate(_shapes(case)):
        b = out.setdefault(k, dict(index=[], at=[], size=[], end=0))
        b["index"].append(i)
        b["at"].append(b["end"])
        b["size"].append(c)
        b["end"] += c if case["flat"] else -(-c // 64) * 64
    return out


def _prepare_clip(s, case, gen):
    count = len(_shapes(case))
    s["grads"], s["out"], s["buckets"] = [None] * count, [None] * count, []
    for k, b in sorted(_buckets(case).items()):
        t = torch.bfloat16 if k else torch.float32
        bucket = torch.zeros(b["end"], dtype=t, device="cuda")
        if case["flat"]:  # the gradients are pieces of one buffer too
            x = torch.randn(b["end"], generator=gen, device="cuda").mul_(1e-3).to(t)
        for i, a, c in zip(b["index"], b["at"], b["size"]):
            s["grads"][i] = x[a:a + c] if case["flat"] else \
                torch.randn(c, generator=gen, device="cuda").mul_(10.0 ** -(2 + i % 3)).to(t)
            s["out"][i] = bucket[a:a + c]
        s["buckets"].append(bucket)
    s["max_norm"] = case["max_norm"]
    if own:
        import reconstruction_lact_chunk_amd as zm

        s["list"] = zm.TensorList(s["grads"], s["out"])
    return s


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "clip":
        return _clip(state)
    if case["op"] == "rotary":
        return _rotary_backward(state, case) if case["backward"] else _rotary(state, case)
    return {"step": _linear_step, "forward": _linear, "backward": _linear_backward}[case["mode"]](state, case)


def _run_own(s, case):
    import reconstruction_lact_chunk_amd as zm

    if case["op"] == "clip":
        norm = zm.clip_grads(s["list"], s["max_norm"])
        return {"norm": norm, "grads": s["buckets"]}
    if case["op"] == "rotary":
        norm = zm.NORM_RMS if case["norm"] == "rms" else zm.NORM_LAYER
        a = (s["q"], s["k"], s["pos"], s["freqs"], s["sections"])
        if case["backward"]:
            dq, dk, dqg, dkg, dqb, dkb = zm.norm_rotary_backward(
                s["dq"], s["dk"], *a, q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=s["eps"], norm=norm,
                layout=case["layout"])
            return {"dq": dq, "dk": dk, "dq_gamma": dqg, "dk_gamma": dkg, "dq_beta": dqb, "dk_beta": dkb}
        q, k = zm.norm_rotary(*a, q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], q_beta=s["q_beta"],
                              k_beta=s["k_beta"], eps=s["eps"], norm=norm, layout=case["layout"])
        return {"q": q, "k": k}
    a = (s["q"], s["k"], s["v"], s["g"])
    if case["mode"] == "step":
        o = zm.linear_attention_step(*a, s["state"], scale=s["scale"])
        return {"o": o, "state": s["state"]}
    if case["mode"] == "backward":
        dq, dk, dv, dg, dstate = zm.linear_attention_backward(
            s["do"], *a, state=s["state"], dstate=s["dstate"], offsets=s["offsets"], scale=s["scale"])
        return _grads(dq, dk, dv, dg, dstate)
    o, end = zm.linear_attention(*a, state=s["state"], offsets=s["offsets"], scale=s["scale"])
    return {"o": o, "state": end}


def _grads(dq, dk, dv, dg, dstate):
    """Without decays there is no dg."""
    out = {"dq": dq, "dk": dk, "dv": dv, "dstate": dstate}
    return out if dg is None else dict(out, dg=dg)


# ---- plain forms ------------------------------------------------------------
def _clip(s):
    norm = torch.stack([x.float().square().sum() for x in s["grads"]]).sum().sqrt()
    c = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    for x, y in zip(s["grads"], s["out"]):
        y.copy_(x.float() * c)
    return {"norm": norm, "grads": s["buckets"]}


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


def _turn(s, case, xf, back):
    """xf [n, heads, d] rotated by the positions, or back."""
    sec = s["sections"]
    ax = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(sec, device="cuda"),
                                 output_size=sum(sec))
    angle = s["pos"].double()[:, ax] * s["freqs"].double()
    c, sn = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    sn = -sn if back else sn
    i, j = _pair_dims(case)
    a, b = xf[..., i], xf[..., j]
    y = xf.clone()
    y[..., i] = a * c - b * sn
    y[..., j] = a * sn + b * c
    return y


def _normed(x, case, eps):
    """(x - mean) r (or x r) and r, in 32 bits."""
    x = x.float()
    if case["norm"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    return x * r, r


def _rotary(s, case):
    out = {}
    for x in ("q", "k"):
        y, _ = _normed(s[x], case, s["eps"])
        if case["affine"]:
            y = y * s[x + "_gamma"] + s[x + "_beta"]
        out[x] = _turn(s, case, y, False).to(s[x].dtype)
    return out


def _rotary_backward(s, case):
    out = {}
    for x in ("q", "k"):
        h, r = _normed(s[x], case, s["eps"])
        u = _turn(s, case, s["d" + x].float(), True)
        out[f"d{x}_gamma"], out[f"d{x}_beta"] = (u * h).sum((0, 1)), u.sum((0, 1))
        a = u * s[x + "_gamma"] if case["affine"] else u
        dx = a - h * (a * h).mean(-1, keepdim=True)
        if case["norm"] == "layer":
            dx = dx - a.mean(-1, keepdim=True)
        out["d" + x] = (dx * r).to(s[x].dtype)
    return out


def _linear_step(s, case):
    rep = case["heads"] // case["heads_k"]
    q, k = (s[x].float().repeat_interleave(rep, 1)[:, :, None] for x in ("q", "k"))
    S = s["state"]
    if s["g"] is not None:
        S.mul_(torch.exp(s["g"]).expand(case["n"], -1)[:, :, None, None])
    S.add_(s["v"].float()[..., None] * k)
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
    rep, n, H = case["heads"] // case["heads_k"], case["n"], case["heads"]
    q, k = (_padded(s[x], s["index"]).repeat_interleave(rep, 1) for x in ("q", "k"))
    v = _padded(s["v"], s["index"])
    g = s["g"].expand(n, H) if s["g"] is not None else torch.zeros((n, H), device="cuda")
    c = torch.cumsum(_padded(g, s["index"]).double(), -1)
    low = torch.ones(CHUNK, CHUNK, device="cuda", dtype=torch.bool).tril()
    G = torch.exp((c[..., :, None] - c[..., None, :]).masked_fill(~low, -math.inf)).float()
    gam, dec = torch.exp(c).float()[..., None], torch.exp(c[..., -1:] - c).float()[..., None]
    q = q * s["scale"]
    return dict(q=q, k=k, v=v, G=G, P=torch.matmul(q, _t(k)) * G, gam=gam, dec=dec, last=gam[..., -1:, :])


def _states(p, M, left, right, reverse):
    """The state before every chunk (behind it, in reverse) and the one at the end."""
    B = torch.matmul(_t(left), right)
    out = []
    order = range(B.shape[2])
    for c in reversed(order) if reverse else order:
        out.append(M)
        M = p["last"][:, :, c] * M + B[:, :, c]
    return torch.stack(out[::-1] if reverse else out, 2), M


def _linear(s, case):
    p = _chunk_parts(s, case)
    M0, M = _states(p, _t(s["state"]), p["k"] * p["dec"], p["v"], False)
    o = p["gam"] * torch.matmul(p["q"], M0) + torch.matmul(p["P"], p["v"])
    return {"o": _back(o, s, s["v"].dtype), "state": _t(M)}


def _linear_backward(s, case):
    p = _chunk_parts(s, case)
    do = _padded(s["do"], s["index"])
    M0, _ = _states(p, _t(s["state"]), p["k"] * p["dec"], p["v"], False)
    D1, D = _states(p, _t(s["dstate"]), p["q"] * p["gam"], do, True)
    dP = torch.matmul(do, _t(p["v"]))
    W = dP * p["G"]
    doM, vD = p["gam"] * torch.matmul(do, _t(M0)), p["dec"] * torch.matmul(p["v"], _t(D1))
    dq = doM + torch.matmul(W, p["k"])
    dk = vD + torch.matmul(_t(W), p["q"])
    dv = p["dec"] * torch.matmul(p["k"], D1) + torch.matmul(_t(p["P"]), do)
    dg = None
    if s["g"] is not None:
        # token t's decay is in all that goes from tokens before t to t and later ones
        X = dP * p["P"]
        inside = (torch.cumsum(X, -1) - X).tril().sum(-2)
        came, goes = (doM * p["q"]).sum(-1), (vD * p["k"]).sum(-1)
        came = torch.flip(torch.cumsum(torch.flip(came, (-1,)), -1), (-1,))
        goes = torch.cumsum(goes, -1) - goes
        through = p["last"][..., 0, 0] * (M0 * D1).sum((-1, -2))
        dg = _back(inside + came + goes + through[..., None], s, torch.float32)
        dg = dg.sum(0) if s["g"].dim() == 1 else dg
    rep, HK = case["heads"] // case["heads_k"], case["heads_k"]
    dq, dk = (x.unflatten(1, (HK, rep)).sum(2) for x in (dq * s["scale"], dk))
    t = s["v"].dtype
    return _grads(_back(dq, s, t), _back(dk, s, t), _back(dv, s, t), dg, _t(D))


# ---- what one pass cannot do without ---------------------------------------
def work(case):
    if case["op"] == "clip":
        shapes = _shapes(case)
        return {"bytes": sum(c * (4 if k else 8) for c, k in shapes), "flops": 3 * sum(c for c, _ in shapes)}
    size, n = 2 if case["dtype"] == "bf16" else 4, case["n"]
    H, HK, d = case["heads"], case["heads_k"], case["d"]
    if case["op"] == "rotary":
        pairs, e = case["s0"] + case["s1"] + case["s2"], n * (H + HK) * d
        back = case["backward"]
        return {"bytes": e * size * (3 if back else 2) + 12 * n, "flops": e * (12 if back else 6) + 6 * n * (H + HK) * pairs}
    states, tokens = case["n_seq"] * H * d * d * 4, n * d * size
    decays = {"token": 4 * n * H, "head": 4 * H, "none": 0}[case["decay"]]
    if case["mode"] == "backward":
        return {"bytes": tokens * (4 * HK + 3 * H) + 2 * decays + 3 * states, "flops": 10 * n * H * d * d}
    return {"bytes": tokens * (2 * HK + 2 * H) + decays + 2 * states, "flops": 4 * n * H * d * d}


# ---- the definitions in 64 bits -----------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        total = sum(float(torch.dot(x.double(), x.double())) for x in s["grads"])
        c = min(1.0, s["max_norm"] / (math.sqrt(total) + 1e-6))
        grads = []
        for _, b in sorted(_buckets(case).items()):
            grads.append(torch.zeros(b["end"], dtype=torch.float64, device="cuda"))
            for i, a, size in zip(b["index"], b["at"], b["size"]):
                grads[-1][a:a + size] = s["grads"][i].double() * c
        return {"norm": torch.tensor(math.sqrt(total), dtype=torch.float64, device="cuda"), "grads": grads}
    if case["op"] == "rotary":
        return _exact_rotary(s, case)
    return _exact_linear(s, case)


def _exact_rotary(s, case):
    P = sum(s["sections"])
    ends = [case["s0"], case["s0"] + case["s1"], P]
    at = []
    for p in range(P):
        a = 0 if p < ends[0] else 1 if p < ends[1] else 2
        begin = ends[a] - s["sections"][a]
        at.append(((p, p + P), (2 * p, 2 * p + 1), (begin + p, begin + p + s["sections"][a]))[case["layout"]] + (a,))
    first, second, axis = (torch.tensor(x, device="cuda") for x in zip(*at))
    z = torch.polar(torch.ones((case["n"], 1, P), dtype=torch.float64, device="cuda"),
                    (s["pos"].double().index_select(1, axis) * s["freqs"].double())[:, None])
    out = {}
    for x in ("q", "k"):
        xd = s[x].double().requires_grad_(case["backward"])
        gamma, beta = (torch.full((case["d"],), v, dtype=torch.float64, device="cuda") if s[x + t] is None
                       else s[x + t].double() for t, v in (("_gamma", 1.0), ("_beta", 0.0)))
        gamma.requires_grad_(case["backward"])
        beta.requires_grad_(case["backward"])
        with torch.enable_grad():
            mu = xd.sum(-1, keepdim=True) / case["d"] if case["norm"] == "layer" else 0.0
            y = (xd - mu) * (((xd - mu) ** 2).sum(-1, keepdim=True) / case["d"] + s["eps"]) ** -0.5 * gamma + beta
            turned = torch.complex(y.index_select(2, first), y.index_select(2, second)) * z
            y = y.index_copy(2, first, turned.real).index_copy(2, second, turned.imag)
        if case["backward"]:
            y.backward(s["d" + x].double())
            out["d" + x], out[f"d{x}_gamma"], out[f"d{x}_beta"] = xd.grad, gamma.grad, beta.grad
        else:
            out[x] = y
    return out


def _exact_linear(s, case):
    """All sequences side by side, BLOCK tokens at a time by the sum over earlier tokens; gradients
    by differentiating that."""
    BLOCK = 192
    n, H, rep, index = case["n"], case["heads"], case["heads"] // case["heads_k"], s["index"]
    back = case["mode"] == "backward"
    leaf = {x: s[x].double().requires_grad_(back) for x in ("q", "k", "v", "state")}
    leaf["g"] = (torch.zeros(H, device="cuda") if s["g"] is None else s["g"]).double().requires_grad_(back)

    def rows(x, group=1):  # [sequences, heads, steps, ...]
        x = torch.cat([x, torch.zeros((1,) + x.shape[1:], dtype=torch.float64, device="cuda")])
        return x.repeat_interleave(group, 1)[index].transpose(1, 2)

    with torch.enable_grad():
        q, k, v = rows(leaf["q"], rep), rows(leaf["k"], rep), rows(leaf["v"])
        g = rows(leaf["g"].expand(n, H))
        S, o = leaf["state"], []
        for a in range(0, q.shape[2], BLOCK):
            qb, kb, vb, c = q[:, :, a:a + BLOCK], k[:, :, a:a + BLOCK], v[:, :, a:a + BLOCK], g[:, :, a:a + BLOCK]
            c = c.cumsum(-1)
            later = torch.ones(c.shape[-1], c.shape[-1], device="cuda").triu(1).bool()
            reach = (c[..., :, None] - c[..., None, :]).masked_fill(later, -math.inf).exp()
            o.append(qb @ S.mT * c.exp()[..., None] + (qb @ kb.mT * reach) @ vb)
            S = S * c[..., -1, None, None].exp() + (vb * (c[..., -1:] - c).exp()[..., None]).mT @ kb
        o = torch.zeros((n + 1, H, case["d"]), dtype=torch.float64, device="cuda").index_put(
            (index,), (torch.cat(o, 2) * s["scale"]).transpose(1, 2))[:-1]
    if not back:
        return {"o": o, "state": S}
    torch.autograd.backward([o, S], [s["do"].double(), s["dstate"].double()])
    return _grads(leaf["q"].grad, leaf["k"].grad, leaf["v"].grad, None if s["g"] is None else leaf["g"].grad,
                  leaf["state"].grad)
