"""A layer of linear attention and its training step: q, k and v where one projection left
them, q and k normalised and rotated, the attention over packed sequences, its gradient back to the
projection's output and the norms' parameters, and the clipping of all gradients by their norm.

Each operator is compared, on what the ones before it gave, with its formula in 64 bits
and its own tolerance; the whole in fp32 with 64-bit autograd of the whole.  The tolerance of that: q
and k are rounded and turned to 2^-18 (test_norm_rotary_gpu.py), and every gradient is a sum over
products of q, k, v, do and states, each of which has moved by at most 2^-17 of its size; up to six
of them follow each other (q, k, v, do, the state's decay and the norm's own), so a tensor's 2-norm moves by
6 * 2^-17 of what its terms' sizes would give, and these are under 2^6 times the tensor's (sums of 128
random terms): 2^-8 of the 2-norm is allowed."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm
import test_grad_clip_gpu as clip
import test_linear_attention_gpu as forwards
import test_linear_backward_gpu as backwards
import test_norm_rotary_gpu as rotary
from linear_reference import forward, inputs

pytestmark = pytest.mark.gpu
N, H, HK, D, SECTIONS, EPS = 300, 4, 2, 64, (8, 12, 12), 1e-6
OFFSETS = [0, 131, 131, 290]  # rows behind the last sequence are padding


def make(dtype, seed):
    lin = inputs(N, H, HK, D, dtype, seed, n_seq=3)
    rot = rotary.inputs(N, HK, HK, D, dtype, SECTIONS, seed + 1)
    x = torch.zeros((N, (2 * HK + H) * D), dtype=dtype, device="cuda")
    t = dict(x=x, q=x[:, :HK * D].unflatten(1, (HK, D)), k=x[:, HK * D:2 * HK * D].unflatten(1, (HK, D)),
             v=x[:, 2 * HK * D:].unflatten(1, (H, D)), pos=rot["pos"], freqs=rot["freqs"], g=lin["g"], state=lin["state"],
             off=torch.tensor(OFFSETS, dtype=torch.int32, device="cuda"))
    for name in "qk":
        t[name].copy_(rot[name])
        t[name + "_gamma"], t[name + "_beta"] = rot[name + "_gamma"], rot[name + "_beta"]
    t["v"].copy_(lin["v"])
    t["do"], _ = backwards.grads_in(lin, seed + 2)
    t["do"][OFFSETS[-1]:] = 0.0
    return t


def buffers(t):
    z = torch.zeros_like
    dx = z(t["x"])
    return dict(qr=z(t["q"]), kr=z(t["k"]), o=z(t["v"]), end=z(t["state"]), dx=dx, flat=torch.zeros(4 * D + N * H, device="cuda"),
                dqr=z(t["q"]), dkr=z(t["k"]), dstart=z(t["state"]), norm=torch.zeros(1, device="cuda"))


def views(t, b):
    dx, flat = b["dx"], b["flat"]
    return dict(dq=dx[:, :HK * D].unflatten(1, (HK, D)), dk=dx[:, HK * D:2 * HK * D].unflatten(1, (HK, D)),
                dv=dx[:, 2 * HK * D:].unflatten(1, (H, D)), params=flat[:4 * D].view(4, D), dg=flat[4 * D:].view(N, H))


def step(t, b, max_norm, raw=None):
    """One forward and backward pass and the clipping; raw takes the gradients before it."""
    w = views(t, b)
    zm.norm_rotary(t["q"], t["k"], t["pos"], t["freqs"], SECTIONS, q_gamma=t["q_gamma"], k_gamma=t["k_gamma"],
                   q_beta=t["q_beta"], k_beta=t["k_beta"], eps=EPS, q_out=b["qr"], k_out=b["kr"])
    zm.linear_attention(b["qr"], b["kr"], t["v"], t["g"], state=t["state"], offsets=t["off"], out=b["o"], state_out=b["end"])
    zm.linear_attention_backward(t["do"], b["qr"], b["kr"], t["v"], t["g"], state=t["state"], offsets=t["off"],
                                 out=(b["dqr"], b["dkr"], w["dv"], w["dg"], b["dstart"]))
    p = w["params"]
    zm.norm_rotary_backward(b["dqr"], b["dkr"], t["q"], t["k"], t["pos"], t["freqs"], SECTIONS, q_gamma=t["q_gamma"],
                            k_gamma=t["k_gamma"], eps=EPS, out=(w["dq"], w["dk"], p[0], p[1], p[2], p[3]))
    if raw is not None:
        raw.extend([b["dx"].clone(), b["flat"].clone()])
    zm.clip_grads([b["dx"], b["flat"]], max_norm, norm=b["norm"])


def whole(t):
    """The gradients by x and the parameters in 64 bits, by autograd of the whole."""
    names = ("q", "k", "v", "q_gamma", "k_gamma", "q_beta", "k_beta", "g")
    leaves = {name: t[name].double().requires_grad_() for name in names}
    rot = (t["pos"], t["freqs"], SECTIONS, 0)
    qr, kr = (rotary.reference(leaves[p], leaves[p + "_gamma"], leaves[p + "_beta"], EPS, zm.NORM_RMS, *rot) for p in "qk")
    o, _ = forward(qr, kr, leaves["v"], leaves["g"], t["state"], OFFSETS)
    return o, dict(zip(names, torch.autograd.grad((o * t["do"].double()).sum(), list(leaves.values()))))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_each_operator_on_what_the_others_give(dtype):
    print(f"case linear block {dtype}", flush=True)
    t = make(dtype, 50)
    b, raw = buffers(t), []
    step(t, b, 1.0, raw)
    w = views(t, dict(b, dx=raw[0], flat=raw[1]))
    rotary.check(t, (b["qr"], b["kr"]), SECTIONS, 0, zm.NORM_RMS, EPS)
    lin = dict(q=b["qr"], k=b["kr"], v=t["v"], g=t["g"], state=t["state"])
    forwards.compare(lin, (b["o"], b["end"]), OFFSETS)
    backwards.compare((b["dqr"], b["dkr"], w["dv"], w["dg"], b["dstart"]), t["do"], None, lin, OFFSETS)
    rotary.check_backward(t, (b["dqr"], b["dkr"]), (w["dq"], w["dk"], *w["params"]), SECTIONS, 0, zm.NORM_RMS, EPS)
    clip.check(raw, [b["dx"], b["flat"]], b["norm"], 1.0)
    assert not b["o"][OFFSETS[-1]:].any() and not raw[0][OFFSETS[-1]:].any()  # padding has no gradient


def test_the_whole_in_fp32():
    t = make(torch.float32, 60)
    b, raw = buffers(t), []
    step(t, b, 1.0, raw)
    w = views(t, dict(b, dx=raw[0], flat=raw[1]))
    o, grads = whole(t)
    got = dict(q=w["dq"], k=w["dk"], v=w["dv"], g=w["dg"], q_gamma=w["params"][0], k_gamma=w["params"][1],
               q_beta=w["params"][2], k_beta=w["params"][3])
    a, e = OFFSETS[0], OFFSETS[-1]
    assert (b["o"][a:e].double() - o[a:e]).norm() <= 2.0 ** -8 * o.norm()
    for name, y in got.items():
        off, size = (y.double() - grads[name]).norm(), grads[name].norm()
        assert off <= 2.0 ** -8 * size, f"{name}: {float(off / size):.3g}"


def test_a_captured_step_of_changing_inputs():
    """Captured on a stream of its own, replayed with other tokens in the same places: the eager step's bits."""
    dtype = torch.bfloat16
    t, b = make(dtype, 70), None
    b = buffers(t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(t, b, 0.5)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(t, b, 0.5)
    for seed in (70, 80, 90):
        fresh = make(dtype, seed)
        want = buffers(fresh)
        step(fresh, want, 0.5)
        for name in ("x", "g", "state", "do", "pos", "freqs", "q_gamma", "k_gamma", "q_beta", "k_beta"):
            t[name].copy_(fresh[name])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name, y in want.items():
            assert torch.equal(b[name], y), f"{name}, seed {seed}"
