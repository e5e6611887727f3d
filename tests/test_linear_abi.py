"""Refusals of linear attention's entry points: checked on the host with the documented
status codes, before any HIP call (the pointers here are never read)."""
import ctypes
import os

import pytest
import torch

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.skipif(not os.path.exists(zm.LIB_PATH),
                                reason="libzmttt.so not built (run the build first)")
INVALID, UNSUPPORTED, WORKSPACE = zm.ERR_INVALID_ARG, zm.ERR_UNSUPPORTED, zm.ERR_WORKSPACE
INPUTS = ("offsets", "q", "k", "v", "g", "state")
BACKWARD_INPUTS = ("do", "dstate") + INPUTS
OUTPUTS = ("dq", "dk", "dv", "dg", "dstart")


def desc(**kw):
    f = dict(heads=2, heads_k=1, d_head=64, io_dtype=zm.BF16, n_seq=2, scale=1.0, ld_q=64, ld_k=64, ld_v=128, ld_o=128,
             ld_g=2)
    f.update(kw)
    return zm.LinearDesc(**f)


def places(names, same=None, **kw):
    """A place of its own for each name; same = (a, b): a lies where b does."""
    p = {name: ctypes.c_void_p((1 + i) << 20) for i, name in enumerate(names)}
    if same:
        p[same[0]] = p[same[1]]
    for name, at in kw.items():
        if name in p:
            p[name] = at if at is None else ctypes.c_void_p(at)
    return p


def forward(n=2000, same=None, size=1 << 40, d=None, **kw):
    names = INPUTS + ("o", "state_out", "ws")
    p = places(names, same, **kw)
    d = d if d is not None else desc(**{k: v for k, v in kw.items() if k not in names})
    return zm.load_library().zm_linear_attention(
        ctypes.byref(d), n, *(p[x] for x in ("offsets", "q", "k", "v", "g", "state", "state_out", "o", "ws")), size, None)


def step(same=None, **kw):
    names = INPUTS + ("o",)
    p = places(names, same, **kw)
    d = desc(**{k: v for k, v in kw.items() if k not in names})
    return zm.load_library().zm_linear_attention_step(ctypes.byref(d), *(p[x] for x in INPUTS[1:]), p["o"], None)


def backward(n=4, same=None, size=1 << 40, ld=(64, 64, 128), **kw):
    names = BACKWARD_INPUTS + OUTPUTS + ("ws",)
    p = places(names, same, **kw)
    d = desc(**{k: v for k, v in kw.items() if k not in names})
    return zm.load_library().zm_linear_attention_backward(
        ctypes.byref(d), n, *(p[x] for x in ("offsets", "do", "q", "k", "v", "g", "state", "dstate")), p["dq"], ld[0],
        p["dk"], ld[1], p["dv"], ld[2], p["dg"], p["dstart"], p["ws"], size, None)


BAD_DESC = [
    (dict(heads=0), INVALID), (dict(heads_k=0), INVALID), (dict(heads=3, heads_k=2, ld_v=192, ld_o=192, ld_g=3), INVALID),
    (dict(heads=65, heads_k=65, ld_q=4160, ld_k=4160, ld_v=4160, ld_o=4160, ld_g=65), UNSUPPORTED),
    (dict(d_head=32, ld_q=32), UNSUPPORTED), (dict(d_head=256, ld_q=256, ld_k=256, ld_v=512, ld_o=512), UNSUPPORTED),
    (dict(io_dtype=2), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(n_seq=-1), INVALID), (dict(ld_q=56), INVALID), (dict(ld_k=68), INVALID), (dict(ld_v=120), INVALID),
    (dict(ld_o=(1 << 24) + 8), INVALID), (dict(ld_g=1), INVALID), (dict(ld_g=-2), INVALID),
    (dict(ld_g=(1 << 24) + 1), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=(1 << 20) + 8), INVALID),
    (dict(g=(1 << 20) + 2), INVALID), (dict(state=(1 << 20) + 4), INVALID),
]


@pytest.mark.parametrize("bad,want", BAD_DESC)
def test_refusals(bad, want):
    assert forward(**bad) == want
    assert backward(**bad) == want
    if "n_seq" not in bad:
        assert step(**bad) == want


@pytest.mark.parametrize("bad,want", [
    (dict(n=-1), INVALID), (dict(n=1 << 31), INVALID), (dict(n_seq=0), INVALID), (dict(offsets=None), INVALID),
    (dict(offsets=(1 << 20) + 2), INVALID), (dict(n_seq=1 << 24), UNSUPPORTED), (dict(n_seq=(1 << 31) - 1), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws=(1 << 20) + 128), INVALID), (dict(size=64), WORKSPACE)])
def test_refusals_of_whole_sequences(bad, want):
    assert forward(**bad) == want
    assert backward(**bad) == want


def test_refusals_of_one_call_alone():
    assert forward(o=None) == INVALID and forward(state_out=(1 << 20) + 8) == INVALID
    assert step(o=None) == INVALID and step(state=None) == INVALID and step(n_seq=1 << 24) == UNSUPPORTED
    for name in ("do", "dq", "dk", "dv"):
        assert backward(**{name: None}) == INVALID
    assert backward(g=None) == INVALID and backward(dg=(1 << 20) + 2) == INVALID
    assert backward(ld=(56, 64, 128)) == INVALID and backward(ld=(64, 68, 128)) == INVALID
    assert backward(ld=(64, 64, 1 << 25)) == INVALID
    lib = zm.load_library()
    assert lib.zm_linear_attention_workspace_size(None, 4, ctypes.byref(ctypes.c_size_t())) == INVALID
    assert lib.zm_linear_attention_workspace_size(ctypes.byref(desc()), 4, None) == INVALID


@pytest.mark.parametrize("other", INPUTS + ("state_out",))
def test_outputs_apart(other):
    assert forward(same=("o", other)) == INVALID
    if other not in ("state", "state_out"):
        assert forward(same=("state_out", other)) == INVALID
    if other not in ("offsets", "state_out"):
        assert step(same=("o", other)) == INVALID
        assert other == "state" or step(same=("state", other)) == INVALID


@pytest.mark.parametrize("out", OUTPUTS)
def test_gradients_apart(out):
    for other in BACKWARD_INPUTS + OUTPUTS:
        if other != out and {out, other} != {"dstart", "dstate"}:
            assert backward(same=(out, other)) == INVALID, f"{out} is {other}"


def test_states_may_be_replaced():
    # these go on to the check of the workspace
    assert forward(same=("state_out", "state"), size=0) == WORKSPACE
    assert backward(same=("dstart", "dstate"), size=0) == WORKSPACE
    assert backward(g=None, dg=None, size=0) == WORKSPACE and backward(dstart=None, size=0) == WORKSPACE


def test_nothing_to_do_is_fine():
    assert forward(n=0, n_seq=0, q=None, k=None, v=None, o=None, ws=None, offsets=1 << 20) in (zm.OK, WORKSPACE)
    assert step(n_seq=0) == zm.OK


@pytest.mark.parametrize("dtype", [zm.BF16, zm.F32])
@pytest.mark.parametrize("heads", [1, 3, 8, 64])
@pytest.mark.parametrize("n_seq", [1, 2, 61, 1000])
def test_workspaces_never_decrease(n_seq, heads, dtype):
    d = desc(heads=heads, heads_k=heads, ld_q=64 * heads, ld_k=64 * heads, ld_v=64 * heads, ld_o=64 * heads, ld_g=0,
             n_seq=n_seq, io_dtype=dtype)
    sizes = [1, 2, 31, 32, 33, 64, 65, 100, 128, 129] + [k * s + t for k in range(1, 80, 3) for s in (512, 4096, 33000)
                                                         for t in (-1, 0, 1)]
    for size in (zm.linear_attention_workspace_size, zm.linear_attention_backward_workspace_size):
        got = [size(d, n) for n in sorted(sizes)]
        assert got == sorted(got)


def test_binding_refusals():
    q, v, g = torch.zeros(4, 1, 64), torch.zeros(4, 2, 64), torch.zeros(4, 2)
    state = torch.zeros(1, 2, 64, 64)
    bad = [dict(q=q[:, 0]), dict(k=q.bfloat16()), dict(v=torch.zeros(4, 2, 32)), dict(k=torch.zeros(3, 1, 64)),
           dict(q=torch.zeros(4, 3, 64), k=torch.zeros(4, 3, 64)), dict(g=g.double()), dict(g=torch.zeros(4, 3)),
           dict(g=torch.zeros(2, 4).T), dict(g=torch.zeros(1, 2).expand(4, 2)), dict(q=q[..., :0], k=q[..., :0]),
           dict(v=torch.zeros(4, 64, 2).transpose(1, 2)), dict(q=q.half(), k=q.half(), v=v.half())]
    for kw in bad:
        a = dict(dict(q=q, k=q, v=v, g=g), **kw)
        with pytest.raises(zm.ZmError):
            zm.linear_attention(**a)
        with pytest.raises(zm.ZmError):
            zm.linear_attention_step(**a, state=torch.zeros(4, 2, 64, 64))
        with pytest.raises(zm.ZmError):
            zm.linear_attention_backward(v, **a)
    for kw in (dict(state=state[:, :1]), dict(state=state.half()), dict(offsets=torch.zeros(2)), dict(out=v[:2]),
               dict(state_out=state.transpose(2, 3)), dict()):
        with pytest.raises(zm.ZmError):  # the last: tensors that are not on the GPU
            zm.linear_attention(q, q, v, g, **kw)
    for kw in (dict(out=(q, q, v, g)), dict(out=(q, q, v, g[:, :1], state)), dict(dstate=state[0]),
               dict(out=(q, q, q, g, state))):
        with pytest.raises(zm.ZmError):
            zm.linear_attention_backward(v, q, q, v, g, **kw)
    with pytest.raises(zm.ZmError, match="no dg"):
        zm.linear_attention_backward(v, q, q, v, None, out=(q, q, v, g, state))
    with pytest.raises(zm.ZmError, match="state"):
        zm.linear_attention_step(q, q, v, g, None)
