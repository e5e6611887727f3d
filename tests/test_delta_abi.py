"""Refusals of the gated delta rule's entry points: checked on the host with the
documented status codes, before any HIP call (the pointers here are never read)."""
import ctypes
import os

import pytest
import torch

import reconstruction_lact_chunk_amd as zm
from reconstruction_lact_chunk_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(zm.LIB_PATH),
                                reason="libzmttt.so not built (run the build first)")
GOOD, OFF = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)
ODD = ctypes.c_void_p((1 << 20) + 2)
OUT = [ctypes.c_void_p((2 + i) << 20) for i in range(4)]
INVALID, UNSUPPORTED, WORKSPACE = zm.ERR_INVALID_ARG, zm.ERR_UNSUPPORTED, zm.ERR_WORKSPACE


def lib():
    return zm.load_library()


def desc(**kw):
    f = dict(heads=4, heads_k=2, d_head=64, io_dtype=zm.BF16, n_seq=1, scale=1.0, ld_q=128, ld_k=128, ld_v=256,
             ld_o=256)
    f.update(kw)
    return zm.DeltaDesc(**f)


POINTERS = ("offsets", "q", "k", "v", "g", "beta")


def forward(n=4, state=GOOD, state_out=GOOD, o=OUT[0], ws=GOOD, size=1 << 40, **kw):
    p = {name: kw.pop(name, GOOD) for name in POINTERS}
    return lib().zm_delta_rule(ctypes.byref(desc(**kw)), n, *(p[x] for x in POINTERS), state, state_out, o, ws, size,
                               None)


def step(state=GOOD, o=OUT[0], **kw):
    p = {name: kw.pop(name, GOOD) for name in POINTERS[1:]}
    return lib().zm_delta_rule_step(ctypes.byref(desc(**kw)), *(p[x] for x in POINTERS[1:]), state, o, None)


def backward(n=4, do=GOOD, state=GOOD, dstate=GOOD, dq=OUT[0], ld_dq=128, dk=OUT[1], ld_dk=128, dv=OUT[2], ld_dv=256,
             dg=GOOD, dbeta=GOOD, dstart=GOOD, ws=GOOD, size=1 << 40, **kw):
    p = {name: kw.pop(name, GOOD) for name in POINTERS}
    return lib().zm_delta_rule_backward(ctypes.byref(desc(**kw)), n, p["offsets"], do,
                                        *(p[x] for x in POINTERS[1:]), state, dstate, dq, ld_dq, dk, ld_dk, dv, ld_dv,
                                        dg, dbeta, dstart, ws, size, None)


DESCRIPTOR = [
    (dict(heads=0), INVALID), (dict(heads_k=0), INVALID), (dict(heads=-4), INVALID), (dict(heads_k=3), INVALID),
    (dict(d_head=0), INVALID), (dict(d_head=72, ld_q=144, ld_k=144, ld_v=288, ld_o=288), UNSUPPORTED),
    (dict(d_head=256, ld_q=512, ld_k=512, ld_v=1024, ld_o=1024), UNSUPPORTED),
    (dict(heads=65, heads_k=1, ld_v=65 * 64, ld_o=65 * 64), UNSUPPORTED), (dict(io_dtype=2), INVALID),
    (dict(io_dtype=-1), INVALID), (dict(n_seq=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(ld_q=120), INVALID), (dict(ld_k=120), INVALID), (dict(ld_v=248), INVALID),
    (dict(ld_o=248), INVALID), (dict(ld_q=132), INVALID), (dict(ld_o=260), INVALID),
    (dict(ld_v=(1 << 24) + 8), INVALID),
]
INPUTS = [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(g=None), INVALID),
    (dict(beta=None), INVALID), (dict(q=OFF), INVALID), (dict(k=OFF), INVALID), (dict(v=OFF), INVALID),
    (dict(g=ODD), INVALID), (dict(beta=ODD), INVALID),
]
COUNTS = [
    (dict(n=-1), INVALID), (dict(n=1 << 31), INVALID), (dict(n_seq=0), INVALID), (dict(n=(1 << 31) - 1), UNSUPPORTED),
    (dict(n_seq=1 << 23), UNSUPPORTED), (dict(n_seq=2, offsets=None), INVALID), (dict(offsets=ODD), INVALID),
]
MEMORY = [(dict(ws=None, n_seq=2), WORKSPACE), (dict(ws=ODD, n_seq=2), INVALID), (dict(size=100, n_seq=2), WORKSPACE)]


@pytest.mark.parametrize("bad,want", DESCRIPTOR + INPUTS + COUNTS + MEMORY + [
    (dict(o=None), INVALID), (dict(o=OFF), INVALID), (dict(state=OFF), INVALID), (dict(state_out=OFF), INVALID),
    (dict(ws=None, io_dtype=zm.F32), WORKSPACE), (dict(ws=None, n=2000), WORKSPACE),
    (dict(o=GOOD), INVALID), (dict(v=OUT[0]), INVALID),   # in place of an input
])
def test_delta_rule_refusals(bad, want):
    assert forward(**bad) == want


@pytest.mark.parametrize("bad,want", DESCRIPTOR + INPUTS + [
    (dict(o=None), INVALID), (dict(o=OFF), INVALID), (dict(state=None), INVALID), (dict(state=OFF), INVALID),
    (dict(n_seq=1 << 23), UNSUPPORTED), (dict(o=GOOD), INVALID),
])
def test_delta_rule_step_refusals(bad, want):
    assert step(**bad) == want


@pytest.mark.parametrize("bad,want", DESCRIPTOR + INPUTS + COUNTS + MEMORY + [
    (dict(do=None), INVALID), (dict(do=OFF), INVALID), (dict(dq=None), INVALID), (dict(dk=OFF), INVALID),
    (dict(dv=None), INVALID), (dict(dg=None), INVALID), (dict(dbeta=ODD), INVALID), (dict(state=OFF), INVALID),
    (dict(dstate=OFF), INVALID), (dict(dstart=OFF), INVALID), (dict(ld_dq=120), INVALID), (dict(ld_dk=132), INVALID),
    (dict(ld_dv=248), INVALID), (dict(ld_dv=(1 << 24) + 8), INVALID), (dict(ws=None), WORKSPACE),
    (dict(dq=GOOD), INVALID), (dict(dv=GOOD), INVALID), (dict(dk=OUT[0]), INVALID), (dict(do=OUT[2]), INVALID),
])
def test_delta_rule_backward_refusals(bad, want):
    assert backward(**bad) == want


def test_null_descriptors():
    assert lib().zm_delta_rule(None, 0, *([None] * 10), 0, None) == INVALID
    assert lib().zm_delta_rule_step(None, *([None] * 8)) == INVALID
    assert lib().zm_delta_rule_workspace_size(None, 0, ctypes.byref(ctypes.c_size_t())) == INVALID
    assert lib().zm_delta_rule_workspace_size(ctypes.byref(desc()), 0, None) == INVALID
    assert lib().zm_delta_rule_backward_workspace_size(ctypes.byref(desc()), -1, ctypes.byref(ctypes.c_size_t())) == INVALID


def test_nothing_to_do_needs_nothing():
    none = dict.fromkeys(POINTERS[1:])
    assert forward(n=0, n_seq=0, state=None, state_out=None, o=None, ws=None, size=0, offsets=None, **none) == zm.OK
    assert step(n_seq=0, state=None, o=None, **none) == zm.OK


def test_workspace_sizes():
    one = desc()
    # one sequence of bf16 tokens that is not cut into segments needs none
    assert zm.delta_rule_workspace_size(one, 400) == 0
    assert zm.delta_rule_workspace_size(desc(io_dtype=zm.F32), 400) > 0
    assert zm.delta_rule_workspace_size(one, 4000) > 0 and zm.delta_rule_workspace_size(desc(n_seq=2), 1) > 0
    # the gradient keeps M and its gradient, 64 x 64 floats each, at every chunk of a head
    chunks, dd = 1000 // 64 + 1, 64 * 64 * 4
    assert zm.delta_rule_backward_workspace_size(one, 1000) >= 2 * 4 * chunks * dd


def test_the_binding_names_what_is_wrong():
    q, v, g = torch.zeros(4, 2, 64), torch.zeros(4, 4, 64), torch.zeros(4, 4)
    state = torch.zeros(1, 4, 64, 64)
    with pytest.raises(zm.ZmError, match="on the GPU"):
        zm.delta_rule(q, q, v, g, g, state=state)
    with pytest.raises(zm.ZmError, match="no multiple"):
        zm.delta_rule(q, q, v[:, :3].contiguous(), g, g)
    with pytest.raises(zm.ZmError, match="k: shape"):
        zm.delta_rule(q, q[:3], v, g, g)
    with pytest.raises(zm.ZmError, match="v: dtype"):
        zm.delta_rule(q, q, v.bfloat16(), g, g)
    with pytest.raises(zm.ZmError, match="dtype"):
        zm.delta_rule(q.half(), q.half(), v.half(), g, g)
    with pytest.raises(zm.ZmError, match="g must be"):
        zm.delta_rule(q, q, v, g.bfloat16(), g)
    with pytest.raises(zm.ZmError, match="beta must be"):
        zm.delta_rule(q, q, v, g, g[:, :2])
    with pytest.raises(zm.ZmError, match="offsets"):
        zm.delta_rule(q, q, v, g, g, offsets=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(zm.ZmError, match="state must be"):
        zm.delta_rule(q, q, v, g, g, state=state, offsets=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(zm.ZmError, match="state_out must be"):
        zm.delta_rule(q, q, v, g, g, state_out=state.transpose(2, 3))
    with pytest.raises(zm.ZmError, match="out: shape"):
        zm.delta_rule(q, q, v, g, g, out=q)
    with pytest.raises(zm.ZmError, match="unit stride"):
        zm.delta_rule(q.transpose(0, 1).contiguous().transpose(0, 1)[:, :, ::1].transpose(1, 2).contiguous().transpose(1, 2),
                      q, v, g, g)
    with pytest.raises(zm.ZmError, match="needs a state"):
        zm.delta_rule_step(q, q, v, g, g, None)
    with pytest.raises(zm.ZmError, match="state must be"):
        zm.delta_rule_step(q, q, v, g, g, state)
    with pytest.raises(zm.ZmError, match="do: shape"):
        zm.delta_rule_backward(q, q, q, v, g, g)
    with pytest.raises(zm.ZmError, match="dstate must be"):
        zm.delta_rule_backward(v, q, q, v, g, g, dstate=state[0])
    with pytest.raises(zm.ZmError, match="six tensors"):
        zm.delta_rule_backward(v, q, q, v, g, g, out=(q, q, v))
    with pytest.raises(zm.ZmError, match="dg must be"):
        zm.delta_rule_backward(v, q, q, v, g, g, out=(q, q, v, g[:2], g, state))


def test_struct_matches_the_header():
    assert ctypes.sizeof(B.DeltaDesc) == 56
