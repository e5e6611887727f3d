"""Outputs of the sequence operators in the place of an input or of each other: refused
on the host, before any HIP call (the pointers here are never read)."""
import ctypes
import os

import pytest

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.skipif(not os.path.exists(zm.LIB_PATH),
                                reason="libzmttt.so not built (run the build first)")
INPUTS = ("offsets", "q", "k", "v", "g", "beta", "state")
BACKWARD_INPUTS = ("do", "dstate") + INPUTS
OUTPUTS = ("dq", "dk", "dv", "dg", "dbeta", "dstart")


def pointers(names, same):
    """A place of its own for each name; same = (a, b): a lies where b does."""
    p = {name: ctypes.c_void_p((1 + i) << 20) for i, name in enumerate(names)}
    if same:
        p[same[0]] = p[same[1]]
    return p


def desc():
    return ctypes.byref(zm.DeltaDesc(2, 1, 64, zm.BF16, 2, 1.0, 64, 64, 128, 128))


def delta(same, size=1 << 40):
    p = pointers(INPUTS + ("o", "state_out", "ws"), same)
    return zm.load_library().zm_delta_rule(
        desc(), 4, *(p[x] for x in ("offsets", "q", "k", "v", "g", "beta", "state", "state_out", "o", "ws")), size, None)


def step(same):
    p = pointers(INPUTS + ("o",), same)
    return zm.load_library().zm_delta_rule_step(desc(), *(p[x] for x in INPUTS[1:]), p["o"], None)


def backward(same, size=1 << 40):
    p = pointers(BACKWARD_INPUTS + OUTPUTS + ("ws",), same)
    return zm.load_library().zm_delta_rule_backward(
        desc(), 4, *(p[x] for x in ("offsets", "do", "q", "k", "v", "g", "beta", "state", "dstate")), p["dq"], 64,
        p["dk"], 64, p["dv"], 128, p["dg"], p["dbeta"], p["dstart"], p["ws"], size, None)


@pytest.mark.parametrize("other", INPUTS + ("state_out",))
def test_delta_rule(other):
    assert delta(("o", other)) == zm.ERR_INVALID_ARG
    if other not in ("state", "state_out"):
        assert delta(("state_out", other)) == zm.ERR_INVALID_ARG


@pytest.mark.parametrize("other", INPUTS[1:])
def test_delta_rule_step(other):
    assert step(("o", other)) == zm.ERR_INVALID_ARG


@pytest.mark.parametrize("out", OUTPUTS)
def test_delta_rule_backward(out):
    for other in BACKWARD_INPUTS + OUTPUTS:
        if other != out and {out, other} != {"dstart", "dstate"}:
            assert backward((out, other)) == zm.ERR_INVALID_ARG, f"{out} is {other}"


def test_the_state_s_gradient_may_be_replaced_and_apart_is_fine():
    # these go on to the check of the workspace
    assert backward(("dstart", "dstate"), size=0) == zm.ERR_WORKSPACE
    assert backward(None, size=0) == zm.ERR_WORKSPACE
    assert delta(("state_out", "state"), size=0) == zm.ERR_WORKSPACE


def test_layer_norm_backward():
    p = pointers(("dy", "x", "gamma", "stats", "dx", "params", "ws"), None)
    d = zm.NormDesc(64, zm.BF16, 1e-6, 0)
    for n in (0, 4):
        assert zm.load_library().zm_layer_norm_backward(
            ctypes.byref(d), n, p["dy"], 64, p["x"], 64, p["gamma"], p["stats"], p["dx"], 64, p["params"], p["params"],
            p["ws"], 1 << 20, None) == zm.ERR_INVALID_ARG
