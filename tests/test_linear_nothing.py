"""Linear attention of no tokens and of no sequences: nothing is needed, last states are the first ones
and the gradient of the first ones that of the last."""
import ctypes
import os

import pytest
import torch

import reconstruction_lact_chunk_amd as zm
from linear_reference import inputs
from test_linear_abi import backward, desc, forward, step

pytestmark = pytest.mark.skipif(not os.path.exists(zm.LIB_PATH),
                                reason="libzmttt.so not built (run the build first)")
NOTHING = dict(n=0, n_seq=0, ws=None, size=0)


def test_no_sequences_need_nothing():
    assert zm.linear_attention_workspace_size(desc(n_seq=0), 0) == 0
    for ld_g in (0, 2):
        for dg in (True, False):
            assert zm.linear_attention_backward_workspace_size(desc(n_seq=0, ld_g=ld_g), 0, dg) == 0
    assert forward(**NOTHING, q=None, k=None, v=None, o=None) == zm.OK
    assert forward(**NOTHING) == zm.OK and step(n_seq=0) == zm.OK
    # a dg of [heads] would be written, so without one
    assert backward(**NOTHING, dg=None) == zm.OK and backward(**NOTHING, dg=None, g=None) == zm.OK
    assert backward(**NOTHING) == zm.OK  # a dg of [0, heads]


def test_no_tokens_need_no_workspace():
    for n_seq in (1, 3, 64):
        assert zm.linear_attention_workspace_size(desc(n_seq=n_seq), 0) == 0
        assert zm.linear_attention_backward_workspace_size(desc(n_seq=n_seq), 0, False) == 0
    out = ctypes.c_size_t()
    size = zm.load_library().zm_linear_attention_workspace_size
    assert size(ctypes.byref(desc(n_seq=0)), 1, ctypes.byref(out)) == zm.ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("decay", ["token", "head", "none"])
@pytest.mark.parametrize("n_seq", [0, 1, 3, 100])
def test_gradient_of_no_tokens(n_seq, decay):
    for dtype, heads_k in ((torch.bfloat16, 4), (torch.float32, 2)):
        print(f"case linear nothing n_seq={n_seq} {decay} {dtype}", flush=True)
        x = inputs(0, 4, heads_k, 64, dtype, 1, n_seq=n_seq)
        g = {"token": x["g"], "head": torch.full((4,), -0.5, device="cuda"), "none": None}[decay]
        dstate = torch.randn((n_seq, 4, 64, 64), device="cuda")
        off = torch.zeros(n_seq + 1, dtype=torch.int32, device="cuda")
        do = torch.empty_like(x["v"])
        for last in (dstate, dstate.clone()):
            into = torch.full_like(dstate, 7.0) if last is dstate else last
            dg = None if g is None else torch.full(g.shape, 7.0, device="cuda")
            out = (torch.empty_like(x["q"]), torch.empty_like(x["k"]), torch.empty_like(x["v"]), dg, into)
            zm.linear_attention_backward(do, x["q"], x["k"], x["v"], g, state=x["state"], dstate=last, offsets=off, out=out)
            assert torch.equal(into, dstate)
            assert dg is None or not dg.any()
        none = zm.linear_attention_backward(do, x["q"], x["k"], x["v"], g, offsets=off)
        assert none[4].shape == (n_seq, 4, 64, 64) and not none[4].any()
        end = zm.linear_attention(x["q"], x["k"], x["v"], g, state=x["state"], offsets=off)[1]
        assert torch.equal(end, x["state"])
