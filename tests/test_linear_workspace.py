"""Workspaces of linear attention's gradient with and without dg: their sizes, on the CPU, and calls
in just enough of one, on the GPU."""
import os

import pytest
import torch

import reconstruction_lact_chunk_amd as zm
from linear_reference import inputs

pytestmark = pytest.mark.skipif(not os.path.exists(zm.LIB_PATH),
                                reason="libzmttt.so not built (run the build first)")
size = zm.linear_attention_backward_workspace_size


def desc(heads, heads_k, d=128, n_seq=1, io=zm.BF16, ld_g=None):
    w, wk = heads * d, heads_k * d
    return zm.LinearDesc(heads, heads_k, d, io, n_seq, 1.0, wk, wk, w, w, heads if ld_g is None else ld_g)


def test_states_of_the_chunks_are_for_dg_alone():
    n, h = 137_400, 8
    chunks = (n + 63) // 64
    for ld_g in (h, 0):
        d = desc(h, h, ld_g=ld_g)
        extra = size(d, n) - size(d, n, dg=False)
        exact = n * h * 4 + chunks * h * (128 * 128 * 4 + 8 + (0 if ld_g else 4))
        assert exact <= extra <= exact + 4 * 256
        # without it: no more than twice the forward's, whose states are at most 512 / heads to a
        # head and one more to its sequence
        assert size(d, n, dg=False) <= 2 * zm.linear_attention_workspace_size(d, n)
    # shared key heads add two fp32 copies of the value heads' tokens either way
    for dg in (True, False):
        more = size(desc(h, 2), n, dg=dg) - size(desc(h, h), n, dg=dg)
        assert 2 * n * h * 128 * 4 <= more <= 2 * n * h * 128 * 4 + 512


@pytest.mark.parametrize("io", [zm.BF16, zm.F32])
@pytest.mark.parametrize("heads", [1, 3, 8, 64])
@pytest.mark.parametrize("n_seq", [1, 2, 61, 1000])
def test_sizes_never_decrease(n_seq, heads, io):
    d = desc(heads, heads, 64, n_seq, io, 0)
    at = sorted([1, 2, 31, 32, 33, 64, 65, 100, 128, 129] + [k * s + t for k in range(1, 80, 3) for s in (512, 4096, 33000)
                                                             for t in (-1, 0, 1)])
    got = [size(d, n, dg=False) for n in at]
    assert got == sorted(got) and all(a <= size(d, n) for a, n in zip(got, at))


def test_refusals_of_the_size():
    lib = zm.load_library()
    import ctypes
    out = ctypes.c_size_t()
    ask = lib.zm_linear_attention_backward_workspace_size_no_dg
    assert ask(None, 4, ctypes.byref(out)) == zm.ERR_INVALID_ARG
    assert ask(ctypes.byref(desc(2, 2)), 4, None) == zm.ERR_INVALID_ARG
    assert ask(ctypes.byref(desc(2, 2)), -1, ctypes.byref(out)) == zm.ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("decay", ["none", "token"])
@pytest.mark.parametrize("n,n_seq,heads_k", [(100, 1, 2), (1374, 1, 4), (1500, 70, 2), (900, 3, 4)])
def test_no_more_is_used(n, n_seq, heads_k, decay, dtype):
    print(f"case linear workspace n={n} n_seq={n_seq} keys={heads_k} {decay} {dtype}", flush=True)
    h, d = 4, 64
    x = inputs(n, h, heads_k, d, dtype, n, n_seq=n_seq)
    gen = torch.Generator(device="cuda").manual_seed(5)
    do = torch.randn((n, h, d), generator=gen, device="cuda").to(dtype)
    dstate = torch.randn((n_seq, h, d, d), generator=gen, device="cuda")
    off = torch.linspace(0, n, n_seq + 1).round().to(dtype=torch.int32, device="cuda")
    g = None if decay == "none" else x["g"]
    a = (do, x["q"], x["k"], x["v"], g)
    kw = dict(state=x["state"], dstate=dstate, offsets=off)
    want = zm.linear_attention_backward(*a, **kw)
    of = desc(h, heads_k, d, n_seq, zm.BF16 if dtype == torch.bfloat16 else zm.F32, 0 if g is None else h)
    out = tuple(torch.empty_like(y) for y in want[:3]) + (None, torch.empty_like(want[4]))
    need = size(of, n, dg=False)
    ws = torch.full((need + 512,), 85, dtype=torch.uint8, device="cuda")
    zm.linear_attention_backward(*a, **kw, out=out, workspace=ws[:need])
    for i in (0, 1, 2, 4):
        assert torch.equal(out[i], want[i])
    assert (ws[need:] == 85).all()
    if need:
        with pytest.raises(zm.ZmError, match="workspace|WORKSPACE"):
            zm.linear_attention_backward(*a, **kw, out=out, workspace=ws[:need - 1])
