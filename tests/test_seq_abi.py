"""Refusals of the layer norm's and the rotary rotation's entry points: checked on
the host with the documented status codes, before any HIP call (the pointers
here are never read)."""
import ctypes
import os

import pytest
import torch

import reconstruction_lact_chunk_amd as zm
from reconstruction_lact_chunk_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(zm.LIB_PATH),
                                reason="libzmttt.so not built (run the build first)")
GOOD, OFF = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)
INVALID, UNSUPPORTED, WORKSPACE = zm.ERR_INVALID_ARG, zm.ERR_UNSUPPORTED, zm.ERR_WORKSPACE


def lib():
    return zm.load_library()


def norm(n=4, width=64, io=zm.BF16, eps=1e-6, reserved=0, x=GOOD, ld_x=64, gamma=GOOD, y=GOOD, ld_y=64, stats=GOOD):
    d = zm.NormDesc(width, io, eps, reserved)
    return lib().zm_layer_norm(ctypes.byref(d), n, x, ld_x, gamma, None, y, ld_y, stats, None)


@pytest.mark.parametrize("bad,want", [
    (dict(n=-1), INVALID), (dict(n=(1 << 31) + 1), INVALID), (dict(width=0), INVALID), (dict(width=60), INVALID),
    (dict(width=8200, ld_x=8200, ld_y=8200), UNSUPPORTED), (dict(io=2), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(reserved=1), INVALID), (dict(x=None), INVALID), (dict(x=OFF), INVALID), (dict(ld_x=56), INVALID),
    (dict(ld_x=68), INVALID), (dict(y=None), INVALID), (dict(ld_y=60), INVALID), (dict(gamma=OFF), INVALID),
    (dict(ld_y=72), INVALID),   # in place, with another stride
    (dict(stats=ctypes.c_void_p(1 << 20 | 2)), INVALID),
])
def test_layer_norm_refusals(bad, want):
    assert norm(**bad) == want


def test_layer_norm_without_rows_is_fine():
    assert norm(n=0, x=None, y=None) == zm.OK
    assert lib().zm_layer_norm(None, 0, None, 0, None, None, None, 0, None, None) == INVALID


def norm_backward(n=4, width=64, dy=GOOD, x=GOOD, stats=GOOD, dx=GOOD, dgamma=GOOD, ws=GOOD, size=1 << 20, ld=64,
                  ld_dx=64):
    d = zm.NormDesc(width, zm.BF16, 1e-6, 0)
    return lib().zm_layer_norm_backward(ctypes.byref(d), n, dy, ld, x, ld, None, stats, dx, ld_dx, dgamma, None, ws,
                                        size, None)


@pytest.mark.parametrize("bad,want", [
    (dict(dy=None), INVALID), (dict(x=OFF), INVALID), (dict(stats=None), INVALID), (dict(dx=None), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=OFF), INVALID), (dict(size=100), WORKSPACE), (dict(ld_dx=72), INVALID),
    (dict(ld=60), INVALID), (dict(n=-1), INVALID), (dict(width=8200, ld=8200, ld_dx=8200), UNSUPPORTED),
])
def test_layer_norm_backward_refusals(bad, want):
    assert norm_backward(**bad) == want


def test_layer_norm_workspace_never_decreases():
    sizes = [zm.layer_norm_backward_workspace_size(n, 1024) for n in (0, 1, 16, 17, 1000, 16384, 16385, 1 << 31)]
    assert sizes == sorted(sizes) and sizes[-1] == 1024 * 2 * 1024 * 4


def rot(n=4, pos=GOOD, freqs=GOOD, q=GOOD, k=GOOD, qo=GOOD, ko=GOOD, sections=(8, 12, 12, 0), **kw):
    f = dict(heads_q=2, heads_k=2, d_head=64, io_dtype=0, layout=0, inverse=0, pos_f32=0, axes=3,
             sections=(ctypes.c_int32 * 4)(*sections), ld_q=128, ld_k=128, ld_q_out=128, ld_k_out=128)
    f.update(kw)
    return lib().zm_rotary(ctypes.byref(zm.RotaryDesc(**f)), n, pos, freqs, q, k, qo, ko, None)


@pytest.mark.parametrize("bad,want", [
    (dict(n=-1), INVALID), (dict(heads_q=0), INVALID), (dict(heads_q=65), UNSUPPORTED), (dict(heads_k=-1), INVALID),
    (dict(heads_k=65), UNSUPPORTED), (dict(d_head=60), INVALID), (dict(d_head=264), UNSUPPORTED),
    (dict(io_dtype=2), INVALID), (dict(layout=3), INVALID), (dict(layout=-1), INVALID), (dict(inverse=2), INVALID),
    (dict(pos_f32=2), INVALID), (dict(axes=0), INVALID), (dict(axes=5), INVALID),
    (dict(sections=(8, 12, 13, 0)), INVALID), (dict(sections=(-1, 12, 12, 0)), INVALID),
    (dict(sections=(8, 12, 4, 8)), INVALID), (dict(sections=(0, 0, 0, 0)), INVALID),
    (dict(sections=(2 ** 31 - 1, 2 ** 31 - 1, 2, 0)), INVALID), (dict(pos=None), INVALID), (dict(freqs=None), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(qo=None), INVALID), (dict(ko=OFF), INVALID),
    (dict(ld_q=120), INVALID), (dict(ld_k=132), INVALID), (dict(ld_q_out=136), INVALID), (dict(ld_k_out=136), INVALID),
])
def test_rotary_refusals(bad, want):
    assert rot(**bad) == want


@pytest.mark.parametrize("q,k,qo,ko", [(1, 2, 2, 3), (1, 2, 3, 1), (1, 2, 3, 3)])
def test_rotary_outputs_in_place_of_the_other_input_or_of_each_other(q, k, qo, ko):
    p = [ctypes.c_void_p(i << 20) for i in (q, k, qo, ko)]
    assert rot(q=p[0], k=p[1], qo=p[2], ko=p[3]) == INVALID


def test_rotary_without_tokens_is_fine():
    assert rot(n=0, pos=None, freqs=None, q=None, k=None, qo=None, ko=None) == zm.OK


def test_the_binding_names_what_is_wrong():
    x = torch.zeros(4, 64)
    with pytest.raises(zm.ZmError, match="on the GPU"):
        zm.layer_norm(x)
    with pytest.raises(zm.ZmError, match="gamma"):
        zm.layer_norm(x, torch.ones(63))
    with pytest.raises(zm.ZmError, match="out must be"):
        zm.layer_norm(x, out=torch.zeros(5, 64))
    with pytest.raises(zm.ZmError, match="stats"):
        zm.layer_norm(x, stats=torch.zeros(2, 5))
    with pytest.raises(zm.ZmError, match="column stride"):
        zm.layer_norm(torch.zeros(64, 4).T)
    with pytest.raises(zm.ZmError, match="2-D bf16 or fp32"):
        zm.layer_norm(x.half())
    with pytest.raises(zm.ZmError, match="dy must be"):
        zm.layer_norm_backward(x.bfloat16(), x, torch.zeros(2, 4))
    q, pos, f = torch.zeros(4, 2, 64), torch.zeros(4, 3, dtype=torch.int32), torch.zeros(32)
    with pytest.raises(zm.ZmError, match="on the GPU"):
        zm.rotary(q, q, pos, f, (8, 12, 12))
    with pytest.raises(zm.ZmError, match="pos must be"):
        zm.rotary(q, q, pos.long(), f, (8, 12, 12))
    with pytest.raises(zm.ZmError, match="freqs"):
        zm.rotary(q, q, pos, f, (8, 12, 11))
    with pytest.raises(zm.ZmError, match="k: "):
        zm.rotary(q, q.bfloat16(), pos, f, (8, 12, 12))
    with pytest.raises(zm.ZmError, match="q_out"):
        zm.rotary(q, q, pos, f, (8, 12, 12), q_out=torch.zeros(4, 2, 32))
    with pytest.raises(zm.ZmError, match="unit stride"):
        zm.rotary(q.transpose(1, 2).contiguous().transpose(1, 2), q, pos, f, (8, 12, 12))


def test_structs_match_the_header():
    assert ctypes.sizeof(B.NormDesc) == 16 and ctypes.sizeof(B.RotaryDesc) == 80
