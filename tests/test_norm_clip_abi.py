"""Refusals of the normed rotation's and of the gradients' entry points: checked on the host with
the documented status codes, before any HIP call (the pointers here are never read)."""
import ctypes
import os

import pytest
import torch

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.skipif(not os.path.exists(zm.LIB_PATH),
                                reason="libzmttt.so not built (run the build first)")
INVALID, UNSUPPORTED, WORKSPACE = zm.ERR_INVALID_ARG, zm.ERR_UNSUPPORTED, zm.ERR_WORKSPACE


def at(i, off=0):
    return ctypes.c_void_p((i << 20) + off)


def desc(norm=0, eps=1e-6, sections=(8, 12, 12, 0), **kw):
    f = dict(heads_q=2, heads_k=2, d_head=64, io_dtype=0, layout=0, inverse=0, pos_f32=0, axes=3,
             sections=(ctypes.c_int32 * 4)(*sections), ld_q=128, ld_k=128, ld_q_out=128, ld_k_out=128)
    f.update(kw)
    return zm.NormRotaryDesc(zm.RotaryDesc(**f), norm, eps)


NAMES = ("pos", "freqs", "q", "k", "q_gamma", "q_beta", "k_gamma", "k_beta", "q_out", "k_out")
BACK = ("pos", "freqs", "dq_out", "dk_out", "q", "k", "q_gamma", "k_gamma", "dq", "dk", "dq_gamma", "dq_beta",
        "dk_gamma", "dk_beta", "ws")


def split(names, kw):
    p = {name: at(1 + i) for i, name in enumerate(names)}
    p.update({k: v for k, v in kw.items() if k in names})
    return p, desc(**{k: v for k, v in kw.items() if k not in NAMES + BACK})


def forward(n=4, **kw):
    p, d = split(NAMES, kw)
    return zm.load_library().zm_norm_rotary(ctypes.byref(d), n, *(p[x] for x in NAMES), None)


def backward(n=4, size=1 << 30, ld=(128, 128), **kw):
    p, d = split(BACK, kw)
    return zm.load_library().zm_norm_rotary_backward(
        ctypes.byref(d), n, *(p[x] for x in BACK[:8]), p["dq"], ld[0], p["dk"], ld[1], *(p[x] for x in BACK[10:]), size,
        None)


@pytest.mark.parametrize("bad,want", [
    (dict(norm=2), INVALID), (dict(norm=-1), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(inverse=1), INVALID), (dict(n=-1), INVALID), (dict(heads_q=0), INVALID),
    (dict(heads_q=65), UNSUPPORTED), (dict(heads_k=65), UNSUPPORTED), (dict(d_head=60), INVALID),
    (dict(d_head=264), UNSUPPORTED), (dict(io_dtype=2), INVALID), (dict(layout=3), INVALID), (dict(pos_f32=2), INVALID),
    (dict(axes=0), INVALID), (dict(axes=5), INVALID), (dict(sections=(8, 12, 13, 0)), INVALID),
    (dict(sections=(0, 0, 0, 0)), INVALID), (dict(sections=(8, 12, 4, 8)), INVALID), (dict(ld_q=120), INVALID),
    (dict(ld_k_out=132), INVALID), (dict(pos=None), INVALID), (dict(freqs=None), INVALID), (dict(q=None), INVALID),
    (dict(k=at(4, 8)), INVALID), (dict(q_gamma=at(5, 4)), INVALID), (dict(k_gamma=at(7, 8)), INVALID)])
def test_refusals(bad, want):
    assert forward(**bad) == want
    assert backward(**bad) == want


def test_refusals_of_one_call_alone():
    assert forward(q_out=None) == INVALID and forward(q_beta=at(6, 4)) == INVALID
    assert forward(q_out=at(3), ld_q_out=136) == INVALID      # in place, with another stride
    assert forward(q_out=at(10)) == INVALID and forward(q_out=at(4)) == INVALID and forward(k_out=at(3)) == INVALID
    for name in ("dq_out", "dk_out", "dq", "dk"):
        assert backward(**{name: None}) == INVALID
    assert backward(ld=(120, 128)) == INVALID and backward(ld=(128, 132)) == INVALID
    assert backward(dq=at(5), ld=(136, 128)) == INVALID and backward(dk=at(4), ld=(128, 136)) == INVALID
    assert backward(dq=at(10)) == INVALID and backward(dq=at(6)) == INVALID and backward(dk=at(5)) == INVALID
    assert backward(dq=at(4)) == INVALID and backward(dk=at(3)) == INVALID
    assert backward(dq_gamma=at(12)) == INVALID and backward(dk_beta=at(14, 2)) == INVALID
    assert backward(ws=None) == WORKSPACE and backward(ws=at(15, 128)) == INVALID and backward(size=100) == WORKSPACE
    lib = zm.load_library()
    assert lib.zm_norm_rotary_backward_workspace_size(ctypes.byref(desc()), 4, None) == INVALID
    assert lib.zm_norm_rotary(None, 4, *[None] * 11) == INVALID


def test_no_tokens_and_workspaces():
    assert forward(n=0, q=None, pos=None) == zm.OK
    sizes = [zm.norm_rotary_backward_workspace_size(desc(), n) for n in (0, 1, 2, 255, 256, 257, 1 << 20, 1 << 31)]
    assert sizes == sorted(sizes) and sizes[-1] == 1024 * 4 * 64 * 4


def test_binding_refusals():
    q, pos, freqs = torch.zeros(4, 2, 64), torch.zeros(4, 1, dtype=torch.int32), torch.zeros(32)
    for kw in (dict(q_gamma=torch.zeros(32)), dict(k_beta=torch.zeros(64).double()), dict(q=q[0]), dict(k=q.half()),
               dict(pos=pos.long()), dict(freqs=freqs[:8]), dict(sections=(16,)), dict(q_out=q[:2]), dict()):
        a = dict(dict(q=q, k=q, pos=pos, freqs=freqs, sections=(32,)), **kw)
        with pytest.raises(zm.ZmError):  # the last: tensors that are not on the GPU
            zm.norm_rotary(**a)
    for kw in (dict(dk_out=None), dict(dq_out=q[:2]), dict(out=(q, q)), dict(out=(q, None) + (None,) * 4),
               dict(out=(q, q, torch.zeros(3), None, None, None)), dict()):
        a = dict(dict(dq_out=q, dk_out=q, q=q, k=q, pos=pos, freqs=freqs, sections=(32,)), **kw)
        with pytest.raises(zm.ZmError):
            zm.norm_rotary_backward(**a)


def tensors(*rows):
    """(x, y, n, dtype[, reserved])"""
    return (zm.Tensor * max(len(rows), 1))(*[zm.Tensor(*r, *([0] * (5 - len(r)))) for r in rows])


def clip(t, count=None, max_norm=1.0, norm=at(90), ws=at(91), size=1 << 20, scale=True):
    lib, count = zm.load_library(), len(t) if count is None else count
    if scale:
        return lib.zm_clip_grads(t, count, max_norm, norm, ws, size, None)
    return lib.zm_grad_norm(t, count, norm, ws, size, None)


X, Y = 1 << 20, 2 << 20


@pytest.mark.parametrize("rows", [
    [(None, Y, 4, 1)], [(X + 1, Y, 4, 0)], [(X + 2, Y, 4, 1)], [(X, Y, -1, 1)], [(X, Y, (1 << 36) + 1, 1)],
    [(X, Y, 4, 2)], [(X, Y, 4, 1, 1)]])
def test_refused_tensors(rows):
    assert clip(tensors(*rows)) == INVALID and clip(tensors(*rows), scale=False) == INVALID


@pytest.mark.parametrize("rows", [
    [(X, None, 4, 1)], [(X, Y + 2, 4, 1)],
    [(X, X + 4, 4, 1)],                                    # an output over its own input, moved
    [(X, X, 4, 1), (X, X, 4, 1)],                          # the same tensor twice
    [(X, Y, 4, 1), (X, Y + 64, 4, 1)],
    [(X, Y, 4, 1), (X + 64, Y + 12, 4, 1)], [(X, Y, 100, 1), (Y + 396, Y + 1000, 4, 0)],
    [(X, X, 4, 1), (90 << 20, 90 << 20, 1, 0)], [(91 << 20, 91 << 20, 1, 0)]])
def test_refused_outputs(rows):
    assert clip(tensors(*rows)) == INVALID
    many = [(X + (1 << 12) * (9000 - i), X + (1 << 12) * (9000 - i), 5, 1) for i in range(1, 500)]  # not in order
    assert clip(tensors(*(many[:250] + rows + many[250:]))) == INVALID


def test_refused_calls():
    t = tensors((X, Y, 4, 1))
    for scale in (True, False):
        assert clip(t, count=-1, scale=scale) == INVALID and clip(None, count=1, scale=scale) == INVALID
        assert clip(t, count=8193, scale=scale) == UNSUPPORTED
        assert clip(t, norm=None, scale=scale) == INVALID and clip(t, norm=at(90, 2), scale=scale) == INVALID
        assert clip(t, ws=None, scale=scale) == WORKSPACE and clip(t, ws=at(91, 8), scale=scale) == INVALID
        assert clip(t, size=64, scale=scale) == WORKSPACE
    for bad in (-1.0, float("nan"), float("inf")):
        assert clip(t, max_norm=bad) == INVALID
    sizes = [zm.grad_norm_workspace_size(c) for c in (0, 1, 127, 128, 129, 8192)]
    assert sizes == sorted(sizes) and sizes[0] == 8192
    lib = zm.load_library()
    assert lib.zm_grad_norm_workspace_size(8193, ctypes.byref(ctypes.c_size_t())) == UNSUPPORTED
    assert lib.zm_grad_norm_workspace_size(1, None) == INVALID


def test_list_refusals():
    x = torch.zeros(8)
    for bad in (lambda: zm.TensorList([x.double()]), lambda: zm.TensorList([x.view(2, 4).T]), lambda: zm.TensorList([x]),
                lambda: zm.TensorList([x], []), lambda: zm.TensorList([x], [x[:4]]),
                lambda: zm.TensorList([x], [x.bfloat16()])):
        with pytest.raises(zm.ZmError):
            bad()
