"""A TensorList of tensors that have moved or changed their size since it was built: the calls refuse
it on the host, before its addresses are used.  On the CPU, without the check that all tensors lie
on one GPU; a list that is as it was goes on to the refusal of a norm that does not."""
import os

import pytest
import torch

import reconstruction_lact_chunk_amd as zm
from reconstruction_lact_chunk_amd import binding

pytestmark = pytest.mark.skipif(not os.path.exists(zm.LIB_PATH),
                                reason="libzmttt.so not built (run the build first)")


@pytest.fixture(autouse=True)
def on_the_cpu(monkeypatch):
    monkeypatch.setattr(binding, "_same_gpu", lambda *tensors: None)


def refused(lst, match):
    for call in (lambda: zm.grad_norm(lst), lambda: zm.clip_grads(lst, 1.0)):
        with pytest.raises(zm.ZmError, match=match):
            call()


MOVES = [
    lambda x: setattr(x, "data", torch.ones(5, 8)),
    lambda x: setattr(x, "data", x.data[1:]),
    lambda x: setattr(x, "data", x.data[:3]),           # at the same place, but shorter
    lambda x: x.set_(torch.ones(40)),
    lambda x: x.resize_(3),
    lambda x: x.resize_(4000),
    lambda x: x.untyped_storage().resize_(0),           # freed, as by sharded training between steps
]


@pytest.mark.parametrize("which", range(len(MOVES)))
def test_moved_tensors(which):
    for side in (0, 1):
        xs, ys = [torch.zeros(5, 8) for _ in range(3)], [torch.zeros(5, 8) for _ in range(3)]
        lists = [zm.TensorList(xs, ys)] + ([zm.TensorList(xs)] if side == 0 else [])
        for lst in lists:
            lst.check()
            refused(lst, "one GPU")
        MOVES[which]((xs, ys)[side][1])
        for lst in lists:
            refused(lst, "moved")


def test_tensors_that_stay():
    xs = [torch.zeros(5, 8), torch.zeros(0), torch.zeros(3, dtype=torch.bfloat16)]
    lst = zm.TensorList(xs)
    xs[0].add_(1.0)
    xs[0].data = xs[0].data.view(40)                    # the same elements
    lst.check()
    zm.TensorList([]).check()
