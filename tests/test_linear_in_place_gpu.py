"""zm.linear_attention_backward with the gradient of the first states written where that of the last
ones is: the bits of a call whose outputs lie apart, for sequences in one segment, which start
from that array, for cut ones, which do not, and for both in one call."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm
from linear_reference import inputs
from test_linear_backward_gpu import NAMES, args, grads_in

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


def both(x, offsets, seed):
    do, dstate = grads_in(x, seed)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    call = lambda last, out: zm.linear_attention_backward(  # noqa: E731
        do, *args(x), state=x["state"], dstate=last, offsets=off, out=out)
    z = torch.zeros_like  # rows outside the sequences are not written

    def outputs(last):
        return z(x["q"]), z(x["k"]), z(x["v"]), None if x["g"] is None else z(x["g"]), last

    want = call(dstate, outputs(z(dstate)))
    for _ in range(2):
        last = dstate.clone()
        out = outputs(last)
        for name, a, b in zip(NAMES, call(last, out), want):
            assert (a is None and b is None) or torch.equal(a, b), name


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 64, 100, 1374])  # the last: cut
def test_one_sequence(n, d, dtype):
    print(f"case linear in place n={n} d={d} {dtype}", flush=True)
    x = inputs(n, 2, 1, d, dtype, n + d)
    both(x, None, 1)
    both(x, [0, n], 2)
    both(x, [0, n // 2], 3)


# heads times sequences past what runs at once, so that the first sequences' workgroups of dv end
# before the last ones' of dk begin
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_seq,length,heads,heads_k,d", [(64, 70, 16, 16, 128), (64, 70, 16, 4, 64), (200, 40, 16, 16, 64),
                                                          (90, 33, 8, 8, 128)])
def test_more_sequences_than_run_at_once(n_seq, length, heads, heads_k, d, dtype):
    print(f"case linear in place {n_seq} x {length} heads={heads} d={d} {dtype}", flush=True)
    n = n_seq * length
    x = inputs(n, heads, heads_k, d, dtype, n_seq, n_seq=n_seq)
    both(x, list(range(0, n + 1, length)), 4)


@pytest.mark.parametrize("dtype", DTYPES)
def test_cut_and_whole_sequences_and_empty_ones(dtype):
    print(f"case linear in place ragged {dtype}", flush=True)
    offsets = [5, 5, 45, 1900, 1900, 1930, 1931, 2040]
    x = inputs(2050, 2, 2, 128, dtype, 6, n_seq=7)
    both(x, offsets, 5)


def test_without_decays():
    x = inputs(300, 16, 16, 64, torch.bfloat16, 7, n_seq=100)
    x["g"] = None
    both(x, list(range(0, 301, 3)), 6)
