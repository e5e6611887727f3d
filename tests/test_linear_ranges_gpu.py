"""Linear attention with decays over its ranges: tables of more sequences than a wave has
lanes (in order and longest first), segments of several chunks, the widest strides, two calls at
once, and the largest tensors of clip_grads.  Compared as in test_linear_attention_gpu.py and
test_linear_backward_gpu.py."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm
import test_linear_attention_gpu as forwards
import test_linear_backward_gpu as backwards
from linear_reference import inputs

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


def both(x, offsets=None):
    forwards.compare(x, forwards.run(x, offsets), offsets)
    do, dstate = backwards.grads_in(x, 31)
    backwards.compare(backwards.run(do, dstate, x, offsets), do, dstate, x, offsets)


def ragged(n, n_seq, seed):
    """Offsets from 3 on, many empty sequences, one of a third of the tokens; some rows behind the last."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(n // 3, n - 11, (n_seq - 1,), generator=g).sort().values.tolist()
    cuts[::5] = cuts[1::5] + cuts[-1:] * (len(cuts[::5]) - len(cuts[1::5]))  # equal ends: empty ones
    return [3] + sorted(cuts) + [n - 11]


# 64 sequences need no table, 65 do; 6 heads: more workgroups than run at once, longest first;
# 600 sequences: too many to sort
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,n_seq,heads", [(1500, 64, 2), (1500, 65, 2), (1800, 70, 6), (2000, 600, 1)])
def test_many_ragged_sequences(n, n_seq, heads, dtype):
    print(f"case linear ranges n={n} n_seq={n_seq} heads={heads} {dtype}", flush=True)
    both(inputs(n, heads, heads, 64, dtype, n_seq, n_seq=n_seq), ragged(n, n_seq, n_seq))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,heads,heads_k,strong", [(1200, 64, 8, False), (2300, 1, 1, True), (2300, 2, 1, False)])
def test_segments_of_several_chunks(n, heads, heads_k, strong, dtype):
    print(f"case linear ranges segments n={n} heads={heads} {dtype}", flush=True)
    x = inputs(n, heads, heads_k, 64, dtype, 33, decay=0.02)
    if strong:
        x["g"][100::97] = -30.0
        x["g"][500:700] = -3.0
        x["g"][1000] = -1e4
        x["g"][1500:1600] = 0.2
    both(x)


def test_the_widest_strides():
    """fp32 rows 2^24 elements apart: byte offsets within a chunk just under 2^32, past it over two."""
    n, h, d, ld = 70, 2, 64, 1 << 24
    print(f"case linear ranges strides, {n * ld * 4 / 1e9:.1f} GB", flush=True)
    x = inputs(n, h, h, d, torch.float32, 34)
    do, dstate = backwards.grads_in(x, 32)
    want, grads = forwards.run(x), backwards.run(do, dstate, x)
    buf = torch.zeros(n, ld, device="cuda")
    w = h * d

    def view(i):  # the last ones end with the row
        at = ld - (8 - i) * w
        return buf[:, at:at + w].unflatten(1, (h, d))

    y = dict(x, q=view(0), k=view(1), v=view(2))
    for name in "qkv":
        y[name].copy_(x[name])
    view(3).copy_(do)
    got = forwards.run(y, out=view(4))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = (view(5), view(6), view(7), torch.empty_like(grads[3]), torch.empty_like(grads[4]))
    for name, a, b in zip(backwards.NAMES, backwards.run(view(3), dstate, y, out=out), grads):
        assert torch.equal(a, b), name
    for name in "qkv":
        assert torch.equal(y[name], x[name])
    assert not buf[:, :ld - 8 * w].any()


def test_two_calls_at_once():
    """On two streams, each with its own workspace and outputs: what they are one after the other."""
    n = 2000
    calls = []
    for seed in (35, 36):
        x = inputs(n, 4, 2, 128, torch.bfloat16, seed, n_seq=2)
        do, dstate = backwards.grads_in(x, seed)
        off = torch.tensor([0, 700, n], dtype=torch.int32, device="cuda")
        call = lambda x=x, do=do, ds=dstate, off=off: (  # noqa: E731
            zm.linear_attention(*forwards.args(x), state=x["state"], offsets=off)
            + tuple(zm.linear_attention_backward(do, *forwards.args(x), state=x["state"], dstate=ds, offsets=off)))
        calls.append(call)
    want = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls[i]())
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for a, b in zip(g, want[i]):
                assert torch.equal(a, b)


def test_a_gradient_past_32_bits():
    n = (1 << 31) + 9
    print(f"case clip of {2 * n / 1e9:.1f} GB", flush=True)
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    x[0], x[-1], x[n // 2] = 3.0, 4.0, 12.0
    norm = zm.clip_grads([x, torch.zeros(3, device="cuda")], 6.5)
    assert float(norm) == 13.0  # 6.5 / 13 is a half but for the 1e-6: each value rounds to its half
    assert [float(x[i]) for i in (0, -1, n // 2)] == [1.5, 2.0, 6.0]
    x[0] = x[-1] = x[n // 2] = 0.0
    assert not x.any()
