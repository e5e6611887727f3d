"""The training step of test_linear_block_gpu.py in fp32 as a whole against 64-bit autograd, so tight
that no step can have dropped to bf16 on the way.

Tolerance.  Every stage's outputs are sums of terms of random signs.  At most 64 roundings follow each other in
a stage's sum (linear_reference.py), of random signs themselves: sqrt(64) = 8 steps of 2^-24 of a
sum's terms, whose root of squares is the sum's own size.  Six stages follow each other (norm and
rotation, state, output, the gradient's two passes, the norm's gradient), and division by the heads' norms
and multiplication by gamma (within 0.3 and 2 here, both ways) can make a stage's share 4 times as large:
6 * 4 * 8 * 2^-24 = 2^-16.4 of the 2-norm.  2^-13 is allowed; a stage rounded to bf16 is off by
2^-8 / sqrt(12) = 2^-9.8 of its own."""
import pytest
import torch

from test_linear_block_gpu import OFFSETS, buffers, make, step, views, whole

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", [60, 61])
def test_the_whole_in_fp32(seed):
    t = make(torch.float32, seed)
    b, raw = buffers(t), []
    step(t, b, 1.0, raw)
    w = views(t, dict(b, dx=raw[0], flat=raw[1]))
    o, grads = whole(t)
    o = o.detach()
    got = dict(q=w["dq"], k=w["dk"], v=w["dv"], g=w["dg"], q_gamma=w["params"][0], k_gamma=w["params"][1],
               q_beta=w["params"][2], k_beta=w["params"][3])
    a, e = OFFSETS[0], OFFSETS[-1]
    pairs = dict({name: (y, grads[name]) for name, y in got.items()}, o=(b["o"][a:e], o[a:e]))
    for name, (y, want) in pairs.items():
        off, size = (y.double() - want).norm(), want.norm()
        print(f"{name}: {float(off / size):.3g}", flush=True)
        assert off <= 2.0 ** -13 * size, f"{name}: {float(off / size):.3g}"
