"""Long sequences of one head: segments of three chunks, and of more where 512 workgroups take fewer,
against the same tokens in two calls that carry the state, whose segments are others."""
import pytest
import torch

import reconstruction_lact_chunk_amd as zm
from linear_reference import chunks, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,dtype", [(26_000, torch.bfloat16), (33_001, torch.bfloat16), (13_007, torch.float32),
                                     (60_011, torch.float32)])
def test_in_two_calls(n, dtype):
    print(f"case linear one head n={n} {dtype}", flush=True)
    x = inputs(n, 1, 1, 64, dtype, n, decay=0.01)
    gen = torch.Generator(device="cuda").manual_seed(1)
    do = torch.randn(x["v"].shape, generator=gen, device="cuda").to(dtype)
    dstate = torch.randn(x["state"].shape, generator=gen, device="cuda")
    cut = n // 3 + 5
    halves = [{k: t if k == "state" else t[a:b] for k, t in x.items()} for a, b in ((0, cut), (cut, n))]
    args = [[y[k] for k in ("q", "k", "v", "g")] for y in (x, *halves)]
    o, end = zm.linear_attention(*args[0], state=x["state"])
    o1, mid = zm.linear_attention(*args[1], state=x["state"])
    o2, end2 = zm.linear_attention(*args[2], state=mid)
    grads = zm.linear_attention_backward(do, *args[0], state=x["state"], dstate=dstate)
    late = zm.linear_attention_backward(do[cut:], *args[2], state=mid, dstate=dstate)
    early = zm.linear_attention_backward(do[:cut], *args[1], state=x["state"], dstate=late[4])
    pairs = dict(o=(o, torch.cat([o1, o2])), end=(end, end2), dstate=(grads[4], early[4]))
    for i, name in enumerate(("dq", "dk", "dv", "dg")):
        pairs[name] = (grads[i], torch.cat([early[i], late[i]]))
    # Both sides are off by the roundings of linear_reference.py, of random signs: sqrt(64) for each of the
    # chunks within a state's reach (a decay of 0.007 a token forgets in some 150: 16 are ample), and twice as many
    # in a gradient; dg's sum of terms of all signs over that reach is smaller than they are by 2^5
    # (sqrt of 150 tokens' and 64 columns' terms and more); outputs' own rounding on top, on both sides.
    reach = min(chunks(n, dtype), 16)
    for name, (y, z) in pairs.items():
        y, z = y.double(), z.double()
        tol = 2 * 8 * 2 * (reach + 2) * 2.0 ** -24 * (2 ** 5 if name == "dg" else 4)
        if dtype == torch.bfloat16 and name in ("o", "dq", "dk", "dv"):
            tol += 2 * 2.0 ** -8 / 12 ** 0.5
        off = float((y - z).norm() / z.norm())
        print(f"{name}: {off:.3g} of {tol:.3g}", flush=True)
        assert off <= tol, name
