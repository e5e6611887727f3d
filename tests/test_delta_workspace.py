"""A workspace of the gated delta rule for some number of tokens serves every smaller one."""
import os

import pytest

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.skipif(not os.path.exists(zm.LIB_PATH),
                                reason="libzmttt.so not built (run the build first)")
SIZES = [zm.delta_rule_workspace_size, zm.delta_rule_backward_workspace_size]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [zm.BF16, zm.F32])
@pytest.mark.parametrize("heads,heads_k,d", [(8, 8, 128), (1, 1, 64), (3, 1, 128), (64, 16, 64), (60, 60, 64)])
@pytest.mark.parametrize("n_seq", [1, 2, 15, 17, 130])
def test_the_size_never_decreases(n_seq, heads, heads_k, d, dtype, size):
    desc = zm.DeltaDesc(heads, heads_k, d, dtype, n_seq, 1.0, heads_k * d, heads_k * d, heads * d, heads * d)
    # every length of the first segments, then each side of a chunk's end, then far ones
    lengths = list(range(0, 700)) + [64 * c + e for c in range(10, 700) for e in (0, 1)]
    lengths += [64 * c for c in range(700, 4000, 7)]
    sizes = [size(desc, n) for n in sorted(lengths)]
    assert sizes == sorted(sizes)
