"""Calls of the sequence operators that have to end in a ZmError and not in Python's own."""
import os

import pytest
import torch

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.skipif(not os.path.exists(zm.LIB_PATH),
                                reason="libzmttt.so not built (run the build first)")


@pytest.mark.parametrize("n", [0, 4])
def test_heads_of_no_elements(n):
    q, g = torch.zeros(n, 2, 0), torch.zeros(n, 2)
    for call in (lambda: zm.delta_rule(q, q, q, g, g), lambda: zm.delta_rule_step(q, q, q, g, g, torch.zeros(n, 2, 0, 0)),
                 lambda: zm.delta_rule_backward(q, q, q, q, g, g)):
        with pytest.raises(zm.ZmError, match="no elements"):
            call()


@pytest.mark.parametrize("dtype", [torch.float16, torch.int32])
def test_layer_norm_workspace_of_another_type(dtype):
    with pytest.raises(zm.ZmError, match="bf16 or fp32"):
        zm.layer_norm_backward_workspace_size(4, 64, dtype)
