"""zm_grad_norm with its workspace over a tensor, whose elements would be overwritten before they are
read: refused on the host (the pointers here are never read: each call ends at a refusal)."""
import ctypes
import os

import pytest

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.skipif(not os.path.exists(zm.LIB_PATH),
                                reason="libzmttt.so not built (run the build first)")
WS = 1 << 30
NEED = 8192  # of up to 127 tensors


def norm(x, n, dtype=zm.F32, first=(1 << 20, 4)):
    t = (zm.Tensor * 2)(zm.Tensor(first[0], None, first[1], zm.F32, 0), zm.Tensor(x, None, n, dtype, 0))
    return zm.load_library().zm_grad_norm(t, 2, ctypes.c_void_p(1 << 21), ctypes.c_void_p(WS), NEED, None)


@pytest.mark.parametrize("x,n,dtype", [
    (WS, 1, zm.F32), (WS - 4, 2, zm.F32), (WS + NEED - 4, 1, zm.F32), (WS + NEED - 2, 1, zm.BF16),
    (WS - (1 << 20), 1 << 30, zm.BF16), (WS - 2, 2, zm.BF16)])
def test_workspace_over_a_tensor(x, n, dtype):
    assert zm.grad_norm_workspace_size(2) == NEED
    assert norm(x, n, dtype) == zm.ERR_INVALID_ARG
    assert norm(1 << 22, 4, first=(WS + 64, 4)) == zm.ERR_INVALID_ARG
