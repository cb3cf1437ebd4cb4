"""CPU test that the gated block and the gradients always ask for a workspace, as
their binding takes for granted, and refuse to go without."""
import ctypes

import pytest

import unstructured_sparse_weight_amd as usw
from test_abi_block import I4, WORKSPACE, back, fmt, gback, grad
from unstructured_sparse_weight_amd import _lib, gated

pytestmark = pytest.mark.host_pointers


@pytest.mark.parametrize("M,K", [(64, 64), (128, 256), (64, 1 << 14)])
@pytest.mark.parametrize("N", [1, 32, 33, 64, 65, 128, 129, 5000])
def test_never_zero(M, K, N):
    for val in (_lib.USW_VAL_F16, _lib.USW_VAL_I4):
        bare = (M, K, 64, 64, val, 0, M * K // 2)
        assert gated._gated_sizes(bare, bare, N)[0] > 0
        for grads in range(8):
            if grads & _lib.USW_GRAD_VALUES and val != _lib.USW_VAL_F16:
                continue
            assert gated._gated_backward_sizes(bare, bare, N, grads)[0] >= 1 << 16
            for out in (_lib.USW_OUT_F16, _lib.USW_OUT_F32):
                assert gated._backward_sizes(bare, N, out, grads)[0] >= 1 << 16


def test_without_one():
    """The bias of one chunk alone, and of nothing at all."""
    assert back(dX=None, dV=None) == WORKSPACE
    assert back(dX=None, dV=None, db=None) == WORKSPACE
    nothing = dict(dX=None, dgate_values=None, dup_values=None, dup_bias=None)
    assert gback(d=grad(**nothing)) == WORKSPACE
    assert gback(gate=fmt(**I4), up=fmt(**I4), d=grad(dgate_bias=None, **nothing)) == WORKSPACE
    need, cb = ctypes.c_size_t(), ctypes.c_size_t()
    f = fmt()
    assert usw.lib().usw_spmm_backward_workspace(ctypes.byref(f), 4, 1, 0, ctypes.byref(need), ctypes.byref(cb)) == 0
    assert need.value == 1 << 16 and cb.value == 0
