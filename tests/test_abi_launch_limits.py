"""CPU tests of the largest launches of the gated block, the gradients, the 4-bit
and the fused product: one of 2^32 threads, HIP's limit, is refused by the call and
by the query of its workspace."""
import ctypes

import pytest

import unstructured_sparse_weight_amd as usw
from test_abi_block import BIG, UNSUPPORTED, WORKSPACE, back, fmt, gated, matmul, w4
from test_abi_fused import fmt as fused_fmt
from test_abi_fused import fused

pytestmark = pytest.mark.host_pointers

TALL = dict(M=1 << 20, K=64)


def query(name, *args):
    need, cb = ctypes.c_size_t(), ctypes.c_size_t()
    return getattr(usw.lib(), name)(*args, ctypes.byref(need), ctypes.byref(cb))


@pytest.mark.parametrize("N,want", [(1 << 21, UNSUPPORTED), ((1 << 21) - 63, UNSUPPORTED), ((1 << 21) - 64, 0)])
def test_many_rows_values(N, want):
    """d's pass takes x's transpose along: 64 tokens by 64 columns of either to 256 threads."""
    f = fmt(M=1 << 14, K=1 << 14)
    at = ctypes.byref(f)
    assert query("usw_spmm_backward_workspace", at, N, 1, 2, ) == want
    assert query("usw_spmm_backward_workspace", at, N, 1, 7) == want
    assert query("usw_spmm_gated_backward_workspace", at, at, N, 3) == want
    assert query("usw_spmm_backward_workspace", at, N, 1, 5) == 0   # no values: no transpose
    assert back(f=f, N=N) == (want or WORKSPACE)


@pytest.mark.parametrize("N,want", [(1 << 17, UNSUPPORTED), (1 << 16, 0)])
def test_gated(N, want):
    """Both weights as one of 2^21 outputs: 2^24 tiles of 128 x 128."""
    f = fmt(**TALL)
    at = ctypes.byref(f)
    assert query("usw_spmm_gated_workspace", at, at, N) == want
    assert gated(gate=f, up=f, N=N, ws=8, ws_bytes=0 if want == 0 else BIG) == (want or WORKSPACE)


@pytest.mark.parametrize("N,want", [(1 << 18, UNSUPPORTED), (1 << 17, 0)])
def test_4_bit(N, want):
    f = w4(**TALL)
    assert query("usw_w4_matmul_workspace", ctypes.byref(f), N) == want
    assert matmul(f=f, N=N) == (want or WORKSPACE)


@pytest.mark.parametrize("N,want", [(1 << 18, UNSUPPORTED), (1 << 17, WORKSPACE)])
def test_fused(N, want):
    assert fused(f=fused_fmt(**TALL), N=N, splits=0) == want
