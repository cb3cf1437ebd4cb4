"""CPU tests of the largest launches of the fused and expert products and of
routing: a grid of 2^32 threads or more is refused, by the call and before its
workspace is asked for."""
import ctypes

import pytest

import unstructured_sparse_weight_amd as usw
from test_abi_fused import P, UNSUPPORTED, WORKSPACE, bank, experts, fmt, fused, route

pytestmark = pytest.mark.host_pointers


def test_fused():
    """65536 strips in 256 splits; half of them on the per-wave kernel are allowed, and lack a workspace."""
    f = fmt(M=1 << 22, K=1 << 16, nnz=1 << 20)
    assert fused(f=f, N=1, splits=256) == UNSUPPORTED
    f = fmt(M=1 << 22, K=1 << 16, val_type=2, nnz=1 << 20)
    assert fused(f=f, N=1, splits=256) == UNSUPPORTED
    assert fused(f=f, N=1, splits=128) == WORKSPACE


def test_experts():
    """1024 tiles by 65536 strips."""
    f = bank(E=1024, M=1 << 22, K=64, values_bytes=1 << 20)
    assert experts(f=f, S=1024, T=1024) == UNSUPPORTED


@pytest.mark.parametrize("T,want", [((1 << 28) - 64, WORKSPACE), ((1 << 28) - 63, UNSUPPORTED), (1 << 30, UNSUPPORTED)])
def test_route(T, want):
    assert route(T=T, E=1, k=1) == want
    need = ctypes.c_size_t()
    st = usw.lib().usw_expert_route_workspace(T, 1, 1, ctypes.byref(need))
    assert st == (UNSUPPORTED if want == UNSUPPORTED else 0)
