"""CPU tests of the epilogue operands' strides on weights of more than 2^20
outputs, which only the decode passes take.  A call that gets past its argument
checks is stopped by the workspace that it lacks; pointers are host buffers
that nothing may touch."""
import ctypes

import pytest

from test_abi_fused import BAD_SHAPE, P, UNSUPPORTED, WORKSPACE, bank, ep, experts, fmt, fused

pytestmark = pytest.mark.host_pointers

TALL = (1 << 20) + 64


@pytest.mark.parametrize("M,ld,want", [
    (TALL, 0, WORKSPACE), (TALL, TALL, WORKSPACE), (TALL, TALL + 8, WORKSPACE), (TALL, 1 << 22, WORKSPACE),
    (TALL, (1 << 22) + 8, BAD_SHAPE), (TALL, TALL - 64, BAD_SHAPE), (1 << 22, 0, WORKSPACE),
    (1 << 20, 0, WORKSPACE), (1 << 20, (1 << 20) + 8, BAD_SHAPE), ((1 << 22) + 64, 0, UNSUPPORTED),
    ((1 << 22) + 64, 1 << 23, UNSUPPORTED),
])
@pytest.mark.parametrize("which", ["mul", "res"])
def test_fused(M, ld, want, which):
    f = fmt(M=M, K=2560, nnz=1 << 20)
    assert fused(f=f, splits=2, e=ep(**{which: P, "ld_" + which: ld})) == want


@pytest.mark.parametrize("ld,want", [(0, WORKSPACE), (TALL + 8, WORKSPACE), ((1 << 22) + 8, BAD_SHAPE)])
def test_by_expert(ld, want):
    f = bank(M=TALL, K=4160, nnz=1 << 20)      # more columns than one workgroup takes: split
    assert experts(f=f, e=ep(mul=P, ld_mul=ld)) == want
