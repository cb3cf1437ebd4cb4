"""CPU tests of the argument checks of the products with an epilogue, of
routing and of the combine: every refusal comes before anything is launched.
Pointers are host buffers that nothing may touch."""
import ctypes

import numpy as np
import pytest

import unstructured_sparse_weight_amd as usw
from unstructured_sparse_weight_amd import _lib

pytestmark = pytest.mark.host_pointers

NULL_ARG, BAD_SHAPE, BAD_DTYPE, BAD_N, UNSUPPORTED, MISALIGNED, WORKSPACE = -1, -2, -3, -4, -5, -6, -7
_BUF = np.zeros(1 << 20, dtype=np.uint8)
P = (_BUF.ctypes.data + 63) & ~63
M, K = 128, 256


def fmt(**kw):
    d = dict(M=M, K=K, gt_m=64, gt_k=64, val_type=1, reserved=0, nnz=100, bitmaps=P, offsets=P, values=P, scales=P)
    d.update(kw)
    return _lib.UswFmt(*[d[n] for n, _ in _lib.UswFmt._fields_])


def ep(**kw):
    d = dict(bias=None, mul=None, res=None, ld_mul=0, ld_res=0, act=0, reserved=0)
    d.update(kw)
    return _lib.UswEpilogue(*[d[n] for n, _ in _lib.UswEpilogue._fields_])


def fused(f=None, X=P, Y=P, yt=1, N=4, e=None, splits=1, ws=None, ws_bytes=0):
    f = f or fmt()
    return usw.lib().usw_spmm_fused(ctypes.byref(f), X, Y, yt, N, ctypes.byref(e) if e else None, splits, ws,
                                    ws_bytes, None)


@pytest.mark.parametrize("want,kw", [
    (BAD_SHAPE, dict(f=fmt(M=100))), (BAD_SHAPE, dict(f=fmt(K=0))), (BAD_SHAPE, dict(f=fmt(reserved=1))),
    (BAD_DTYPE, dict(f=fmt(val_type=3))), (BAD_DTYPE, dict(yt=2)), (BAD_N, dict(N=0)), (BAD_N, dict(N=-3)),
    (UNSUPPORTED, dict(f=fmt(gt_m=32))), (NULL_ARG, dict(X=None)), (NULL_ARG, dict(Y=None)),
    (NULL_ARG, dict(f=fmt(bitmaps=None))), (NULL_ARG, dict(f=fmt(offsets=None))), (NULL_ARG, dict(f=fmt(values=None))),
    (NULL_ARG, dict(f=fmt(val_type=2, scales=None))), (MISALIGNED, dict(X=P + 2)), (MISALIGNED, dict(Y=P + 8)),
    (MISALIGNED, dict(f=fmt(val_type=2, scales=P + 8))), (MISALIGNED, dict(f=fmt(offsets=P + 2))),
    (BAD_DTYPE, dict(e=ep(act=5))), (BAD_DTYPE, dict(e=ep(act=-1))), (BAD_SHAPE, dict(e=ep(reserved=1))),
    (MISALIGNED, dict(e=ep(bias=P + 8))), (MISALIGNED, dict(e=ep(mul=P + 2))), (MISALIGNED, dict(e=ep(res=P + 8))),
    (BAD_SHAPE, dict(e=ep(mul=P, ld_mul=M - 8))), (BAD_SHAPE, dict(e=ep(res=P, ld_res=-8))),
    (MISALIGNED, dict(e=ep(res=P, ld_res=M + 4))), (BAD_SHAPE, dict(e=ep(mul=P, ld_mul=(1 << 20) + 8))),
])
def test_fused_refuses(want, kw):
    assert fused(**kw) == want


def test_fused_workspace_is_asked_for():
    L = usw.lib()
    f = fmt(M=64, K=64 * 64, nnz=64 * 64 * 32)
    need, cb = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.usw_spmm_fused_workspace(ctypes.byref(f), 4, 4, ctypes.byref(need), ctypes.byref(cb)) == 0
    assert need.value > cb.value > 0
    assert fused(f=f, splits=4) == WORKSPACE
    assert fused(f=f, splits=4, ws=P, ws_bytes=need.value - 1) == WORKSPACE
    assert fused(f=f, splits=4, ws=P + 4, ws_bytes=need.value) == MISALIGNED
    assert L.usw_spmm_fused_workspace(ctypes.byref(f), 0, 1, ctypes.byref(need), ctypes.byref(cb)) == BAD_N
    assert L.usw_spmm_fused_workspace(None, 4, 1, ctypes.byref(need), ctypes.byref(cb)) == NULL_ARG
    assert L.usw_spmm_fused_workspace(ctypes.byref(f), 4, 1, None, ctypes.byref(cb)) == NULL_ARG


def bank(**kw):
    d = dict(E=3, M=M, K=K, val_type=1, reserved=0, nnz=100, values_bytes=16 * 64, bitmaps=P, offsets=P, values=P,
             starts=P, scales=P)
    d.update(kw)
    return _lib.UswExpertFmt(*[d[n] for n, _ in _lib.UswExpertFmt._fields_])


def experts(f=None, X=P, T=4, slots=P, rows=P, S=6, Y=P, yt=1, e=None, ws=None, ws_bytes=0):
    f = f or bank()
    return usw.lib().usw_expert_spmm(ctypes.byref(f), X, T, slots, rows, S, Y, yt, ctypes.byref(e) if e else None, ws,
                                     ws_bytes, None)


@pytest.mark.parametrize("want,kw", [
    (BAD_SHAPE, dict(f=bank(M=96))), (BAD_SHAPE, dict(f=bank(E=0))), (UNSUPPORTED, dict(f=bank(E=1025, values_bytes=1 << 20))),
    (BAD_SHAPE, dict(f=bank(reserved=2))), (BAD_DTYPE, dict(f=bank(val_type=3))), (BAD_DTYPE, dict(yt=0)),
    (BAD_N, dict(S=-1)), (BAD_N, dict(T=-1)), (BAD_N, dict(T=0)), (BAD_N, dict(rows=None)),
    (BAD_SHAPE, dict(f=bank(nnz=-1))), (BAD_SHAPE, dict(f=bank(nnz=3 * M * K + 1))), (BAD_SHAPE, dict(f=bank(values_bytes=32))),
    (BAD_SHAPE, dict(f=bank(values_bytes=16 * 64 + 8))), (NULL_ARG, dict(f=bank(starts=None))),
    (NULL_ARG, dict(f=bank(val_type=2, scales=None))), (NULL_ARG, dict(slots=None)), (NULL_ARG, dict(X=None)),
    (NULL_ARG, dict(Y=None)), (MISALIGNED, dict(slots=P + 2)), (MISALIGNED, dict(rows=P + 1)), (MISALIGNED, dict(Y=P + 4)),
    (MISALIGNED, dict(f=bank(starts=P + 4))), (BAD_DTYPE, dict(e=ep(act=9))), (MISALIGNED, dict(e=ep(bias=P + 4))),
])
def test_experts_refuse(want, kw):
    assert experts(**kw) == want


def test_experts_without_slots_do_nothing():
    assert experts(S=0, T=0, X=None, Y=None, rows=None) == 0
    need, cb = ctypes.c_size_t(5), ctypes.c_size_t(5)
    f = bank()
    assert usw.lib().usw_expert_spmm_workspace(ctypes.byref(f), 0, ctypes.byref(need), ctypes.byref(cb)) == 0
    assert need.value == cb.value == 0
    assert usw.lib().usw_expert_spmm_workspace(ctypes.byref(f), -1, ctypes.byref(need), ctypes.byref(cb)) == BAD_N


def route(logits=P, lt=3, ld=0, T=4, E=8, k=2, ids=P, weights=P, slots=P, rows=P, pos=P, ws=None, ws_bytes=0):
    return usw.lib().usw_expert_route(logits, lt, ld, T, E, k, 1, ids, weights, slots, rows, pos, ws, ws_bytes, None)


@pytest.mark.parametrize("want,kw", [
    (BAD_N, dict(T=-1)), (BAD_SHAPE, dict(E=0)), (BAD_SHAPE, dict(k=0)), (BAD_SHAPE, dict(k=9)), (BAD_SHAPE, dict(ld=7)),
    (UNSUPPORTED, dict(E=1025)), (UNSUPPORTED, dict(E=64, k=17)), (UNSUPPORTED, dict(T=(1 << 31) - 1, k=2)),
    (BAD_DTYPE, dict(lt=2)), (NULL_ARG, dict(logits=None)), (NULL_ARG, dict(ids=None)), (NULL_ARG, dict(weights=None)),
    (NULL_ARG, dict(slots=None)), (NULL_ARG, dict(rows=None)), (NULL_ARG, dict(pos=None)), (MISALIGNED, dict(logits=P + 2)),
    (MISALIGNED, dict(pos=P + 2)), (WORKSPACE, dict(T=300)), (WORKSPACE, dict(T=300, ws=P, ws_bytes=16)),
])
def test_route_refuses(want, kw):
    assert route(**kw) == want


def combine(Y=P, yt=1, S=4, M=64, pos=P, weights=P, T=2, k=2, res=None, ld=0, out=P, ot=1):
    return usw.lib().usw_expert_combine(Y, yt, S, M, pos, weights, T, k, res, ld, out, ot, None)


@pytest.mark.parametrize("want,kw", [
    (BAD_N, dict(T=-1)), (BAD_N, dict(S=-1)), (BAD_SHAPE, dict(M=0)), (BAD_SHAPE, dict(M=12)), (BAD_SHAPE, dict(k=0)),
    (BAD_SHAPE, dict(res=P, ld=56)), (BAD_DTYPE, dict(yt=2)), (BAD_DTYPE, dict(ot=0)), (NULL_ARG, dict(Y=None)),
    (NULL_ARG, dict(pos=None)), (NULL_ARG, dict(weights=None)), (NULL_ARG, dict(out=None)), (MISALIGNED, dict(Y=P + 8)),
    (MISALIGNED, dict(out=P + 8)), (MISALIGNED, dict(res=P + 2)), (MISALIGNED, dict(res=P, ld=68)),
])
def test_combine_refuses(want, kw):
    assert combine(**kw) == want


def test_combine_of_no_tokens():
    assert combine(T=0, Y=None, pos=None, weights=None, out=None, S=0) == 0
