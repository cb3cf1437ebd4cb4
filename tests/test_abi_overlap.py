"""CPU tests that the gradients refuse outputs that overlap each other or what the
call reads: up to 64 rows the input's and the values' gradients are one launch, so
either may be stored while the other's operands are still read.  Pointers are host
buffers; every call here is refused before anything is launched."""
import ctypes

import numpy as np
import pytest

import unstructured_sparse_weight_amd as usw
from unstructured_sparse_weight_amd import _lib

pytestmark = pytest.mark.host_pointers

UNSUPPORTED = -5
M, K, N, NNZ = 128, 256, 4, 1000
_BUF = np.zeros(4 << 20, dtype=np.uint8)
_AT = (_BUF.ctypes.data + 63) & ~63
_WS = 1 << 20


class Places:
    """Addresses one behind the other, named, of the sizes the call reads or writes."""

    def __init__(self, i4):
        self.next = _AT
        sizes = dict(x=2 * N * K, dy=2 * N * M, g=2 * N * M, u=2 * N * M, dx=2 * N * K, dv0=2 * NNZ, dv1=2 * NNZ, db0=4 * M,
                     db1=4 * M, ws=_WS)
        for h in "01":
            sizes.update({"bitmaps" + h: M * K // 8, "offsets" + h: 4 * (M * K // 4096 + 1),
                          "values" + h: NNZ // 2 + 16 if i4 else 2 * NNZ + 16, "scales" + h: 2 * M})
        for name, size in sizes.items():
            setattr(self, name, self.next)
            self.next += (size + 15) // 16 * 16
        self.sizes = sizes

    def fmt(self, h, i4):
        return _lib.UswFmt(M, K, 64, 64, 2 if i4 else 1, 0, NNZ, getattr(self, "bitmaps" + h), getattr(self, "offsets" + h),
                           getattr(self, "values" + h), getattr(self, "scales" + h))


def single(p, i4=False, rows=N):
    f = p.fmt("0", i4)
    return usw.lib().usw_spmm_backward(ctypes.byref(f), p.x, p.dy, rows, p.dx, None if i4 else p.dv0, p.db0, 1, p.ws, _WS, None)


def pair(p, i4=False, rows=N):
    gate, up = p.fmt("0", i4), p.fmt("1", i4)
    d = _lib.UswGatedGrad(p.dy, p.g, p.u, p.dx, None if i4 else p.dv0, None if i4 else p.dv1, p.db0, p.db1, 4, 0)
    return usw.lib().usw_spmm_gated_backward(ctypes.byref(gate), ctypes.byref(up), p.x, rows, ctypes.byref(d), p.ws, _WS, None)


READ = ["x", "dy", "bitmaps0", "offsets0", "values0"]
OUT = ["dx", "dv0", "db0"]


@pytest.mark.parametrize("call,read,out", [
    (single, READ, OUT), (pair, READ + ["g", "u", "bitmaps1", "offsets1", "values1"], OUT + ["dv1", "db1"])])
def test_overlapping_outputs_are_refused(call, read, out):
    for o in out:
        for r in read + ["ws"] + [q for q in out if q != o]:
            p = Places(False)
            setattr(p, o, getattr(p, r))
            assert call(p) == UNSUPPORTED, (o, r)
            p = Places(False)   # the last 16 bytes of one, the first of the other
            setattr(p, o, getattr(p, r) + (p.sizes[r] - 1) // 16 * 16)
            assert call(p) == UNSUPPORTED, (o, r, "end")


def test_neighbours_are_taken():
    """The buffers of Places, each where the one before ends: the call goes on to launch, which fails without a GPU."""
    for call in (single, pair):
        for i4 in (False, True):
            assert call(Places(i4), i4) not in (UNSUPPORTED, 0)


def test_int4_scales_and_x():
    """INT4 has no values' gradient, so x is not read; its scales are."""
    for call in (single, pair):
        for o in ("dx", "db0"):
            p = Places(True)
            setattr(p, o, p.scales0)
            assert call(p, True) == UNSUPPORTED, o
