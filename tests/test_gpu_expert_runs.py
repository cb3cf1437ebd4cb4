"""GPU test of the product by expert on offsets that no router makes: runs that
overlap, fall, or lie outside the slots.  They may give any rows, but nothing
may be written outside the workspace and Y, the counters end at zero, and the
expanded product takes an offset below one before it for that one.  The calls
go through the C ABI, with a workspace and a Y between guard bytes."""
import ctypes
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

import unstructured_sparse_weight_amd as usw  # noqa: E402
from unstructured_sparse_weight_amd import USW_OUT_F32  # noqa: E402

DEV = "cuda:0"
GUARD = 1 << 20

# E, M, K, S: expanded by small tiles in splits, small ones whole, medium ones
# in splits, large ones; and not expanded, whole and in splits.
SHAPES = {"small, split": (16, 64, 4096, 3584), "small": (4, 192, 320, 700), "medium, split": (4, 512, 8256, 1000),
          "large": (4, 2560, 5120, 6600), "passes": (6, 192, 256, 90), "passes, split": (6, 128, 4160, 30)}


def offsets_of(kind, E, S):
    if kind == "alternating":
        return [0 if e % 2 == 0 else S for e in range(E + 1)]
    if kind == "falling":
        return [S - S * e // E for e in range(E + 1)]
    if kind == "outside":
        return [[-7, S + 9, -(1 << 31), (1 << 31) - 1][e % 4] for e in range(E + 1)]
    if kind == "one step back":
        up = [S * e // E for e in range(E + 1)]
        up[E // 2] = up[E // 2 - 1] // 2
        return up
    assert kind == "beyond"
    return [S + 100 * e for e in range(E + 1)]


def guarded(nbytes):
    whole = torch.full((nbytes + 2 * GUARD,), 0xA5, dtype=torch.uint8, device=DEV)
    return whole, whole[GUARD:GUARD + nbytes]


@pytest.mark.parametrize("what", list(SHAPES))
@pytest.mark.parametrize("kind", ["alternating", "falling", "outside", "one step back", "beyond"])
def test_offsets_out_of_order(what, kind):
    E, M, K, S = SHAPES[what]
    g = torch.Generator(device=DEV).manual_seed(E + M)
    W = torch.randint(-3, 4, (E, M, K), device=DEV, generator=g).half()
    mask = torch.rand(E, M, K, device=DEV, generator=g) < 0.4
    W = torch.where(mask, W, 0)
    bank = usw.expert_bank([usw.encode_device(W[e], mask[e]) for e in range(E)])
    x = torch.randint(-4, 5, (S, K), device=DEV, generator=g).half()
    offsets = np.array(offsets_of(kind, E, S), dtype=np.int64)
    slots = torch.from_numpy(offsets.astype(np.int32)).to(DEV)
    L, f = usw.lib(), bank.fmt()
    need, cb = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.usw_expert_spmm_workspace(ctypes.byref(f), S, ctypes.byref(need), ctypes.byref(cb)) == 0
    assert (cb.value > 0) == (what in ("small, split", "medium, split", "large", "passes, split"))
    expanded = not what.startswith("passes")
    ws_whole, ws = guarded(need.value)
    ws[:cb.value].zero_()
    y_whole, yb = guarded(4 * S * M)
    print(f"[runs] {what} {kind}", file=sys.stderr, flush=True)
    for _ in range(2):
        st = L.usw_expert_spmm(ctypes.byref(f), x.data_ptr(), S, slots.data_ptr(), None, S, yb.data_ptr(), USW_OUT_F32,
                               None, ws.data_ptr() if need.value else None, need.value,
                               torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()
        for whole in (ws_whole, y_whole):
            assert bool((whole[:GUARD] == 0xA5).all()) and bool((whole[-GUARD:] == 0xA5).all())
        assert not ws[:cb.value].any()
    if expanded:
        y = yb.view(torch.float32).view(S, M)
        untouched = torch.full((1,), 0xA5A5A5A5 - (1 << 32), dtype=torch.int32, device=DEV).view(torch.float32)
        want = untouched.expand(S, M).contiguous()
        ends = np.maximum.accumulate(np.clip(offsets, 0, S))
        for e in range(E):
            a, b = int(ends[e]), int(ends[e + 1])
            if b > a:
                want[a:b] = x[a:b].float() @ W[e].float().t()
        assert torch.equal(y, want)
