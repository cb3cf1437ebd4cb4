"""CPU tests of the workspace that the fused and expert products share on a
stream: whatever the order of the calls, the leading counter bytes that a call
asks for are zero when it starts."""
import random

import pytest

from unstructured_sparse_weight_amd import _lib, fused

torch = pytest.importorskip("torch")

KEPT = 1 << 16   # bytes that a call without counters leaves alone


@pytest.fixture
def workspace(monkeypatch):
    monkeypatch.setattr(fused, "_WS", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return lambda need, cb: fused._workspace(torch.device("cpu"), 0, need, cb)


def call(workspace, need, cb):
    """What a product does with its workspace: finds its counters zero, leaves
    them zero and writes sums or weights behind them."""
    ws = workspace(need, cb)
    assert ws.numel() >= need
    assert not ws[:cb].any(), f"{int(ws[:cb].count_nonzero())} of {cb} counter bytes are not zero"
    ws[max(cb, KEPT):need] = 0xA5


def test_many_counters_after_an_expanded_weight(workspace):
    """More than 64 KiB of counters, a call without any, and the first again."""
    call(workspace, 1 << 20, 0)
    for _ in range(2):
        call(workspace, 200000, 69632)
        call(workspace, 300000, 0)
    call(workspace, 200000, 69632)


@pytest.mark.parametrize("seed", range(20))
def test_any_order_of_calls(workspace, seed):
    rng = random.Random(seed)
    for _ in range(60):
        cb = rng.choice([0, 0, KEPT, KEPT, KEPT + 256, 69632, 116992, 262144])
        call(workspace, max(cb, KEPT) + 256 * rng.randint(1, 2000), cb)


@pytest.mark.parametrize("M,K", [(64, 64), (256, 5120), (2048, 512), (20480, 5120), (1 << 20, 512), ((1 << 20) + 1024, 512)])
@pytest.mark.parametrize("val", [_lib.USW_VAL_F16, _lib.USW_VAL_I4])
@pytest.mark.parametrize("N", [1, 16, 77, 300, 4000])
def test_the_library_asks_for_none_or_64_kib(M, K, val, N):
    """The rule that the shared workspace rests on."""
    for splits in (0, 2):
        need, cb = fused._fused_sizes(M, K, 64, 64, val, M * K // 2, N, splits)
        assert cb == 0 or KEPT <= cb < need
        assert need == 0 or need > KEPT
    for E in (1, 8, 128):
        need, cb = fused._expert_sizes(E, M, K, val, E * M * K // 2, E * M * K, N)
        assert cb == 0 or KEPT <= cb < need
        assert need == 0 or need > KEPT


def test_release(workspace):
    """Released workspaces are made again, their counters zero."""
    call(workspace, 300000, 69632)
    assert len(fused._WS) == 1
    fused.release_workspaces()
    assert not fused._WS
    call(workspace, 200000, 69632)
    fused.release_workspaces()
    fused.release_workspaces()
