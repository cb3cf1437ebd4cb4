"""GPU test of the fused and expert products on the LDS-poisoning debug build:
every kernel fills its LDS staging buffers with NaNs at entry, so a read of LDS
that no stage wrote would put NaN into Y; on integer-exact inputs the results
must be bitwise right.  The debug library is called through the binding."""
import ctypes
import os
import sys

import numpy as np
import pytest

import workloads as wl

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

import unstructured_sparse_weight_amd as usw  # noqa: E402
from unstructured_sparse_weight_amd import _lib, fused  # noqa: E402
from unstructured_sparse_weight_amd import build as _build  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(scope="module")
def dbg():
    if not os.path.exists(_build.DEBUG_LIB):
        pytest.fail(f"{_build.DEBUG_LIB} is missing: build() compiles it beside libusw.so")
    return _lib._declare(ctypes.CDLL(_build.DEBUG_LIB))


def exact(M, K, density, i4, seed):
    rng = np.random.default_rng(seed)
    mask = wl.mask_bernoulli(M, K, density, rng)
    W = wl.weight_int4_exact(M, K, rng, mask) if i4 else wl.weight_dyadic(M, K, rng)
    return usw.encode(W, mask, dtype="i4" if i4 else "f16", device=DEV), np.where(mask, W, np.float16(0)).astype(np.float64)


# The ring kernel, the per-wave kernel (more rows, denser, INT4), with splits;
# expanded: small, medium and large tiles, columns that end a ring early.
CASES = [(512, 1024, 8, 0.5, False, 3), (256, 512, 40, 0.5, False, 0), (256, 512, 9, 0.9, False, 0),
         (256, 512, 9, 0.5, True, 2), (256, 512, 60, 0.5, True, 0), (256, 512, 77, 0.5, False, 1),
         (256, 1088, 90, 0.9, False, 2), (256, 512, 120, 0.5, True, 1), (192, 64, 70, 0.5, False, 0),
         (192, 320, 200, 0.7, True, 0), (2624, 832, 2050, 0.5, False, 0), (4096, 768, 4096, 0.5, False, 0)]


@pytest.mark.parametrize("M,K,N,density,i4,splits", CASES)
def test_fused(dbg, monkeypatch, M, K, N, density, i4, splits):
    enc, Wd = exact(M, K, density, i4, 400 + N)
    rng = np.random.default_rng(401)
    x = wl.activations_small_int(N, K, rng)
    res = rng.integers(-8, 9, size=(N, M)).astype(np.float16)
    print(f"[poison] fused {M}x{K} N={N} {density} i4={i4}", file=sys.stderr, flush=True)
    monkeypatch.setattr(fused, "lib", lambda: dbg)
    y = usw.spmm_fused(enc, torch.from_numpy(x).to(DEV), act="relu", residual=torch.from_numpy(res).to(DEV),
                       out_dtype=torch.float32, splits=splits).cpu().numpy().astype(np.float64)
    r = np.unique(np.concatenate([rng.integers(0, N, 60), [0, N - 1]]))
    assert not np.isnan(y).any()
    assert np.array_equal(y[r], np.maximum(x[r].astype(np.float64) @ Wd.T, 0) + res[r])


@pytest.mark.parametrize("counts", [[3, 0, 20], [150, 300, 0, 240]])
@pytest.mark.parametrize("i4", [False, True])
def test_experts(dbg, monkeypatch, counts, i4):
    M, K = 192, 320
    made = [exact(M, K, 0.5, i4, 410 + e) for e in range(len(counts))]
    bank = usw.expert_bank([m[0] for m in made])
    slots = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x = wl.activations_small_int(int(slots[-1]), K, np.random.default_rng(411))
    print(f"[poison] experts {counts} i4={i4}", file=sys.stderr, flush=True)
    monkeypatch.setattr(fused, "lib", lambda: dbg)
    y = usw.expert_spmm(bank, torch.from_numpy(x).to(DEV), torch.from_numpy(slots).to(DEV), out_dtype=torch.float32)
    y = y.cpu().numpy().astype(np.float64)
    assert not np.isnan(y).any()
    for e, (_, Wd) in enumerate(made):
        a, b = slots[e], slots[e + 1]
        assert np.array_equal(y[a:b], x[a:b].astype(np.float64) @ Wd.T)
