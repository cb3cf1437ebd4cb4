"""GPU test of the activations' negative tails, where they are far smaller than
their argument: the error is bounded relative to the value itself.  Weights are
the identity, so the kernels' sums are x without any error."""
import math
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

import unstructured_sparse_weight_amd as usw  # noqa: E402

DEV = "cuda:0"
U = 2.0 ** -24


def exact(v, name):
    if name == "gelu":
        return np.array([0.5 * t * math.erfc(-t / math.sqrt(2)) for t in v])
    if name == "gelu_tanh":
        return v / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v / (1 + np.exp(-v))


def relative_bound(v, name):
    """Roundings up to the fp32 output, in units of U, relative to the value.

    GELU: the argument -v c is off by 2 (c's rounding and the product's), which
    erfc turns into at most 2 (v^2 + 2); erfc itself 32 (16 units in the last
    place, the most that the language allows it); two products.
    tanh GELU, SiLU: the exponent is off by at most 8 roundings relative to
    itself, hence the exponential by 8 |exponent| + 4; the sum below it, the
    reciprocal (2) and the product add at most 6.
    """
    if name == "gelu":
        return (2 * (v * v + 2) + 34) * U
    z = np.abs(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)) if name == "gelu_tanh" else np.abs(v)
    return (8 * z + 10) * U


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("N", [1, 40, 130])
@pytest.mark.parametrize("val", ["f16", "i4"])
def test_negative_tail(name, N, val):
    enc = usw.encode(np.eye(64, dtype=np.float16) * np.float16(0.875 if val == "i4" else 1.0), None, dtype=val, device=DEV)
    one = 0.875 if val == "i4" else 1.0            # a code of 7 and a scale of 1/8
    rng = np.random.default_rng(N)
    x = rng.uniform(-6.0, -2.0, size=(N, 64)).astype(np.float16)
    v = x.astype(np.float64) * one
    print(f"[tail] {name} N={N} {val}", file=sys.stderr, flush=True)
    y = usw.spmm_fused(enc, torch.from_numpy(x).to(DEV), act=name, out_dtype=torch.float32).cpu().numpy().astype(np.float64)
    want = exact(v.ravel(), name).reshape(v.shape)
    off, bound = np.abs(y - want), relative_bound(v, name) * np.abs(want)
    print(f"[tail] worst/bound={float((off / bound).max()):.3f}", file=sys.stderr, flush=True)
    assert np.all(off <= bound), float((off / bound).max())


def test_gelu_far_out():
    """Where erfc ends: zeros, infinities and NaN come out as from the formula's limit."""
    enc = usw.encode(np.eye(64, dtype=np.float16), None, device=DEV)
    v = np.zeros((2, 64), dtype=np.float16)
    v[0, :6] = [-10.0, -13.0, -20.0, -65504.0, 65504.0, 10.0]
    v[1] = np.nan
    y = usw.spmm_fused(enc, torch.from_numpy(v).to(DEV), act="gelu", out_dtype=torch.float32).cpu().numpy()
    assert abs(y[0, 0] / (-5 * math.erfc(10 / math.sqrt(2))) - 1) < 260 * U
    assert -1e-37 < y[0, 1] <= 0 and y[0, 2] == 0 and y[0, 3] == 0
    assert y[0, 4] == 65504.0 and y[0, 5] == 10.0 and np.all(y[0, 6:] == 0)
    assert np.isnan(y[1]).all()
