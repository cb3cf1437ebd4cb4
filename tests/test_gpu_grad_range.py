"""GPU tests of gated gradients whose dg is beyond fp16 under masks that keep a part
of the weights: every dx of the row is infinite or a NaN, so a scaled loss is seen to
overflow, and rows without such a dg are as without them."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

import unstructured_sparse_weight_amd as usw  # noqa: E402

DEV = "cuda:0"
M, K = 128, 192


@pytest.mark.parametrize("dtype", ["f16", "i4"])
@pytest.mark.parametrize("density", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("N", [3, 32, 33, 64, 128, 200])
def test_overflow_shows(N, density, dtype):
    r = torch.Generator(device=DEV).manual_seed(41)
    W = torch.randint(1, 8, (M, K), generator=r, device=DEV).half()
    mask = torch.rand(M, K, generator=r, device=DEV) < density
    up = usw.encode_device(W, mask, dtype=dtype)
    x = torch.ones(N, K, dtype=torch.float16, device=DEV)
    g = torch.ones(N, M, dtype=torch.float16, device=DEV)
    u, dy = g * 2, g * 0.5
    want = usw.spmm_gated_backward(up, up, x, g, u, dy, act="none", bias=True)
    u[1, 7], dy[1, 7] = 4096.0, 4096.0   # dg = 2^24
    got = usw.spmm_gated_backward(up, up, x, g, u, dy, act="none", bias=True)
    rest = torch.arange(N, device=DEV) != 1
    if dtype == "i4" and not density:   # INT4's scales, all 0 here, meet dg in fp32
        assert bool((got.x == 0).all())
    else:
        assert not bool(torch.isfinite(got.x[1]).any()) and torch.equal(got.x[rest], want.x[rest])
    # fp32 sums of dg as it is: from 2^24 on their step is 2, so each of N - 1 additions of 1 is off by at most 1.
    assert abs(float(got.gate_bias[7]) - (2.0 ** 24 + N - 1)) <= N - 1
    if dtype == "f16" and density:
        row = mask[7].sum()
        assert int(torch.isinf(got.gate).sum()) == int(row) and not bool(torch.isnan(got.gate).any())
