"""GPU tests of the gated block's gradients where a pre-activation is beyond fp16, so
that the g kept for them is infinite: the activation and its slope are their limits
there, 0 and 0 on the left, infinite and 1 on the right, as the forward pass, whose
g is fp32, has them."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

import unstructured_sparse_weight_amd as usw  # noqa: E402

DEV = "cuda:0"
M, K = 128, 64
ACTS = ["relu", "gelu", "gelu_tanh", "silu"]


def dense(W):
    return usw.encode_device(W, torch.ones_like(W, dtype=torch.bool))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N", [1, 20, 40, 200])
def test_far_left(N, act):
    """g = -131072 in every other output: nothing comes from there; the others are as without them."""
    x = torch.full((N, K), 64.0, dtype=torch.float16, device=DEV)
    Wg = torch.full((M, K), 2.0 ** -11, dtype=torch.float16, device=DEV)   # g = 2
    Wg[1::2] = -32.0
    Wu = torch.full((M, K), 2.0 ** -12, dtype=torch.float16, device=DEV)   # u = 1
    dy = torch.full((N, M), 0.5, dtype=torch.float16, device=DEV)
    gate, up = dense(Wg), dense(Wu)
    h, g, u = usw.spmm_gated(gate, up, x, act=act, save=True)
    assert bool((g[:, 1::2] == -float("inf")).all()) and bool((h[:, 1::2] == 0).all())
    got = usw.spmm_gated_backward(gate, up, x, g, u, dy, act=act, bias=True)
    near = g.clone()
    near[:, 1::2] = -65504.0
    want = usw.spmm_gated_backward(gate, up, x, near, u, dy, act=act, bias=True)
    for name in ("x", "gate", "up", "gate_bias", "up_bias"):
        a, b = getattr(got, name), getattr(want, name)
        assert bool(torch.isfinite(b).all()) and torch.equal(a, b), name
    assert bool((got.gate_bias[1::2] == 0).all()) and bool((got.up_bias[1::2] == 0).all())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N", [1, 20, 40, 200])
def test_far_right(N, act):
    """g = 131072: the slope is 1, so the gate's gradients are dy u x; the up weight's are infinite, as act(g) is."""
    x = torch.full((N, K), 64.0, dtype=torch.float16, device=DEV)
    gate = dense(torch.full((M, K), 32.0, dtype=torch.float16, device=DEV))
    up = dense(torch.full((M, K), 2.0 ** -22, dtype=torch.float16, device=DEV))   # u = 2^-10
    dy = torch.full((N, M), 0.5, dtype=torch.float16, device=DEV)
    h, g, u = usw.spmm_gated(gate, up, x, act=act, save=True)
    assert bool((g == float("inf")).all()) and bool((h == 128.0).all())
    got = usw.spmm_gated_backward(gate, up, x, g, u, dy, act=act, dx=False, bias=True)
    assert bool((got.gate == N * 64.0 * 2.0 ** -11).all()) and bool((got.gate_bias == N * 2.0 ** -11).all())
    assert bool((got.up == float("inf")).all()) and bool((got.up_bias == float("inf")).all())


@pytest.mark.parametrize("act", ACTS[1:])
def test_nan(act):
    """A NaN stays one."""
    x = torch.ones(3, K, dtype=torch.float16, device=DEV)
    gate = up = dense(torch.ones(M, K, dtype=torch.float16, device=DEV))
    one = torch.ones(3, M, dtype=torch.float16, device=DEV)
    g = one.clone()
    g[1, 5] = float("nan")
    got = usw.spmm_gated_backward(gate, up, x, g, one, one, act=act, bias=True)
    for b in (got.gate_bias, got.up_bias):
        assert bool(torch.isnan(b[5])) and int(torch.isnan(b).sum()) == 1
    assert bool(torch.isnan(got.x[1]).all()) and bool(torch.isfinite(got.x[0]).all())
