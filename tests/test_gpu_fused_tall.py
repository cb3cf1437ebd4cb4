"""GPU test of the epilogue's operands on weights of more than 2^20 outputs:
a vocabulary's worth of rows several times over, mul and residual with the
default stride and a longer one, Y over the residual."""
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

import unstructured_sparse_weight_amd as usw  # noqa: E402

DEV = "cuda:0"
M, K = (1 << 20) + 64, 128


def integers(g, *shape, top=3):
    return torch.randint(-top, top + 1, shape, device=DEV, generator=g).half()


def weight(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    mask = torch.rand(M, K, device=DEV, generator=g) < 0.4
    W = integers(g, M, K)
    return usw.encode_device(W, mask), torch.where(mask, W, 0).float()


@pytest.mark.parametrize("N", [1, 3, 40, 150])
def test_operands(N):
    """Whole numbers below 2^24 throughout: exact in fp32."""
    enc, W = weight(1)
    g = torch.Generator(device=DEV).manual_seed(N)
    x, wide = integers(g, N, K), integers(g, N, M + 192)
    mul, res = wide[:, :M], wide[:, 192:]
    print(f"[tall] N={N}", file=sys.stderr, flush=True)
    want = x.float() @ W.t() * mul.float() + res.float()
    assert torch.equal(usw.spmm_fused(enc, x, mul=mul, residual=res, out_dtype=torch.float32), want)
    mul, res = mul.clone(), res.clone()      # one row of wide is contiguous already, and Y may not overlap mul
    assert torch.equal(usw.spmm_fused(enc, x, mul=mul, residual=res, out_dtype=torch.float32), want)
    y = usw.spmm_fused(enc, x, mul=mul, residual=res, y=res)
    assert y.data_ptr() == res.data_ptr() and torch.equal(y, want.half())


def test_by_expert():
    made = [weight(2), weight(3)]
    bank = usw.expert_bank([m[0] for m in made])
    g = torch.Generator(device=DEV).manual_seed(4)
    x, mul = integers(g, 7, K), integers(g, 7, M)
    slots = torch.tensor([0, 2, 7], dtype=torch.int32, device=DEV)
    print("[tall] by expert", file=sys.stderr, flush=True)
    y = usw.expert_spmm(bank, x, slots, mul=mul, out_dtype=torch.float32)
    assert torch.equal(y[:2], x[:2].float() @ made[0][1].t() * mul[:2].float())
    assert torch.equal(y[2:], x[2:].float() @ made[1][1].t() * mul[2:].float())
