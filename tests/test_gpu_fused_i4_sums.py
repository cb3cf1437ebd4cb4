"""GPU test of the INT4 products' sums where x is all positive, as a ReLU leaves
it: whole numbers whose products and partial sums stay below 2^24, so that any
order of fp32 sums is exact, and whose results are small multiples of 1/8, which
fp16 holds exactly.  Kernels that carry an offset in every code must not let it
grow with the sum of x."""
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

import unstructured_sparse_weight_amd as usw  # noqa: E402

DEV = "cuda:0"
K = 20480


def balanced_weight(M, seed):
    """Neighbouring columns hold opposite codes, half of the pairs are kept, and
    every row's scale is 1/8 (its largest code is 7)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = torch.randint(-7, 8, (M, K // 2), device=DEV, generator=g)
    kept = torch.rand(M, K // 2, device=DEV, generator=g) < 0.5
    c[:, 0], kept[:, 0] = 7, True
    W = (torch.stack([c, -c], 2).view(M, K) / 8).half()
    mask = kept.repeat_interleave(2, 1)
    return usw.encode_device(W, mask, dtype="i4"), torch.where(mask, W, 0)


def nearly_equal_pairs(N, seed):
    """Whole numbers of 200 to 255, equal in the columns of a pair but for a few that are one larger."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randint(200, 255, (N, K // 2), device=DEV, generator=g).repeat_interleave(2, 1)
    x.scatter_add_(1, torch.randint(0, K // 2, (N, 20), device=DEV, generator=g) * 2,
                   torch.ones(N, 20, dtype=x.dtype, device=DEV))
    return x.half()


def exact(W, x):
    want = x.double() @ W.double().t()
    assert float((x.double() @ W.double().abs().t()).max()) * 8 < 2 ** 24     # in units of the codes
    assert torch.equal(want.half().double(), want)
    return want


@pytest.mark.parametrize("N", [1, 16, 20, 33, 64, 70, 90, 128, 300])
@pytest.mark.parametrize("splits", [0, 1])
@pytest.mark.parametrize("out", [torch.float16, torch.float32])
def test_one_weight(N, splits, out):
    enc, W = balanced_weight(128, 1)
    x = nearly_equal_pairs(N, 2 + N)
    print(f"[i4 sums] N={N} splits={splits} {out}", file=sys.stderr, flush=True)
    y = usw.spmm_fused(enc, x, splits=splits, out_dtype=out)
    assert torch.equal(y.double(), exact(W, x))


@pytest.mark.parametrize("each", [5, 20, 60, 250])
@pytest.mark.parametrize("out", [torch.float16, torch.float32])
def test_by_expert(each, out):
    E = 16
    enc, W = balanced_weight(2048, 3)
    bank = usw.expert_bank([enc] * E)
    x = nearly_equal_pairs(E * each, 4 + each)
    slots = torch.arange(E + 1, dtype=torch.int32, device=DEV) * each
    print(f"[i4 sums] experts, {each} rows each {out}", file=sys.stderr, flush=True)
    y = usw.expert_spmm(bank, x, slots, out_dtype=out)
    assert torch.equal(y.double(), exact(W, x))
