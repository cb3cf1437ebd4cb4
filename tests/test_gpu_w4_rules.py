"""GPU tests of the 4-bit product on both sides of its rules: workgroups of one to
five row blocks, in one round of compute units and in more, one and two tiles ahead,
and the rows from which a weight is expanded.  Whole inputs make the sums exact."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

import unstructured_sparse_weight_amd as usw  # noqa: E402
from unstructured_sparse_weight_amd import w4  # noqa: E402

DEV = "cuda:0"


def whole(seed, most, *shape):
    r = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=r, device=DEV).half()


def encoded(M, K, group, seed):
    W = whole(seed, 7, M, K)
    W[:, ::32] = 7   # every group's scale is 1
    return usw.w4_encode_device(W, group), W


def check(enc, W, N, seed):
    """Sums below 21 K < 2^24."""
    x, res = whole(seed, 3, N, W.shape[1]), whole(seed + 1, 9, N, W.shape[0])
    want = (x.float() @ W.float().t()).clamp(min=0) + res.float()
    y = usw.w4_matmul(enc, x, act="relu", residual=res, out_dtype=torch.float32)
    assert torch.equal(y, want), int((y != want).sum())
    y16 = usw.w4_matmul(enc, x, act="relu", residual=res)
    assert torch.equal(y16, want.half())


@pytest.mark.parametrize("K", [64, 192, 1920, 1984, 2048, 2112, 4224, 6080])
@pytest.mark.parametrize("M", [16, 272, 4096])
def test_one_row_block(M, K):
    """One tile ahead below 16 tiles, two from there on; waves of one to six tiles."""
    enc, W = encoded(M, K, 64, K)
    for N in (1, 2, 15, 16):
        check(enc, W, N, N)


@pytest.mark.parametrize("M", [4112, 8208, 12288, 12304, 16384, 16400, 20480, 20496, 24576, 36864, 36880, 65536, 128256])
def test_rounds(M):
    """The last row block of a round and the first behind it."""
    enc, W = encoded(M, 320, 128, M)
    for N in (1, 16, 17, 33):
        check(enc, W, N, N)


@pytest.mark.parametrize("M,K,last", [(20480, 5120, 320), (16384, 8192, 320), (24576, 4096, 192), (8192, 4096, 192),
                                      (8176, 4096, 128)])
def test_rows_before_expansion(M, K, last):
    enc, W = encoded(M, K, 64, 3)
    for N in (last - 64, last - 1, last, last + 1):
        assert (w4._sizes(M, K, 64, N)[0] > 0) == (N > last)
        check(enc, W, N, N)
