"""GPU tests of fused and expert products that take turns on one stream, and so
on one workspace, with counters and partial sums of very different sizes."""
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

import unstructured_sparse_weight_amd as usw  # noqa: E402
from unstructured_sparse_weight_amd import fused  # noqa: E402

DEV = "cuda:0"


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def integer_weight(M, K, density, seed):
    """(encoding, pruned weight): whole numbers from -3 to 3."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    mask = torch.rand(M, K, device=DEV, generator=g) < density
    W = torch.randint(-3, 4, (M, K), device=DEV, generator=g).half()
    return usw.encode_device(W, mask), torch.where(mask, W, 0)


def integers(N, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-4, 5, (N, K), device=DEV, generator=g).half()


def product(W, x):
    """x W^T in fp32, exact: all sums are whole and far below 2^24."""
    out = torch.empty(x.shape[0], W.shape[0], device=DEV)
    for m in range(0, W.shape[0], 1 << 17):
        out[:, m:m + (1 << 17)] = x.float() @ W[m:m + (1 << 17)].float().t()
    return out


def test_many_strips_after_an_expanded_weight():
    """A weight of 16400 strips split in two keeps more than 64 KiB of counters;
    an unsplit expanded product then writes its weight over those behind 64 KiB."""
    M, K = (1 << 20) + 1024, 512
    tall, Wt = integer_weight(M, K, 0.02, 1)
    flat, Wf = integer_weight(2048, K, 0.5, 2)
    need, cb = fused._fused_sizes(M, K, 64, 64, tall.val_type, tall.nnz, 3, 2)
    need2, cb2 = fused._fused_sizes(2048, K, 64, 64, flat.val_type, flat.nnz, 300, 0)
    assert cb > 65536 and cb2 == 0 and cb < need2 < need
    xt, xf = integers(3, K, 3), integers(300, K, 4)
    want_t, want_f = product(Wt, xt), product(Wf, xf)
    for rep in range(3):
        say(f"[sequence] many strips, {rep}")
        y = torch.full((3, M), float("nan"), device=DEV)
        assert torch.equal(usw.spmm_fused(tall, xt, splits=2, y=y), want_t), rep
        assert torch.equal(usw.spmm_fused(flat, xf, out_dtype=torch.float32), want_f), rep


def test_sizes_in_turn():
    """Split and unsplit passes, expanded weights and experts in every order."""
    cases = []
    for i, (M, K, N, splits) in enumerate([(256, 4096, 5, 0), (2048, 512, 300, 0), (128, 2048, 40, 3),
                                           (512, 8256, 1000, 0), (192, 320, 70, 0)]):
        enc, W = integer_weight(M, K, 0.4, 10 + i)
        x = integers(N, K, 20 + i)
        cases.append((lambda e=enc, x=x, s=splits: usw.spmm_fused(e, x, splits=s, out_dtype=torch.float32),
                      product(W, x)))
    made = [integer_weight(64, 4160, 0.4, 30 + e) for e in range(3)]
    bank, x = usw.expert_bank([m[0] for m in made]), integers(9, 4160, 40)
    slots = torch.tensor([0, 4, 4, 9], dtype=torch.int32, device=DEV)
    want = torch.cat([product(made[0][1], x[:4]), product(made[2][1], x[4:])])
    cases.append((lambda: usw.expert_spmm(bank, x, slots, out_dtype=torch.float32), want))
    for i, (a, wa) in enumerate(cases):
        for j, (b, wb) in enumerate(cases):
            say(f"[sequence] {i} {j}")
            assert torch.equal(a(), wa) and torch.equal(b(), wb), (i, j)


def test_released_workspaces():
    """The memory goes back to torch's allocator, calls go on, a captured call
    keeps its own."""
    enc, W = integer_weight(4096, 4096, 0.5, 50)
    x = integers(300, 4096, 51)
    want = product(W, x)
    say("[sequence] release")
    fused.release_workspaces()
    assert torch.equal(usw.spmm_fused(enc, x, out_dtype=torch.float32), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = usw.spmm_fused(enc, x, out_dtype=torch.float32)
    held = torch.cuda.memory_allocated()
    usw.release_workspaces()
    assert held - torch.cuda.memory_allocated() >= 2 * 4096 * 4096
    for _ in range(3):
        y.zero_()
        g.replay()
        assert torch.equal(usw.spmm_fused(enc, x, out_dtype=torch.float32), want)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        usw.release_workspaces()
