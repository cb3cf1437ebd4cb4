"""GPU test of the combine over more tokens than one launch has threads for."""
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

import unstructured_sparse_weight_amd as usw  # noqa: E402

DEV = "cuda:0"


@pytest.mark.parametrize("T,M,residual", [((1 << 26) + 5, 8, False), ((1 << 25) + 3, 16, True), ((1 << 24) + 1, 520, False)])
def test_many_tokens(T, M, residual):
    """Whole numbers: exact.  Tokens read rows of a short Y in an uneven order."""
    S = 251
    g = torch.Generator(device=DEV).manual_seed(T)
    y = torch.randint(-9, 10, (S, M), device=DEV, generator=g).half()
    pos = torch.randint(-1, S + 1, (T, 1), dtype=torch.int32, device=DEV, generator=g)   # -1 and S count nothing
    w = torch.randint(1, 4, (T, 1), device=DEV, generator=g).float()
    res = torch.randint(-9, 10, (T, M), device=DEV, generator=g).half() if residual else None
    print(f"[combine] T={T} M={M}", file=sys.stderr, flush=True)
    out = usw.expert_combine(y, pos, w, residual=res)
    for a in range(0, T, 1 << 21):
        p = pos[a:a + (1 << 21), 0].long()
        live = ((p >= 0) & (p < S)).half()[:, None]
        want = y[p.clamp(0, S - 1)] * live * w[a:a + (1 << 21)].half()
        if residual:
            want = want + res[a:a + (1 << 21)]
        assert torch.equal(out[a:a + (1 << 21)], want), a
