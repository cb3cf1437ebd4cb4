"""GPU tests of infinities in what the gradients multiply d with: up to 32 rows d of
a gated block goes along as an fp16 value and its remainder, and an infinity times
the value stays one whatever the remainder is (zero where d is an fp16 number, else
of either sign).  From 33 rows on there is no remainder."""
import pytest

import block_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

import unstructured_sparse_weight_amd as usw  # noqa: E402

DEV = "cuda:0"
M, K = 128, 192
INF = float("inf")


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def signs(r, *shape):
    return torch.randint(0, 2, shape, generator=r, device=DEV).half() * 2 - 1


def operands(N, exact):
    """x, g, u, dy whose dg = dy u and du = dy g are fp16 numbers, or have remainders of both signs."""
    r = gen(31)
    x = torch.randint(-2, 3, (N, K), generator=r, device=DEV).half()
    one = torch.ones(N, M, dtype=torch.float16, device=DEV)
    if not exact:
        # (1 + a 2^-10)(1 + b 2^-10) has a b 2^-20 behind fp16's last place, from 0 to 2^-10.
        one = one + torch.randint(1, 32, (N, M), generator=r, device=DEV).half() * 2.0 ** -10
    dy, g, u = one * signs(r, N, M), one.flip(1) * signs(r, N, M), one.flip(0) * signs(r, N, M)
    d = [dy.double() * t.double() for t in (u, g)]
    rest = torch.cat([(t - t.half().double()).reshape(-1) for t in d])
    assert bool((rest == 0).all()) if exact else bool((rest > 0).any()) and bool((rest < 0).any())
    return x, g, u, dy, d


def weights(seed):
    r = gen(seed)
    W = torch.randint(-3, 4, (M, K), generator=r, device=DEV).half()
    mask = torch.rand(M, K, generator=r, device=DEV) < 0.5
    return W, mask


def kept_at(mask):
    at = ref.storage_order(M, K, DEV)
    return at[mask.view(-1)[at]]


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("N", [1, 2, 16, 20, 32, 33, 64])
@pytest.mark.parametrize("dx", [True, False])
def test_an_infinity_in_x(N, exact, dx):
    """The values of its column are infinite, with the signs of d; no other changes."""
    x, g, u, dy, d = operands(N, exact)
    (Wg, mg), (Wu, mu) = weights(32), weights(33)
    gate, up = usw.encode_device(Wg, mg), usw.encode_device(Wu, mu)
    for n, value in ((0, INF), (N - 1, -INF)):
        xi = x.clone()
        xi[n, 5] = value
        clean = usw.spmm_gated_backward(gate, up, x, g, u, dy, act="none", dx=dx)
        got = usw.spmm_gated_backward(gate, up, xi, g, u, dy, act="none", dx=dx)
        for name, mask, dd in (("gate", mg, d[0]), ("up", mu, d[1])):
            at = kept_at(mask)
            hit = at % K == 5
            a, b = getattr(got, name), getattr(clean, name)
            assert torch.equal(a[~hit], b[~hit]), name
            assert torch.equal(a[hit].double(), value * torch.sign(dd[n][at[hit] // K])), name
        assert not dx or torch.equal(got.x, clean.x)


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("N", [1, 2, 16, 20, 32, 33, 64])
@pytest.mark.parametrize("values", [True, False])
def test_an_infinite_weight(N, exact, values):
    """dx of its column is infinite, with the signs of d of its row; no other changes."""
    x, g, u, dy, d = operands(N, exact)
    pairs = [weights(34), weights(35)]
    for which, (m, k), value in ((0, (70, 17), INF), (1, (3, 190), -INF)):
        clean = [(W.clone(), mask.clone()) for W, mask in pairs]
        W, mask = clean[which]
        mask[m, k] = True
        W[m, k] = 1.0
        encs = [usw.encode_device(*p) for p in clean]
        want = usw.spmm_gated_backward(*encs, x, g, u, dy, act="none", values=values)
        W[m, k] = value
        encs = [usw.encode_device(*p) for p in clean]
        got = usw.spmm_gated_backward(*encs, x, g, u, dy, act="none", values=values)
        assert torch.equal(got.x[:, k].double(), value * torch.sign(d[which][:, m]))
        rest = torch.arange(K, device=DEV) != k
        assert torch.equal(got.x[:, rest], want.x[:, rest])
        if values:
            assert torch.equal(got.gate, want.gate) and torch.equal(got.up, want.up)


@pytest.mark.parametrize("N", [2, 32])
def test_a_nan_stays_one(N):
    """In x and in a weight: the column's results are NaN, no other changes."""
    x, g, u, dy, _ = operands(N, False)
    (Wg, mg), (Wu, mu) = weights(36), weights(37)
    mg[9, 11] = True
    clean = usw.spmm_gated_backward(usw.encode_device(Wg, mg), usw.encode_device(Wu, mu), x, g, u, dy, act="none")
    Wg[9, 11] = float("nan")
    x[N - 1, 7] = float("nan")
    got = usw.spmm_gated_backward(usw.encode_device(Wg, mg), usw.encode_device(Wu, mu), x, g, u, dy, act="none")
    rest = torch.arange(K, device=DEV) != 11
    assert bool(torch.isnan(got.x[:, 11]).all()) and torch.equal(got.x[:, rest], clean.x[:, rest])
    for name, mask in (("gate", mg), ("up", mu)):
        at = kept_at(mask)
        hit = at % K == 7
        a, b = getattr(got, name), getattr(clean, name)
        assert bool(torch.isnan(a[hit]).all()) and torch.equal(a[~hit], b[~hit])


@pytest.mark.parametrize("N", [1, 20, 32, 33])
@pytest.mark.parametrize("rows,cols,density", [(128, 192, 1.0), (1088, 576, 0.5), (64, 4160, 0.9), (4160, 64, 0.3)])
def test_an_infinite_weight_of_other_shapes(rows, cols, density, N):
    """GroupTiles that keep nearly everything, strips of one GroupTile and of many."""
    r = gen(38)
    W = torch.randint(1, 4, (rows, cols), generator=r, device=DEV).half()
    mask = torch.rand(rows, cols, generator=r, device=DEV) < density
    mask[rows - 2, cols - 3] = True
    x = torch.ones(N, cols, dtype=torch.float16, device=DEV)
    dy = signs(r, N, rows) * (1 + 5 * 2.0 ** -10)
    g = signs(r, N, rows) * (1 + 7 * 2.0 ** -10)
    up = usw.encode_device(W, mask)
    want = usw.spmm_gated_backward(up, up, x, g, g, dy, act="none")
    Wi = W.clone()
    Wi[rows - 2, cols - 3] = INF
    got = usw.spmm_gated_backward(usw.encode_device(Wi, mask), up, x, g, g, dy, act="none")
    assert torch.equal(got.x[:, cols - 3].double(), INF * torch.sign(dy[:, rows - 2].double() * g[:, rows - 2].double()))
    rest = torch.arange(cols, device=DEV) != cols - 3
    assert torch.equal(got.x[:, rest], want.x[:, rest])
    assert torch.equal(got.gate, want.gate) and torch.equal(got.up, want.up)
