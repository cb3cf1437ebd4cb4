"""GPU tests of usw_spmm_fused: the sparse product with bias, activation,
factor and residual in its epilogue, against 64-bit references on the dense
weight, over value types, row counts on every side of the kernels' passes,
densities, output types, strides and split factors."""
import sys

import numpy as np
import pytest

import ffn_reference as ref
import workloads as wl
from oracle import tca_bme as ob

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU containers
    pytest.skip("needs a GPU", allow_module_level=True)

import unstructured_sparse_weight_amd as usw  # noqa: E402

DEV = "cuda:0"
DT = {"f16": torch.float16, "f32": torch.float32}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def weight(M, K, density, val, seed, exact=False):
    """(encoding, dense weight in 64 bits)."""
    rng = np.random.default_rng(seed)
    mask = wl.mask_bernoulli(M, K, density, rng)
    if exact:
        W = wl.weight_int4_exact(M, K, rng, mask) if val == "i4" else wl.weight_dyadic(M, K, rng)
    else:
        W = wl.weight_normal(M, K, rng)
    enc = usw.encode(W, mask, dtype=val, device=DEV)
    o = ob.encode_i4(W, mask) if val == "i4" else ob.encode(W, mask)
    return enc, ob.dense_weight(o).astype(np.float64)


def half(rng, *shape, scale=1.0):
    return (rng.normal(0.0, scale, size=shape)).astype(np.float16)


def gpu(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def near(y, want, bound, what):
    y = y.cpu().numpy().astype(np.float64)
    off = np.abs(y - want)
    worst = float(np.max(off / bound)) if y.size else 0.0
    say(f"[fused] {what}: worst/bound={worst:.3f}")
    assert np.all(off <= bound), f"{what}: worst/bound {worst:.3f}"


SHAPES = [(64, 64, 1), (128, 192, 16), (256, 128, 17), (64, 1024, 33), (192, 320, 64), (320, 256, 65), (128, 64, 129),
          (256, 512, 200), (192, 256, 300), (64, 4160, 5), (1024, 128, 2)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("val", ["f16", "i4"])
def test_full_epilogue(M, K, N, val):
    for i, (name, out) in enumerate([("silu", "f16"), ("gelu", "f32"), ("gelu_tanh", "f16"), ("relu", "f32")]):
        density = (0.5, 0.3, 0.9, 0.6)[i]
        say(f"[fused] {M}x{K} N={N} {val} {name} {out} density {density}")
        enc, Wd = weight(M, K, density, val, 1000 + M + K + N + i)
        rng = np.random.default_rng(2000 + N + i)
        x, b = half(rng, N, K, scale=2.0), half(rng, M)
        mul, res = half(rng, N, M), half(rng, N, M)
        y = usw.spmm_fused(enc, gpu(x), bias=gpu(b), act=name, mul=gpu(mul), residual=gpu(res), out_dtype=DT[out])
        want, bound = ref.product(Wd, x, b, name, mul, res, out, val == "i4")
        near(y, want, bound, f"{name} {out}")


@pytest.mark.parametrize("use", ["none", "bias", "mul", "res", "act"])
@pytest.mark.parametrize("N", [3, 40, 260])
def test_each_operand_alone(use, N):
    M, K = 192, 256
    enc, Wd = weight(M, K, 0.5, "f16", 40 + N)
    rng = np.random.default_rng(41)
    x = half(rng, N, K)
    b = half(rng, M) if use == "bias" else None
    mul = half(rng, N, M) if use == "mul" else None
    res = half(rng, N, M) if use == "res" else None
    name = "relu" if use == "act" else "none"
    say(f"[fused] alone {use} N={N}")
    y = usw.spmm_fused(enc, gpu(x), bias=gpu(b), act=name, mul=gpu(mul), residual=gpu(res))
    want, bound = ref.product(Wd, x, b, name, mul, res)
    near(y, want, bound, use)


@pytest.mark.parametrize("val", ["f16", "i4"])
@pytest.mark.parametrize("density", [0.0, 0.02, 0.5, 1.0])
@pytest.mark.parametrize("N", [1, 16, 33, 150, 513])
def test_integer_exact_is_bitwise(val, density, N):
    """Dyadic weights and small integers: every sum, factor and residual is
    exact in fp32, so any order gives the same bits."""
    M, K = 320, 448
    enc, Wd = weight(M, K, density, val, 60 + N, exact=True)
    rng = np.random.default_rng(61 + N)
    x = wl.activations_small_int(N, K, rng)
    b = rng.integers(-8, 9, size=M).astype(np.float16)
    mul = rng.integers(-2, 3, size=(N, M)).astype(np.float16)
    res = rng.integers(-8, 9, size=(N, M)).astype(np.float16)
    say(f"[fused] exact {val} density {density} N={N}")
    y = usw.spmm_fused(enc, gpu(x), bias=gpu(b), act="relu", mul=gpu(mul), residual=gpu(res), out_dtype=torch.float32)
    want, _ = ref.product(Wd, x, b, "relu", mul, res, "f32")
    assert np.array_equal(y.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("N", [2, 64, 300])
def test_equals_the_plain_product_without_epilogue(N):
    M, K = 256, 640
    enc, Wd = weight(M, K, 0.5, "f16", 70, exact=True)
    x = gpu(wl.activations_small_int(N, K, np.random.default_rng(71)))
    say(f"[fused] plain N={N}")
    assert torch.equal(usw.spmm_fused(enc, x, out_dtype=torch.float32), usw.spmm(enc, x, out_dtype=torch.float32))


@pytest.mark.parametrize("N", [5, 90, 300])
def test_strided_operands_and_residual_in_place(N):
    """mul and residual as halves of wider tensors, an x that is a slice, and
    y written over the residual."""
    M, K = 128, 256
    enc, Wd = weight(M, K, 0.5, "f16", 80)
    rng = np.random.default_rng(81)
    x, wide, res = half(rng, N, K + 16), half(rng, N, 2 * M), half(rng, N, M)
    say(f"[fused] strided N={N}")
    gx, gw, gr = gpu(x), gpu(wide), gpu(res)
    y = usw.spmm_fused(enc, gx[:, 8:8 + K], mul=gw[:, M:], residual=gw[:, :M])
    want, bound = ref.product(Wd, x[:, 8:8 + K], None, "none", wide[:, M:], wide[:, :M])
    near(y, want, bound, "strided")
    y = usw.spmm_fused(enc, gx[:, :K], residual=gr, y=gr)
    assert y.data_ptr() == gr.data_ptr()
    want, bound = ref.product(Wd, x[:, :K], res=res)
    near(y, want, bound, "in place")


@pytest.mark.parametrize("splits", [1, 2, 5, 1000])
@pytest.mark.parametrize("val", ["f16", "i4"])
@pytest.mark.parametrize("N", [4, 30, 70])
def test_split_factors(splits, val, N):
    M, K = 128, 2560
    enc, Wd = weight(M, K, 0.5, val, 90)
    rng = np.random.default_rng(91)
    x, b, mul = half(rng, N, K), half(rng, M), half(rng, N, M)
    say(f"[fused] splits={splits} {val} N={N}")
    y = usw.spmm_fused(enc, gpu(x), bias=gpu(b), act="silu", mul=gpu(mul), splits=splits)
    z = usw.spmm_fused(enc, gpu(x), bias=gpu(b), act="silu", mul=gpu(mul), splits=splits)
    assert torch.equal(y, z)
    want, bound = ref.product(Wd, x, b, "silu", mul, None, "f16", val == "i4")
    near(y, want, bound, "splits")


@pytest.mark.parametrize("val", ["f16", "i4"])
@pytest.mark.parametrize("N", [65, 80, 81, 96, 97, 128, 129, 200, 300])
def test_long_passes(val, N):
    """One pass of more than 64 rows, equal passes of up to 128 and a shorter
    last one; slots of both sizes and the path of GroupTiles that fit none."""
    M, K = 128, 1344
    for density, splits in ((0.4, 1), (0.65, 3), (0.97, 2), (0.5, 5)):
        enc, Wd = weight(M, K, density, val, 95)
        rng = np.random.default_rng(96 + N)
        x, b, mul, res = half(rng, N, K), half(rng, M), half(rng, N, M), half(rng, N, M)
        for out in ("f16", "f32"):
            say(f"[fused] long pass N={N} {val} density {density} splits={splits} {out}")
            y = usw.spmm_fused(enc, gpu(x), bias=gpu(b), act="gelu", mul=gpu(mul), residual=gpu(res),
                               out_dtype=DT[out], splits=splits)
            z = usw.spmm_fused(enc, gpu(x), bias=gpu(b), act="gelu", mul=gpu(mul), residual=gpu(res),
                               out_dtype=DT[out], splits=splits)
            assert torch.equal(y, z)
            want, bound = ref.product(Wd, x, b, "gelu", mul, res, out, val == "i4")
            near(y, want, bound, "long pass")


@pytest.mark.parametrize("val", ["f16", "i4"])
@pytest.mark.parametrize("N", [66, 90, 127])
def test_long_passes_integer_exact(val, N):
    M, K = 2112, 2048   # more than 2^22 elements: passes without a split factor asked for
    enc, Wd = weight(M, K, 0.5, val, 97, exact=True)
    x = wl.activations_small_int(N, K, np.random.default_rng(98))
    say(f"[fused] long pass exact {val} N={N}")
    y = usw.spmm_fused(enc, gpu(x), act="relu", out_dtype=torch.float32)
    want, _ = ref.product(Wd, x, None, "relu", None, None, "f32")
    assert np.array_equal(y.cpu().numpy().astype(np.float64), want)


# Every tiling of the expanded product: small tiles with and without splits,
# medium ones with and without, large ones in whole rounds and with tiles left
# over; outputs and rows that end inside a tile.  The references are of some
# rows: those around the tiles' edges and a few between.
EXPANDED = [(320, 1024, 70, "small, split"), (1600, 512, 700, "small"), (512, 8256, 1000, "medium, split"),
            (2624, 832, 2050, "medium"), (4096, 768, 4096, "large"), (4160, 3840, 4900, "large, left over")]


def some_rows(N, rng):
    edges = [r for e in range(0, N + 1, 64) for r in (e - 1, e) if 0 <= r < N]
    return np.unique(np.concatenate([rng.choice(edges, min(40, len(edges)), replace=False), rng.integers(0, N, 20),
                                     [0, N - 1]]))


@pytest.mark.parametrize("M,K,N,what", EXPANDED, ids=[e[3] for e in EXPANDED])
@pytest.mark.parametrize("val", ["f16", "i4"])
def test_expanded_tilings(M, K, N, what, val):
    enc, Wd = weight(M, K, 0.5, val, 300 + N)
    rng = np.random.default_rng(301)
    x, b, mul = half(rng, N, K), half(rng, M), half(rng, N, M)
    say(f"[fused] expanded {what} {val}")
    y = usw.spmm_fused(enc, gpu(x), bias=gpu(b), act="relu", mul=gpu(mul))
    assert torch.equal(y, usw.spmm_fused(enc, gpu(x), bias=gpu(b), act="relu", mul=gpu(mul)))
    r = some_rows(N, rng)
    want, bound = ref.product(Wd, x[r], b, "relu", mul[r])
    near(y[torch.from_numpy(r).to(DEV)], want, bound, what)


@pytest.mark.parametrize("M,K,N,what", EXPANDED, ids=[e[3] for e in EXPANDED])
def test_expanded_is_exact_on_integers(M, K, N, what):
    enc, Wd = weight(M, K, 0.6, "f16", 310 + N, exact=True)
    rng = np.random.default_rng(311)
    x = wl.activations_small_int(N, K, rng)
    res = rng.integers(-8, 9, size=(N, M)).astype(np.float16)
    say(f"[fused] expanded exact {what}")
    y = usw.spmm_fused(enc, gpu(x), residual=gpu(res), out_dtype=torch.float32)
    r = some_rows(N, rng)
    want = x[r].astype(np.float64) @ Wd.T + res[r].astype(np.float64)
    assert np.array_equal(y.cpu().numpy()[r].astype(np.float64), want)


def test_relu_and_large_values():
    """Sums far out: ReLU keeps zeros, SiLU and GELU go to 0 and to v, and an
    fp16 result past the range is an infinity."""
    M = K = 64
    W = np.eye(64, dtype=np.float16)
    enc = usw.encode(W, None, device=DEV)
    v = np.array([0.0, -0.5, 1.0, -60000.0, 60000.0, -100.0, 100.0, -20.0] * 8, dtype=np.float16)
    x = gpu(v[None, :])
    say("[fused] large values")
    for name in ("relu", "gelu", "gelu_tanh", "silu"):
        y = usw.spmm_fused(enc, x, act=name, out_dtype=torch.float32).cpu().numpy().astype(np.float64)
        with np.errstate(over="ignore"):
            want = ref.act(v.astype(np.float64)[None, :], name)
        assert np.allclose(y, want, rtol=2e-5, atol=1e-30 if name == "relu" else 2e-4), name
    y = usw.spmm_fused(enc, x, mul=gpu(np.full((1, M), 2.0, dtype=np.float16)))
    assert torch.isinf(y[0, 4]) and torch.isinf(y[0, 3]) and y[0, 2] == 2.0


def test_captured_calls_keep_their_own_workspaces():
    """Two graphs captured on one stream, replayed several times with eager
    calls and new inputs between: each replay equals the eager result."""
    say("[fused] graphs")
    cases = [(256, 2560, 8, "f16"), (128, 1024, 100, "i4"), (192, 1280, 300, "f16"), (2112, 2048, 77, "f16"),
             (2112, 2048, 120, "i4")]
    made = []
    for i, (M, K, N, val) in enumerate(cases):
        enc, Wd = weight(M, K, 0.5, val, 200 + i)
        rng = np.random.default_rng(210 + i)
        made.append((enc, gpu(half(rng, N, K)), gpu(half(rng, M)), gpu(half(rng, N, M))))
    call = lambda c: usw.spmm_fused(c[0], c[1], bias=c[2], act="silu", residual=c[3])  # noqa: E731
    for c in made:
        call(c)
    torch.cuda.synchronize()
    graphs = []
    for c in made:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = call(c)
        graphs.append((g, y))
    for rep in range(4):
        for c in made:
            c[1].copy_(torch.randn_like(c[1]))
        want = [call(c) for c in made]
        if rep % 2:
            torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (_, y), w in zip(graphs, want):
            assert torch.equal(y, w), rep


def test_two_streams():
    """The same encoding on two streams at once, split K on both."""
    say("[fused] streams")
    M, K = 256, 5120
    enc, Wd = weight(M, K, 0.5, "f16", 230)
    rng = np.random.default_rng(231)
    xs = [gpu(half(rng, 8, K)), gpu(half(rng, 12, K))]
    b = gpu(half(rng, M))
    want = [usw.spmm_fused(enc, x, bias=b, act="gelu") for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device=DEV) for _ in xs]
    got = [[], []]
    for _ in range(8):
        for i, (x, s) in enumerate(zip(xs, streams)):
            got[i].append(usw.spmm_fused(enc, x, bias=b, act="gelu", stream=s))
    torch.cuda.synchronize()
    for ys, w in zip(got, want):
        assert all(torch.equal(y, w) for y in ys)


def test_two_threads_on_one_stream():
    """Calls of two threads on the current stream, one with partial sums and
    one with an expanded weight, share the stream's workspace."""
    import threading
    say("[fused] threads")
    cases = []
    for i, (M, K, N) in enumerate([(128, 5120, 9), (256, 512, 300), (512, 2048, 200)]):
        enc, _ = weight(M, K, 0.5, "f16", 235 + i)
        cases.append((enc, gpu(half(np.random.default_rng(236 + i), N, K))))
    want = [usw.spmm_fused(e, x, act="silu") for e, x in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]

    def work(i):
        for _ in range(30):
            got[i].append(usw.spmm_fused(*cases[i], act="silu"))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for ys, w in zip(got, want):
        assert len(ys) == 30 and all(torch.equal(y, w) for y in ys)


def test_ffn_chain():
    """OPT's and Llama's feed-forward blocks from these calls, against the
    same blocks in 64 bits with the hidden activations rounded to fp16 as the
    chain rounds them."""
    D, F, N = 256, 640, 9
    up, Wu = weight(F, D, 0.5, "f16", 240)
    gate, Wg = weight(F, D, 0.5, "f16", 241)
    down, Wdn = weight(D, F, 0.5, "i4", 242)
    rng = np.random.default_rng(243)
    x, b1, b2 = half(rng, N, D), half(rng, F), half(rng, D)
    say("[fused] chain")
    h = usw.spmm_fused(up, gpu(x), bias=gpu(b1), act="relu")
    want, bound = ref.product(Wu, x, b1, "relu")
    near(h, want, bound, "relu(W1 x + b1)")
    y = usw.spmm_fused(down, h, bias=gpu(b2), residual=gpu(x))
    want, bound = ref.product(Wdn, h.cpu().numpy(), b2, "none", None, x, "f16", True)
    near(y, want, bound, "W2 h + b2 + x")
    u = usw.spmm(up, gpu(x))
    h = usw.spmm_fused(gate, gpu(x), act="silu", mul=u)
    want, bound = ref.product(Wg, x, None, "silu", u.cpu().numpy())
    near(h, want, bound, "silu(Wg x) * u")


def test_refusals():
    enc, _ = weight(128, 128, 0.5, "f16", 250)
    x = torch.zeros(4, 128, dtype=torch.float16, device=DEV)
    m = torch.zeros(4, 128, dtype=torch.float16, device=DEV)
    bad = [dict(act="tanh"), dict(bias=m), dict(bias=m[0].float()), dict(mul=m[:3]), dict(mul=m.float()),
           dict(residual=m[:, :64]), dict(residual=m.cpu()), dict(y=m.float(), out_dtype=torch.float16),
           dict(y=m[:2]), dict(y=m.to(torch.bfloat16)), dict(out_dtype=torch.float64)]
    for kw in bad:
        with pytest.raises(ValueError):
            usw.spmm_fused(enc, x, **kw)
    for xb in (x.float(), x[:, :64], x.cpu(), x[0]):
        with pytest.raises(ValueError):
            usw.spmm_fused(enc, xb)
    with pytest.raises(usw.UswError):
        usw.spmm_fused(enc, x[:0])
