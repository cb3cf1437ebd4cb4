"""GPU tests of routing, of the sparse product by expert and of the combine,
alone and together, against 64-bit references: uneven and empty runs, tokens
without experts, one slot to many, gathered rows, both value types, every tile
height, captured and on several streams."""
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


def gpu(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def half(rng, *shape, scale=1.0):
    return rng.normal(0.0, scale, size=shape).astype(np.float16)


def bank_of(E, M, K, val, seed, density=0.5, exact=False):
    """(bank, dense weights [E][M][K] in 64 bits); the experts' densities differ."""
    rng = np.random.default_rng(seed)
    encs, dense = [], []
    for e in range(E):
        mask = wl.mask_bernoulli(M, K, min(1.0, density * (0.6 + 0.8 * e / max(1, E - 1))) if E > 1 else density, rng)
        if exact:
            W = wl.weight_int4_exact(M, K, rng, mask) if val == "i4" else wl.weight_dyadic(M, K, rng)
        else:
            W = wl.weight_normal(M, K, rng)
        encs.append(usw.encode(W, mask, dtype=val, device=DEV))
        o = ob.encode_i4(W, mask) if val == "i4" else ob.encode(W, mask)
        dense.append(ob.dense_weight(o).astype(np.float64))
    return usw.expert_bank(encs), dense


def runs_reference(dense, x, slots, rows, bias, name, mul, out, codes=False):
    """(y, bound) of the rows in runs; rows behind them are NaN."""
    S = len(rows) if rows is not None else x.shape[0]
    y = np.full((S, dense[0].shape[0]), np.nan)
    bound = np.zeros_like(y)
    for e, Wd in enumerate(dense):
        a, b = slots[e], slots[e + 1]
        if a == b:
            continue
        xe = x[rows[a:b]] if rows is not None else x[a:b]
        y[a:b], bound[a:b] = ref.product(Wd, xe, None if bias is None else bias[e], name,
                                         None if mul is None else mul[a:b], None, out, codes)
    return y, bound


def near(y, want, bound, what):
    y = y.cpu().numpy().astype(np.float64)
    live = ~np.isnan(want)
    off = np.abs(y - want)[live]
    worst = float(np.max(off / bound[live])) if off.size else 0.0
    say(f"[experts] {what}: worst/bound={worst:.3f}")
    assert np.all(off <= bound[live]), f"{what}: worst/bound {worst:.3f}"


# Rows per expert: one slot, empty experts at both ends and inside, all in
# one, uneven ones around the tiles' heights.
LOADS = {
    "one slot": [0, 1, 0],
    "one expert": [70],
    "all in the last": [0, 0, 0, 40],
    "around 16": [15, 16, 17, 0, 1, 33],
    "around 32": [31, 32, 33, 20, 28],
    "around 64": [63, 64, 65, 0, 129, 40],
    "many experts": [(7 * e) % 5 for e in range(70)],
    "long": [300, 0, 257, 512, 100],
}


@pytest.mark.parametrize("load", list(LOADS))
@pytest.mark.parametrize("val", ["f16", "i4"])
@pytest.mark.parametrize("gather", [True, False])
def test_product_by_expert(load, val, gather):
    counts = LOADS[load]
    E, M, K = len(counts), 128, 192
    bank, dense = bank_of(E, M, K, val, 10 + E)
    slots = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    live, spare = int(slots[-1]), 5
    S = live + spare
    rng = np.random.default_rng(20 + live)
    T = max(3, live // 2)
    rows = rng.integers(0, T, size=S).astype(np.int32) if gather else None
    if gather:
        rows[live:] = -1
    x = half(rng, T if gather else S, K)
    bias, mul = half(rng, E, M), half(rng, S, M)
    for name, out, b, m in (("silu", "f16", bias, mul), ("none", "f32", None, None), ("gelu", "f32", bias, None)):
        say(f"[experts] {load} {val} gather={gather} {name} {out}")
        y = torch.full((S, M), 7.0, dtype=DT[out], device=DEV)
        usw.expert_spmm(bank, gpu(x), gpu(slots), rows=gpu(rows), bias=gpu(b), act=name, mul=gpu(m), y=y)
        want, bound = runs_reference(dense, x, slots, rows, b, name, m, out, val == "i4")
        near(y, want, bound, f"{name} {out}")
        assert torch.all(y[live:] == 7.0)            # rows behind the last run stay


@pytest.mark.parametrize("val", ["f16", "i4"])
@pytest.mark.parametrize("density", [0.0, 0.4, 0.8])
@pytest.mark.parametrize("counts", [[3, 0, 9], [40, 17, 100], [400, 3, 260]])
def test_integer_exact_is_bitwise(val, density, counts):
    E, M, K = len(counts), 192, 320
    bank, dense = bank_of(E, M, K, val, 30, density, exact=True)
    slots = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    S = int(slots[-1])
    rng = np.random.default_rng(31)
    x = wl.activations_small_int(S, K, rng)
    bias = rng.integers(-8, 9, size=(E, M)).astype(np.float16)
    mul = rng.integers(-2, 3, size=(S, M)).astype(np.float16)
    say(f"[experts] exact {val} {density} {counts}")
    y = usw.expert_spmm(bank, gpu(x), gpu(slots), bias=gpu(bias), act="relu", mul=gpu(mul), out_dtype=torch.float32)
    want, _ = runs_reference(dense, x, slots, None, bias, "relu", mul, "f32")
    assert np.array_equal(y.cpu().numpy().astype(np.float64), want)


# Expanded weights: small, medium and large tiles, runs that end inside tiles,
# and experts without rows (whose weights are not expanded).  The references
# are of some rows of every run.
EXPANDED = [([200, 0, 320, 131], 192, 320, "small"), ([500, 900, 0, 700], 1280, 1664, "medium"),
            ([2100, 100, 1900, 0, 2300], 2112, 128, "small, many"), ([2100, 300, 1900, 0, 2300], 2560, 5120, "large"),
            ([40, 35, 0, 90], 192, 64, "one column"), ([150, 90, 3, 100], 320, 256, "few columns")]


@pytest.mark.parametrize("counts,M,K,what", EXPANDED, ids=[e[3] for e in EXPANDED])
@pytest.mark.parametrize("val", ["f16", "i4"])
def test_expanded_tilings(counts, M, K, what, val):
    E = len(counts)
    bank, dense = bank_of(E, M, K, val, 100 + M)
    slots = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    live = int(slots[-1])
    S = live + 7
    rng = np.random.default_rng(101)
    T = 1000
    rows = rng.integers(0, T, size=S).astype(np.int32)
    rows[live:] = -1
    x, bias = half(rng, T, K), half(rng, E, M)
    say(f"[experts] expanded {what} {val}")
    y = torch.full((S, M), 7.0, dtype=torch.float16, device=DEV)
    usw.expert_spmm(bank, gpu(x), gpu(slots), rows=gpu(rows), bias=gpu(bias), act="relu", y=y)
    assert torch.all(y[live:] == 7.0)
    z = usw.expert_spmm(bank, gpu(x), gpu(slots), rows=gpu(rows), bias=gpu(bias), act="relu")
    assert torch.equal(y[:live], z[:live])
    for e in range(E):
        if counts[e] == 0:
            continue
        r = np.unique(np.concatenate([[slots[e], slots[e + 1] - 1], rng.integers(slots[e], slots[e + 1], 30)]))
        want, bound = ref.product(dense[e], x[rows[r]], bias[e], "relu", None, None, "f16")
        near(y[torch.from_numpy(r).to(DEV)], want, bound, f"{what}, expert {e}")


def test_weights_expanded_in_groups():
    """More weights than are expanded at a time (1 GiB of fragments): the same
    encoding in every place, so each expert's rows have one reference."""
    E, M, K = 36, 4096, 4096
    rng = np.random.default_rng(120)
    W, mask = wl.weight_dyadic(M, K, rng), wl.mask_bernoulli(M, K, 0.5, rng)
    enc = usw.encode(W, mask, device=DEV)
    bank = usw.expert_bank([enc] * E)
    counts = [240 + (e % 5) for e in range(E)]
    counts[3], counts[17], counts[35] = 0, 900, 1
    slots = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    S = int(slots[-1])
    x = gpu(wl.activations_small_int(S, K, rng))
    say("[experts] groups")
    y = usw.expert_spmm(bank, x, gpu(slots), out_dtype=torch.float32)
    want = usw.spmm_fused(enc, x, out_dtype=torch.float32)      # exact sums: one weight for all rows
    assert torch.equal(y, want)
    r = rng.integers(0, S, 20)
    Wd = np.where(mask, W, np.float16(0)).astype(np.float64)
    assert np.array_equal(y[torch.from_numpy(r).to(DEV)].cpu().numpy().astype(np.float64),
                          x.cpu().numpy()[r].astype(np.float64) @ Wd.T)


def test_long_rows_split_k_twice_the_same():
    """Few slots and long rows: several workgroups a strip; two calls give the
    same bits."""
    E, M, K = 4, 128, 5120
    for val in ("f16", "i4"):
        bank, dense = bank_of(E, M, K, val, 40)
        slots = np.array([0, 1, 1, 4, 6], dtype=np.int32)
        rng = np.random.default_rng(41)
        x = half(rng, 6, K)
        say(f"[experts] long rows {val}")
        y = usw.expert_spmm(bank, gpu(x), gpu(slots), act="gelu_tanh")
        assert torch.equal(y, usw.expert_spmm(bank, gpu(x), gpu(slots), act="gelu_tanh"))
        want, bound = runs_reference(dense, x, slots, None, None, "gelu_tanh", None, "f16", val == "i4")
        near(y, want, bound, "long rows")


def check_route(logits, k, renormalize, what):
    plan = usw.expert_route(logits, k, renormalize)
    x = logits.float().cpu().numpy()
    ids, weights, slots, rows, pos = ref.route(x, k, renormalize)
    for name, got, want in (("ids", plan.ids, ids), ("offsets", plan.offsets, slots), ("rows", plan.rows, rows),
                            ("pos", plan.pos, pos)):
        assert np.array_equal(got.cpu().numpy(), want), f"{what}: {name}"
    # An exponential of a difference d is off by (|d| + 3) U, a sum of n of
    # them and a quotient by (n + 2) U more.
    fine = x[np.isfinite(x)]
    spread = float(fine.max() - fine.min()) if fine.size else 0.0
    tol = (x.shape[1] + spread + 8) * ref.U32
    got = plan.weights.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - weights) <= 2 * tol * weights + 1e-37), what
    return plan


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 8, 8), (64, 16, 4), (65, 5, 2), (255, 64, 6), (256, 65, 3),
                                   (257, 128, 8), (640, 129, 2), (1000, 300, 16), (3001, 40, 1), (70, 1024, 9),
                                   (300, 1024, 4)])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_route(T, E, k, dtype):
    rng = np.random.default_rng(50 + T + E)
    x = rng.normal(0.0, 2.0, size=(T, E))
    x[rng.random((T, E)) < 0.2] = np.round(x[rng.random((T, E)) < 0.2].mean() if T * E > 8 else 0.0)   # equal ones
    logits = torch.from_numpy(x).to(DEV).to(DT[dtype])
    for renormalize in (True, False):
        say(f"[experts] route T={T} E={E} k={k} {dtype} renormalize={renormalize}")
        check_route(logits, k, renormalize, "random")
    # Masked experts, whole rows masked, NaN, infinities, equal logits, zeros of both signs.
    logits[torch.rand(T, E, device=DEV) < 0.3] = -float("inf")
    logits[::5] = -float("inf")
    if T > 3:
        logits[1, 0] = float("nan")
        logits[2, E // 2] = float("inf")
        logits[3] = 0.0
        logits[3, ::2] = -0.0
    say(f"[experts] route masked T={T} E={E} k={k}")
    for renormalize in (True, False):
        plan = check_route(logits, k, renormalize, "masked")
    assert torch.all(plan.ids[::5] == -1) and torch.all(plan.weights[::5] == 0)


@pytest.mark.parametrize("E", [2, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 512, 513, 1000])
def test_route_lane_layouts(E):
    """Both layouts of a token over lanes, full and partly filled, at each number of logits to a lane."""
    gen = torch.Generator(device=DEV).manual_seed(E)
    for T in (2, 16, 17, 63, 64, 66):
        say(f"[experts] route layouts T={T} E={E}")
        logits = torch.randn(T, E, device=DEV, generator=gen)
        logits[:, E // 2:] = logits[:, :E - E // 2]   # every value twice
        check_route(logits, min(E, 16), False, "twice the same")
        check_route(logits.half(), min(E, 3), True, "half")


@pytest.mark.parametrize("T,E,k", [(4096, 33, 3), (4097, 9, 2), (16384, 5, 2), (16389, 130, 8), (20000, 3, 1)])
def test_route_many_tokens(T, E, k):
    """Each size of a block of tokens, and the prefixes made by a launch of their own."""
    gen = torch.Generator(device=DEV).manual_seed(T)
    say(f"[experts] route many tokens T={T} E={E}")
    logits = torch.randn(T, E, device=DEV, generator=gen).half()
    logits[T // 3:T // 2] = -float("inf")
    check_route(logits, k, True, "many tokens")


def test_route_all_masked_and_strided():
    logits = torch.full((300, 8), -float("inf"), device=DEV)
    say("[experts] route all masked")
    plan = check_route(logits, 2, False, "all masked")
    assert int(plan.offsets[-1]) == 0
    wide = torch.randn(300, 24, device=DEV)
    check_route(wide[:, :8], 2, True, "strided")
    check_route(wide[:40, 8:16], 2, True, "strided, small")
    check_route(wide.t()[:24, :40].contiguous().t(), 3, True, "transposed")
    empty = usw.expert_route(torch.empty(0, 8, device=DEV), 2)
    assert empty.ids.shape == (0, 2) and torch.all(empty.offsets == 0)


@pytest.mark.parametrize("T,k,M", [(1, 1, 8), (4, 2, 4096), (33, 3, 200), (257, 8, 64), (50, 11, 520)])
@pytest.mark.parametrize("yt,out", [("f16", "f16"), ("f32", "f16"), ("f16", "f32"), ("f32", "f32")])
def test_combine(T, k, M, yt, out):
    rng = np.random.default_rng(60 + T + M)
    S = T * k
    y = half(rng, S, M).astype(np.float32 if yt == "f32" else np.float16)
    pos = rng.permutation(S).reshape(T, k).astype(np.int32)
    pos[rng.random((T, k)) < 0.2] = -1
    w = rng.random((T, k)).astype(np.float32)
    res = half(rng, T, 2 * M)
    say(f"[experts] combine T={T} k={k} M={M} {yt} {out}")
    got = usw.expert_combine(gpu(y), gpu(pos), gpu(w), out_dtype=DT[out])
    want, bound = ref.combine(y, pos, w, None, out)
    near(got, want, bound, "no residual")
    got = usw.expert_combine(gpu(y), gpu(pos), gpu(w), residual=gpu(res)[:, M:], out_dtype=DT[out])
    want, bound = ref.combine(y, pos, w, res[:, M:], out)
    near(got, want, bound, "strided residual")
    if out == "f16":
        r = gpu(res[:, :M])
        usw.expert_combine(gpu(y), gpu(pos), gpu(w), residual=r, out=r)
        want, bound = ref.combine(y, pos, w, res[:, :M], out)
        near(r, want, bound, "in place")




@pytest.mark.parametrize("T,val,gated", [(1, "f16", True), (7, "i4", True), (150, "f16", False), (700, "f16", True)])
def test_expert_ffn(T, val, gated):
    """The whole path in 64 bits.  Hidden rows are rounded to fp16 where the
    path rounds them, so the bounds of the three products add: the down
    projection carries the hidden rows' error, at most sum |w| times it."""
    E, k, D, F = 6, 2, 128, 256
    up, Wu = bank_of(E, F, D, val, 70)
    gate, Wg = bank_of(E, F, D, val, 71)
    down, Wd = bank_of(E, D, F, val, 72)
    rng = np.random.default_rng(73 + T)
    x, logits = half(rng, T, D), half(rng, T, E, scale=2.0)
    if T > 3:
        logits[2] = -np.inf
        logits[3, 1:] = -np.inf
    bu, bg, bd = half(rng, E, F), half(rng, E, F), half(rng, E, D)
    say(f"[experts] ffn T={T} {val} gated={gated}")
    kw = dict(gate=gate, gate_bias=gpu(bg)) if gated else {}
    got = usw.expert_ffn(gpu(x), gpu(logits), k, up, down, act="silu", up_bias=gpu(bu), down_bias=gpu(bd),
                         residual=gpu(x), out_dtype=torch.float32, **kw)
    ids, weights, slots, rows, pos = ref.route(logits, k, True)
    S = T * k
    y, ybound = np.zeros((S, D)), np.zeros((S, D))
    for e in range(E):
        a, b = slots[e], slots[e + 1]
        if a == b:
            continue
        xe = x[rows[a:b]]
        if gated:
            u, ub = ref.product(Wu[e], xe, bu[e], out="f16", codes=val == "i4")
            g, gb = ref.product(Wg[e], xe, bg[e], "silu", out="f16", codes=val == "i4")
            h = g * u
            hb = np.abs(g) * ub + gb * (np.abs(u) + ub)
            hb = hb + 2.0 ** -11 * (np.abs(h) + hb) + 2.0 ** -25
        else:
            h, hb = ref.product(Wu[e], xe, bu[e], "silu", out="f16", codes=val == "i4")
        y[a:b], ybound[a:b] = ref.product(Wd[e], h, bd[e], out="f16", codes=val == "i4")
        # The kernel's own sums run over its rounded hidden rows, larger by hb.
        ybound[a:b] += 1.01 * hb @ np.abs(Wd[e]).T
    want, bound = ref.combine(y, pos, weights, x, "f32")
    live = pos >= 0
    bound = bound + (np.where(live, weights, 0.0)[:, :, None] * ybound[np.where(live, pos, 0)]).sum(1) * 1.0001
    bound = bound + (np.where(live, weights, 0.0)[:, :, None] * np.abs(y[np.where(live, pos, 0)])).sum(1) * 64 * ref.U32
    near(got, want, bound, "ffn")
    if T > 3:                                          # a token without experts keeps its residual
        assert np.array_equal(got[2].cpu().numpy(), x[2].astype(np.float32))


def test_captured_and_replayed_with_other_routing():
    """One captured block: the routing, so the runs, changes between replays;
    every replay equals the eager result."""
    E, k, D, F, T = 8, 2, 128, 192, 40
    up, _ = bank_of(E, F, D, "f16", 80)
    gate, _ = bank_of(E, F, D, "f16", 81)
    down, _ = bank_of(E, D, F, "f16", 82)
    x = torch.randn(T, D, device=DEV).half()
    logits = torch.randn(T, E, device=DEV)
    say("[experts] graph")
    call = lambda: usw.expert_ffn(x, logits, k, up, down, gate=gate, residual=x)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = call()
        graphs.append((g, y))
    for rep in range(5):
        x.copy_(torch.randn_like(x))
        logits.copy_(torch.randn_like(logits) + 3 * torch.randn(E, device=DEV))
        if rep == 3:
            logits[:, 1:] = -float("inf")
        want = call()
        if rep % 2:
            torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, y in graphs:
            assert torch.equal(y, want), rep


def test_streams_at_once():
    E, k, D, F = 4, 2, 128, 2560
    up, _ = bank_of(E, F, D, "f16", 90)
    down, _ = bank_of(E, D, F, "f16", 91)
    say("[experts] streams")
    made = [(torch.randn(T, D, device=DEV).half(), torch.randn(T, E, device=DEV)) for T in (5, 300)]
    want = [usw.expert_ffn(x, lg, k, up, down, act="gelu") for x, lg in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device=DEV) for _ in made]
    got = [[], []]
    for _ in range(6):
        for i, ((x, lg), s) in enumerate(zip(made, streams)):
            got[i].append(usw.expert_ffn(x, lg, k, up, down, act="gelu", stream=s))
    torch.cuda.synchronize()
    for ys, w in zip(got, want):
        assert all(torch.equal(y, w) for y in ys)


def test_empty_batch():
    bank, _ = bank_of(2, 64, 64, "f16", 95)
    x = torch.zeros(0, 64, dtype=torch.float16, device=DEV)
    slots = torch.zeros(3, dtype=torch.int32, device=DEV)
    say("[experts] empty")
    assert usw.expert_spmm(bank, x, slots).shape == (0, 64)
    y = usw.expert_ffn(x, torch.empty(0, 2, device=DEV), 1, bank, bank)
    assert y.shape == (0, 64)
    y = usw.expert_combine(torch.zeros(0, 64, device=DEV), torch.full((3, 1), -1, dtype=torch.int32, device=DEV),
                           torch.ones(3, 1, device=DEV))
    assert torch.all(y == 0)


def test_refusals():
    bank, _ = bank_of(2, 64, 128, "f16", 96)
    x = torch.zeros(4, 128, dtype=torch.float16, device=DEV)
    slots = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    rows = torch.zeros(4, dtype=torch.int32, device=DEV)
    for kw in (dict(rows=rows.long()), dict(rows=rows.cpu()), dict(rows=rows.view(2, 2)), dict(act="x"),
               dict(bias=torch.zeros(64, dtype=torch.float16, device=DEV)),
               dict(mul=torch.zeros(3, 64, dtype=torch.float16, device=DEV)),
               dict(y=torch.zeros(4, 128, dtype=torch.float16, device=DEV))):
        with pytest.raises(ValueError):
            usw.expert_spmm(bank, x, slots, **kw)
    for s in (slots.long(), slots[:2], slots.cpu()):
        with pytest.raises(ValueError):
            usw.expert_spmm(bank, x, s)
    with pytest.raises(usw.UswError):                  # rows to read, and no x
        usw.expert_spmm(bank, x[:0], slots, rows=rows)
    lg = torch.zeros(4, 2, device=DEV)
    for bad in (lg[0], lg.double(), lg.cpu()):
        with pytest.raises(ValueError):
            usw.expert_route(bad, 1)
    for k in (0, 3, -1):
        with pytest.raises(usw.UswError):
            usw.expert_route(lg, k)
    with pytest.raises(usw.UswError):
        usw.expert_route(torch.zeros(2, 1025, device=DEV), 1)
    y, pos, w = torch.zeros(4, 64, device=DEV), torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.ones(2, 2, device=DEV)
    for args in ((y, pos.long(), w), (y, pos, w.double()), (y, pos, w[:1]), (y.double(), pos, w), (y[0], pos, w)):
        with pytest.raises(ValueError):
            usw.expert_combine(*args)
    with pytest.raises(usw.UswError):
        usw.expert_combine(torch.zeros(4, 4, device=DEV), pos, w)
    e1 = usw.encode(np.ones((64, 64), dtype=np.float16), None, device=DEV)
    e2 = usw.encode(np.ones((64, 128), dtype=np.float16), None, device=DEV)
    for encs in ([], [e1, e2]):
        with pytest.raises(ValueError):
            usw.expert_bank(encs)
    with pytest.raises(ValueError):
        usw.expert_ffn(x, lg, 1, bank, bank)           # down does not take up's outputs
