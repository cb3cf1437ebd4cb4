"""Cases of the framework's fused and expert-grouped sparse products.

Four operators of a pruned transformer's feed-forward block:

* ``fused``:   y = residual + mul * act(W_sp x + bias), one sparse weight;
* ``experts``: the same product for E sparse weights, each with its own run of
               rows (slots sorted by expert, ragged, offsets on the GPU);
* ``route``:   the k largest logits of every token, their softmax weights, and
               the slots sorted by expert;
* ``combine``: each token's weighted sum of its experts' rows, plus a residual.

With ``own`` false ``run`` computes them from dense weights with elementary
torch operations in fp32; with ``own`` true it calls the framework.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    fused, experts = {"op": "fused"}, {"op": "experts"}
    return [
        # One small layer, 8 tokens: nothing but latency.
        {"name": "fused small layer", **fused, "M": 256, "K": 256, "N": 8, "val": "f16", "act": "gelu", "bias": True,
         "mul": False, "residual": True, "out": "f16", "density": 0.5},
        # OPT-13B FFN up, a decode batch of 16: bias and ReLU.
        {"name": "fused ffn up N=16", **fused, "M": 20480, "K": 5120, "N": 16, "val": "f16", "act": "relu",
         "bias": True, "mul": False, "residual": False, "out": "f16", "density": 0.5},
        # OPT-13B FFN down with INT4 values, one sequence decoding: bias and residual.
        {"name": "fused ffn down i4 N=1", **fused, "M": 5120, "K": 20480, "N": 1, "val": "i4", "act": "none",
         "bias": True, "mul": False, "residual": True, "out": "f16", "density": 0.5},
        # Llama-7B down projection for a ragged batch of 77 tokens, fp32 residual stream out.
        {"name": "fused down N=77", **fused, "M": 4096, "K": 11008, "N": 77, "val": "f16", "act": "none",
         "bias": False, "mul": False, "residual": True, "out": "f32", "density": 0.4},
        # Llama-7B gate projection of a 2048-token prompt, times the up projection.
        {"name": "fused gate N=2048", **fused, "M": 11008, "K": 4096, "N": 2048, "val": "f16", "act": "silu",
         "bias": False, "mul": True, "residual": False, "out": "f16", "density": 0.5},
        # One token through 2 of 8 experts: the serving step of a single sequence.
        {"name": "experts T=1", **experts, "E": 8, "k": 2, "T": 1, "M": 11008, "K": 4096, "val": "f16", "act": "silu",
         "bias": False, "mul": False, "gather": True, "out": "f16", "density": 0.5},
        # A decode batch of 48 over 16 small INT4 experts with biases, uneven loads.
        {"name": "experts i4 T=48", **experts, "E": 16, "k": 2, "T": 48, "M": 5120, "K": 2048, "val": "i4",
         "act": "gelu_tanh", "bias": True, "mul": True, "gather": True, "out": "f16", "density": 0.5},
        # The down projections of a 2000-token prompt over 8 experts.
        {"name": "experts prompt", **experts, "E": 8, "k": 2, "T": 2000, "M": 4096, "K": 11008, "val": "f16",
         "act": "none", "bias": False, "mul": False, "gather": False, "out": "f16", "density": 0.5},
        # Routing of one decode step, and of a long prompt with padding over many experts.
        {"name": "route T=4", "op": "route", "T": 4, "E": 8, "k": 2, "logits": "f32", "renormalize": True,
         "padded": False},
        {"name": "route prompt", "op": "route", "T": 8191, "E": 128, "k": 8, "logits": "f16", "renormalize": False,
         "padded": True},
        # Joining the experts' rows of one decode step, and of a long prompt.
        {"name": "combine T=4", "op": "combine", "T": 4, "k": 2, "M": 4096, "residual": True, "out": "f16"},
        {"name": "combine prompt", "op": "combine", "T": 8191, "k": 4, "M": 5120, "residual": True, "out": "f16"},
    ]


def _log(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["fused", "fused", "experts", "experts", "route", "combine"])
    if op == "route":
        E = rng.randint(2, 256)
        return {"op": op, "T": _log(rng, 1, 8191 * 128 // max(E, 128)), "E": E, "k": rng.randint(1, min(8, E)),
                "logits": rng.choice(["f16", "f32"]), "renormalize": rng.random() < 0.5, "padded": rng.random() < 0.5}
    if op == "combine":
        k, M = rng.randint(1, 8), 8 * _log(rng, 8, 1280)
        return {"op": op, "T": _log(rng, 1, 8191 * 4 * 5120 // max(k * M, 4 * 5120)), "k": k, "M": M,
                "residual": rng.random() < 0.5, "out": rng.choice(["f16", "f32"])}
    common = {"op": op, "val": rng.choice(["f16", "f16", "i4"]),
              "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), "bias": rng.random() < 0.5,
              "mul": rng.random() < 0.4, "out": rng.choice(["f16", "f16", "f32"]),
              "density": round(rng.uniform(0.2, 0.8), 2)}
    while True:
        M, K = 64 * _log(rng, 1, 320), 64 * _log(rng, 1, 320)
        if op == "fused":
            N = _log(rng, 1, 2048)
            if M * K <= 20480 * 5120 and M * K * N <= 11008 * 4096 * 2048:
                return {**common, "M": M, "K": K, "N": N, "residual": rng.random() < 0.5}
        else:
            E = _log(rng, 2, 64)
            k, T = rng.randint(1, min(4, E)), _log(rng, 1, 2000)
            if E * M * K <= 8 * 4096 * 11008 and T * k * M * K <= 2000 * 2 * 4096 * 11008 and E * T * K <= 8 * 2000 * 11008:
                return {**common, "E": E, "k": k, "T": T, "M": M, "K": K, "gather": rng.random() < 0.5}


_OUT = {"f16": torch.float16, "f32": torch.float32}


def _generator(seed, part):
    g = torch.Generator(device=DEV)
    g.manual_seed((seed * 1000003 + part) % (1 << 62))
    return g


def _normal(g, *shape, scale=1.0, dtype=torch.float16):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _weight(g, M, K, density, val):
    """A pruned weight as a user holds it: dense (fp16, or INT4 codes and fp16
    row scales) and in the framework's documented bitmap format."""
    mask = torch.rand(M, K, generator=g, device=DEV) < density
    W = _normal(g, M, K, scale=0.02) * mask
    scales = None
    if val == "i4":
        scales = (W.abs().amax(1).double() / 7).half()
        step = scales.double()[:, None]
        W = torch.where(step > 0, (W.double() / step).round().clamp(-8, 7), 0.0).to(torch.int8)
    # GroupTiles of 64 x 64, TCTiles of 16 x 16, BitmapTiles of 8 x 8, all row-major.
    def order(a):
        return a.view(M // 64, 4, 2, 8, K // 64, 4, 2, 8).permute(0, 4, 1, 5, 2, 6, 3, 7).reshape(-1)

    kept = order(mask)
    bits = torch.tensor([1 << i for i in range(8)], dtype=torch.uint8, device=DEV)
    bitmaps = (kept.view(-1, 8).to(torch.uint8) * bits).sum(1, dtype=torch.uint8).view(torch.int64)
    counts = kept.view(-1, 4096).sum(1)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    values = order(W)[kept]
    nnz = values.numel()
    if val == "i4":
        codes = torch.zeros((nnz + 1) // 2 * 2, dtype=torch.uint8, device=DEV)
        codes[:nnz] = values.view(torch.uint8) & 15
        values = codes[0::2] | (codes[1::2] << 4)
    else:
        values = values.view(torch.uint8)
    stream = torch.zeros((values.numel() & ~15) + 16, dtype=torch.uint8, device=DEV)
    stream[: values.numel()] = values
    return W, scales, bitmaps, offsets, stream, nnz


def _plan(g, T, E, k):
    """Slots sorted by (expert, token) for uneven random routing."""
    score = torch.randn(T, E, generator=g, device=DEV) + torch.randn(E, generator=g, device=DEV)
    ids = score.argsort(dim=1, descending=True, stable=True)[:, :k].reshape(-1)
    expert, slots = ids.sort(dim=0, stable=True)
    counts = torch.bincount(expert, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return offsets, torch.div(slots, k, rounding_mode="floor").to(torch.int32), expert, counts


def prepare(case, seed):
    g = _generator(seed, 1)
    s = dict(case)
    if case["op"] == "route":
        x = torch.randn(case["T"], case["E"], generator=g, device=DEV) * 1.5
        x += torch.randn(case["E"], generator=g, device=DEV) * 0.5
        x = x.to(_OUT[case["logits"]])
        if case["padded"]:   # padding tokens and a few experts out of some tokens' reach
            x[torch.rand(case["T"], generator=g, device=DEV) < 0.1] = -math.inf
            x[torch.rand(x.shape, generator=g, device=DEV) < 0.05] = -math.inf
        s["x"] = x
        return s
    if case["op"] == "combine":
        T, k, M = case["T"], case["k"], case["M"]
        S = T * k
        s["y"] = _normal(g, S, M)
        s["pos"] = torch.randperm(S, generator=g, device=DEV).view(T, k).to(torch.int32)
        dropped = torch.rand(T, k, generator=g, device=DEV) < 0.03
        s["pos"][dropped] = -1
        w = torch.rand(T, k, generator=g, device=DEV) + 0.05
        s["w"] = torch.where(dropped, 0.0, w / w.sum(1, keepdim=True))
        s["res"] = _normal(g, T, M) if case["residual"] else None
        return s
    M, K = case["M"], case["K"]
    if case["op"] == "fused":
        s["W"], s["scales"], s["bitmaps"], s["offsets"], s["values"], s["nnz"] = _weight(g, M, K, case["density"], case["val"])
        rows = case["N"]
        s["x"] = _normal(g, rows, K)
        s["b"] = _normal(g, M, scale=0.5) if case["bias"] else None
        s["res"] = _normal(g, rows, M) if case["residual"] else None
    else:
        E, T, k = case["E"], case["T"], case["k"]
        rows = T * k
        made = [_weight(_generator(seed, 2 + e), M, K, case["density"], case["val"]) for e in range(E)]
        s["W"] = torch.stack([m[0] for m in made])
        s["scales"] = torch.stack([m[1] for m in made]) if case["val"] == "i4" else None
        s["bitmaps"] = torch.stack([m[2] for m in made])
        s["offsets"] = torch.stack([m[3] for m in made])
        s["values"] = torch.cat([m[4] for m in made])
        sizes = torch.tensor([0] + [m[4].numel() for m in made])
        s["starts"] = sizes.cumsum(0).to(DEV)
        s["nnz"] = sum(m[5] for m in made)
        s["slots"], s["rows"], s["expert"], counts = _plan(g, T, E, k)
        s["active"] = counts.nonzero().view(-1)
        s["most"] = int(counts.max())
        s["x"] = _normal(g, T if case["gather"] else rows, K)
        s["b"] = _normal(g, E, M, scale=0.5) if case["bias"] else None
        s["res"] = None
    s["mul"] = _normal(g, rows, M) if case["mul"] else None
    return s


def _act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _epilogue(s, v, bias):
    if bias is not None:
        v = v + bias.float()
    v = _act(v, s["act"])
    if s["mul"] is not None:
        v = v * s["mul"].float()
    if s["res"] is not None:
        v = v + s["res"].float()
    return v.to(_OUT[s["out"]])


def _plain_fused(s):
    W = s["W"].float()
    if s["scales"] is not None:
        W = W * s["scales"].float()[:, None]
    return _epilogue(s, s["x"].float() @ W.t(), s["b"])


def _plain_experts(s):
    """Each active expert's rows padded to the longest run, one batched product."""
    active, expert = s["active"], s["expert"]
    every = active.numel() == s["E"]
    W = (s["W"] if every else s["W"][active]).float()
    if s["scales"] is not None:
        W = W * (s["scales"] if every else s["scales"][active]).float()[:, :, None]
    S, K = expert.numel(), s["K"]
    at = torch.searchsorted(active, expert)
    within = torch.arange(S, device=DEV) - s["slots"].long()[expert]
    x = s["x"][s["rows"].long()] if s["gather"] else s["x"]
    xp = torch.zeros(active.numel(), s["most"], K, device=DEV)
    xp[at, within] = x.float()
    v = torch.bmm(xp, W.transpose(1, 2))[at, within]
    return _epilogue(s, v, None if s["b"] is None else s["b"][expert])


def _plain_route(s):
    x, E, k = s["x"].float(), s["E"], s["k"]
    T = x.shape[0]
    value, ids = x.sort(dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    live = value > -math.inf
    top = value[:, :1].clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(value - top)
    total = e.sum(1, keepdim=True) if s["renormalize"] else torch.exp(x - top).sum(1, keepdim=True)
    weights = torch.where(live, e / total.clamp(min=1e-30), 0.0)
    key, slots = torch.where(live, ids, E).reshape(-1).sort(dim=0, stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    pos = torch.empty_like(slots)
    pos[slots] = torch.arange(T * k, device=DEV)
    rows = torch.where(key < E, torch.div(slots, k, rounding_mode="floor"), -1)
    return {"ids": torch.where(live, ids, -1).to(torch.int32), "weights": weights, "offsets": offsets.to(torch.int32),
            "rows": rows.to(torch.int32), "pos": torch.where(live, pos.view(T, k), -1).to(torch.int32)}


def _plain_combine(s):
    pos = s["pos"].long()
    v = torch.where(pos < 0, 0.0, s["w"])[:, :, None] * s["y"][pos.clamp(min=0)].float()
    v = v.sum(1)
    if s["res"] is not None:
        v = v + s["res"].float()
    return v.to(_OUT[s["out"]])


def _own(s):
    import unstructured_sparse_weight_amd as usw

    op = s["op"]
    if op == "route":
        p = usw.expert_route(s["x"], s["k"], renormalize=s["renormalize"])
        return {"ids": p.ids, "weights": p.weights, "offsets": p.offsets, "rows": p.rows, "pos": p.pos}
    if op == "combine":
        return usw.expert_combine(s["y"], s["pos"], s["w"], residual=s["res"], out_dtype=_OUT[s["out"]])
    val = usw.USW_VAL_I4 if s["val"] == "i4" else usw.USW_VAL_F16
    if op == "fused":
        enc = usw.Encoding(s["M"], s["K"], 64, 64, val, s["nnz"], s["bitmaps"], s["offsets"], s["values"], s["scales"])
        return usw.spmm_fused(enc, s["x"], bias=s["b"], act=s["act"], mul=s["mul"], residual=s["res"],
                              out_dtype=_OUT[s["out"]])
    bank = usw.ExpertBank(s["E"], s["M"], s["K"], val, s["nnz"], s["bitmaps"], s["offsets"], s["values"], s["starts"],
                          s["scales"])
    return usw.expert_spmm(bank, s["x"], s["slots"], rows=s["rows"] if s["gather"] else None, bias=s["b"], act=s["act"],
                           mul=s["mul"], out_dtype=_OUT[s["out"]])


def run(state):
    if own:
        return _own(state)
    return {"fused": _plain_fused, "experts": _plain_experts, "route": _plain_route,
            "combine": _plain_combine}[state["op"]](state)


def work(case):
    out = 2 if case.get("out") == "f16" else 4
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * (2 if case["logits"] == "f16" else 4) + 16 * T * k + 4 * (E + 1), "flops": 2 * T * E}
    if case["op"] == "combine":
        T, k, M = case["T"], case["k"], case["M"]
        return {"bytes": T * k * (2 * M + 8) + T * M * (out + (2 if case["residual"] else 0)), "flops": 2 * T * k * M}
    M, K = case["M"], case["K"]
    payload = 0.5 if case["val"] == "i4" else 2
    weight = M * K / 8 + 4 * (M // 64) * (K // 64) + payload * case["density"] * M * K
    weight += 2 * M if case["val"] == "i4" else 0
    if case["op"] == "fused":
        rows, x, weights = case["N"], case["N"], 1
    else:
        rows, x = case["T"] * case["k"], case["T"] if case["gather"] else case["T"] * case["k"]
        weights = min(case["E"], rows)   # the experts that can have rows
    operands = (2 if case["mul"] else 0) + (2 if case.get("residual") else 0)
    moved = weights * weight + 2 * x * K + rows * M * (out + operands) + (2 * M * weights if case["bias"] else 0)
    return {"bytes": moved, "flops": 2 * case["density"] * M * K * rows}


def _act64(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "gelu":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2))
    if act == "gelu_tanh":   # (1 + tanh z) / 2 is the logistic function of 2 z
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "silu":
        return v * torch.special.expit(v)
    return v


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        x, k = s["x"].double(), s["k"]
        ids = torch.argsort(-x, dim=1, stable=True)[:, :k]
        value = torch.gather(x, 1, ids)
        weights = torch.softmax(value if s["renormalize"] else x, 1)
        weights = weights if s["renormalize"] else torch.gather(weights, 1, ids)
        return {"ids": None, "weights": torch.nan_to_num(weights, nan=0.0), "offsets": None, "rows": None, "pos": None}
    if case["op"] == "combine":
        out = s["res"].double() if s["res"] is not None else torch.zeros(s["T"], s["M"], dtype=torch.float64, device=DEV)
        for j in range(s["k"]):
            p = s["pos"][:, j].long()
            out = out + torch.where((p >= 0)[:, None], s["w"][:, j, None].double() * s["y"][p.clamp(min=0)].double(), 0.0)
        return out
    rows = case["N"] if case["op"] == "fused" else case["T"] * case["k"]
    v = torch.empty(rows, s["M"], dtype=torch.float64, device=DEV)
    if case["op"] == "fused":
        runs = [(0, rows, s["W"], s["scales"], s["b"])]
    else:
        at = s["slots"].tolist()
        runs = [(at[e], at[e + 1], s["W"][e], None if s["scales"] is None else s["scales"][e],
                 None if s["b"] is None else s["b"][e]) for e in range(s["E"])]
    gathered = case["op"] == "experts" and s["gather"]
    for a, b, W, scale, bias in runs:
        x = s["x"][s["rows"][a:b].long()] if gathered else s["x"][a:b]
        p = torch.matmul(W.double(), x.double().t()).t()
        if scale is not None:
            p = p * scale.double()
        v[a:b] = p if bias is None else p + bias.double()
    v = _act64(v, s["act"])
    if s["mul"] is not None:
        v = v * s["mul"].double()
    return v if s["res"] is None else v + s["res"].double()
