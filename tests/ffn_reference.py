"""64-bit references of the products with an epilogue, of routing and of the
combine, and how far a 32-bit computation rounded once may be from them.
Plain NumPy on the dense weights; nothing here calls the library."""
import math

import numpy as np

U32 = 2.0 ** -24                                  # half a step of fp32, relative
HALF_STEP = {"f16": (2.0 ** -11, 2.0 ** -25), "f32": (2.0 ** -24, 2.0 ** -150)}   # relative, and of the smallest subnormal

_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(v, name):
    if name == "relu":
        return np.where(v < 0, 0.0, v)
    if name == "gelu":
        return 0.5 * v * (1 + _erf(v / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if name == "silu":
        return v / (1 + np.exp(-v))
    return v


def product(Wd, x, bias=None, name="none", mul=None, res=None, out="f16", codes=False):
    """(y, bound): the value in 64 bits, and the most that fp32 sums, an fp32
    epilogue and one rounding may be off it.

    * A sum of K exact products in fp32, in any order, is off by at most
      (K + 1) U sum|w x|; INT4 kernels sum codes and scale once, one rounding
      more (codes times fp16 x are exact too).  With fp16 output they may be
      off from zero by 72 (``codes``), which adds sum|72 x| times the row's
      scale, a seventh of its largest weight.
    * Bias: one more rounding.  The activations' slopes are at most 1.13; their
      own error is that of an exponential whose argument is rounded (2 U |z|
      relative, z up to |v| (1 + 0.05 v^2) + 1) or of erf (a few U), a sum and
      a quotient: at most 16 U (1 + |z|) relative to v, which bounds act(v).
    * mul, res: one rounding each.  Output: half a step.
    """
    Wd, x = np.asarray(Wd, dtype=np.float64), np.asarray(x, dtype=np.float64)
    v = x @ Wd.T
    mag = np.abs(x) @ np.abs(Wd).T
    if codes and out == "f16":
        mag = mag + 72 / 7 * np.abs(x).sum(1)[:, None] * np.abs(Wd).max(1)[None, :]
    err = (x.shape[1] + 4) * U32 * mag
    if bias is not None:
        v = v + np.asarray(bias, dtype=np.float64)
    err = err + 2 * U32 * np.abs(v)
    a = act(v, name)
    if name in ("gelu", "gelu_tanh", "silu"):
        z = 1.6 * np.abs(v) * (1 + 0.05 * v * v)
        err = 1.13 * err + 16 * U32 * (1 + z) * np.maximum(np.abs(a), U32 * np.abs(v)) + 4 * U32 * np.abs(v)
    if mul is not None:
        m = np.asarray(mul, dtype=np.float64)
        a = a * m
        err = err * np.abs(m) + U32 * np.abs(a)
    if res is not None:
        a = a + np.asarray(res, dtype=np.float64)
        err = err + U32 * np.abs(a)
    rel, tiny = HALF_STEP[out]
    return a, err + rel * (np.abs(a) + err) + tiny


def route(logits, k, renormalize):
    """(ids, weights, slots, rows, pos) of usw_expert_route, token by token."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    ids = np.full((T, k), -1, dtype=np.int32)
    weights = np.zeros((T, k))
    pos = np.full((T, k), -1, dtype=np.int32)
    for t in range(T):
        able = [e for e in range(E) if x[t, e] > -np.inf]
        chosen = sorted(able, key=lambda e: (-x[t, e], e))[:k]
        if not chosen:
            continue
        top = x[t, chosen[0]]
        p = {e: 1.0 if x[t, e] == top else math.exp(x[t, e] - top) for e in able}
        total = math.fsum(p[e] for e in (chosen if renormalize else able))
        for j, e in enumerate(chosen):
            ids[t, j], weights[t, j] = e, p[e] / total
    slots = np.zeros(E + 1, dtype=np.int32)
    rows = np.full(T * k, -1, dtype=np.int32)
    s = 0
    for e in range(E):
        slots[e] = s
        for t, j in zip(*np.nonzero(ids == e)):
            rows[s], pos[t, j] = t, s
            s += 1
    slots[E] = s
    return ids, weights, slots, rows, pos


def combine(y, pos, weights, res=None, out="f16"):
    """(out, bound) of usw_expert_combine: k products and sums in fp32."""
    y, w = np.asarray(y, dtype=np.float64), np.asarray(weights, dtype=np.float64)
    pos = np.asarray(pos)
    live = (pos >= 0) & (pos < y.shape[0])
    terms = np.where(live, w, 0.0)[:, :, None] * y[np.where(live, pos, 0)]
    v = terms.sum(1)
    mag = np.abs(terms).sum(1)
    if res is not None:
        v = v + np.asarray(res, dtype=np.float64)
        mag = mag + np.abs(np.asarray(res, dtype=np.float64))
    err = (pos.shape[1] + 2) * U32 * mag
    rel, tiny = HALF_STEP[out]
    return v, err + rel * (np.abs(v) + err) + tiny
