"""The sparse product with an epilogue, of one weight and by expert.

    y = spmm_fused(enc, x, bias=b, act="relu")                 # relu(W_sp x + b)
    h = spmm_fused(gate, x, act="silu", mul=spmm(up, x))       # silu(Wg x) * (Wu x)
    y = spmm_fused(down, h, bias=b2, residual=x)               # x + W2 h + b2

    plan = expert_route(logits, k=2)                           # logits [T][E]
    y = expert_spmm(bank, x, plan.offsets, rows=plan.rows)       # one row per slot
    out = expert_combine(y, plan.pos, plan.weights, residual=x)
    out = expert_ffn(x, logits, 2, up, down, gate=gate, residual=x)   # all of it

Argument marshalling only, like the rest of the binding: the work runs in
libusw's kernels (include/usw.h), on torch's current stream or ``stream``.
Calls may be captured in a HIP graph; a captured call has a workspace of its
own, in the graph's memory pool.  The others share one a stream, which grows
to the largest call's and is kept until ``release_workspaces()``.
"""
from __future__ import annotations

import ctypes
import threading
from dataclasses import dataclass
from functools import lru_cache

from ._lib import (USW_ACT, USW_OUT_F16, USW_OUT_F32, USW_VAL_I4, UswEpilogue, UswExpertFmt, UswFmt,  # noqa: F401
                   check, lib)

__all__ = ["ExpertBank", "RoutePlan", "spmm_fused", "expert_bank", "expert_route", "expert_spmm", "expert_combine",
           "expert_ffn", "release_workspaces"]


@dataclass
class ExpertBank:
    """E TCA-BME encodings of one shape and value type, one after the other
    (torch tensors on a GPU): bitmaps int64 [E][M*K/64], offsets int32
    [E][NGT+1], values uint8 (the experts' padded values), starts int64 [E+1]
    (byte offset of each expert's values), scales fp16 bits [E][M] (INT4) or
    None, nnz over all experts.  ``expert_bank`` makes one."""
    E: int
    M: int
    K: int
    val_type: int
    nnz: int
    bitmaps: "object"
    offsets: "object"
    values: "object"
    starts: "object"
    scales: "object"

    def fmt(self) -> UswExpertFmt:
        return UswExpertFmt(self.E, self.M, self.K, self.val_type, 0, self.nnz, self.values.numel(),
                            self.bitmaps.data_ptr(), self.offsets.data_ptr(), self.values.data_ptr(),
                            self.starts.data_ptr(), self.scales.data_ptr() if self.scales is not None else None)

    @property
    def device(self):
        return self.bitmaps.device


@dataclass
class RoutePlan:
    """What expert_route decides: ids int32 [T][k], weights fp32 [T][k],
    offsets int32 [E+1] (the first slot of each expert), rows int32 [T*k],
    pos int32 [T][k]."""
    ids: "object"
    weights: "object"
    offsets: "object"
    rows: "object"
    pos: "object"


def expert_bank(encodings) -> ExpertBank:
    """The experts' device encodings (``encode``, ``encode_device`` or
    ``to_device``) as one bank.  Copies their buffers."""
    import torch
    encs = list(encodings)
    if not encs:
        raise ValueError("a bank needs at least one expert")
    e0 = encs[0]
    for e in encs:
        if (e.M, e.K, e.val_type) != (e0.M, e0.K, e0.val_type) or (e.gt_m, e.gt_k) != (64, 64):
            raise ValueError("the experts must have one shape, one value type and 64x64 GroupTiles")
        if e.device != e0.device:
            raise ValueError("the experts must be on one device")
    starts = [0]
    for e in encs:
        if e.values.numel() % 16:
            raise ValueError("an expert's values are not padded to 16 bytes")
        starts.append(starts[-1] + e.values.numel())
    scales = None
    if e0.val_type == USW_VAL_I4:
        scales = torch.stack([e.scales.view(torch.int16) for e in encs])
    return ExpertBank(len(encs), e0.M, e0.K, e0.val_type, sum(e.nnz for e in encs),
                      torch.stack([e.bitmaps for e in encs]), torch.stack([e.offsets for e in encs]),
                      torch.cat([e.values for e in encs]), torch.tensor(starts, dtype=torch.int64, device=e0.device),
                      scales)


_OUT = None   # {torch dtype: USW_OUT_*}, filled at the first call


def _out_type(dtype, what):
    import torch
    global _OUT
    if _OUT is None:
        _OUT = {torch.float16: USW_OUT_F16, torch.float32: USW_OUT_F32}
    t = _OUT.get(dtype)
    if t is None:
        raise ValueError(f"{what} must be float16 or float32")
    return t


def _on(device, stream, body):
    """body(raw stream handle) with ``device`` and the call's stream as
    torch's current ones, where its allocations then go."""
    import torch
    if device.type != "cuda":
        raise ValueError("the tensors must be on a GPU")
    if stream is None:
        if torch.cuda.current_device() == device.index:
            return body(torch._C._cuda_getCurrentRawStream(device.index))
        with torch.cuda.device(device):
            return body(torch._C._cuda_getCurrentRawStream(device.index))
    if stream.device_index != device.index:
        raise ValueError("the stream is of another device than the tensors")
    with torch.cuda.stream(stream):
        return body(stream.cuda_stream)


_WS = {}   # (device index, raw stream) -> [workspace, its leading bytes that are zero between calls]
_KEPT = 1 << 16   # leading bytes that a call without counters leaves alone
# Held from taking a workspace until the call is enqueued: two threads on one
# stream share it, and a call's launches must stay together.
_LOCK = threading.Lock()


def _workspace(device, handle, nbytes, counter_bytes):
    """The workspace of a call that needs nbytes > 0, its counter bytes zero.
    Outside capture it is the binding's, one per stream, which orders its uses; every
    call leaves its counters zero again.  A captured call gets one from the
    graph's pool, because a graph may be replayed at the same time as other
    work of the stream it was captured on."""
    import torch
    if torch.cuda.is_current_stream_capturing():
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        if counter_bytes:
            ws[:counter_bytes].zero_()
        return ws
    ent = _WS.get((device.index, handle))
    if ent is None or ent[0].numel() < nbytes:
        ent = _WS[(device.index, handle)] = [torch.empty(nbytes, dtype=torch.uint8, device=device), 0]
    # Counters are none, or 64 KiB and more.  Behind its own a call writes sums
    # or weights, and one without counters does so from 64 KiB on, so no more
    # than that is still zero after it.
    if ent[1] < counter_bytes:
        ent[0][:counter_bytes].zero_()
    ent[1] = counter_bytes or min(ent[1], _KEPT)
    return ent[0]


def release_workspaces() -> None:
    """Gives the workspaces that the fused and expert products keep, one per
    stream they ran on, back to torch's allocator.  Each is as large as the
    largest call on its stream asked for: 2 M K bytes where a weight was
    expanded, up to 1 GiB and more.  The next call on a stream makes its own
    again; graphs have theirs and are not touched."""
    with _LOCK:
        _WS.clear()


def _rows_operand(t, rows, M, device, what):
    """An epilogue operand [rows][M] fp16; rows may be strided, columns not."""
    import torch
    if t.dtype != torch.float16 or t.shape != (rows, M):
        raise ValueError(f"{what} must be [{rows}][{M}] float16")
    if t.device != device:
        raise ValueError(f"{what} is on another device")
    ld, one = t.stride()
    if rows == 1:
        ld = M
    if one != 1 or ld & 7 or ld < M or ld > (1 << 20 if M <= 1 << 20 else 1 << 22) or t.data_ptr() & 15:
        t, ld = t.clone(memory_format=torch.contiguous_format), M
    return t, ld


def _epilogue(bias, act, mul, residual, rows, M, bias_shape, device):
    """(usw_epilogue, the tensors it points to)."""
    code = USW_ACT.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(USW_ACT)}")
    bp = mp = rp = None
    ld_mul = ld_res = 0
    if bias is not None:
        import torch
        if bias.dtype != torch.float16 or bias.shape != bias_shape or bias.device != device:
            raise ValueError(f"bias must be {list(bias_shape)} float16 on the weight's device")
        if not bias.is_contiguous() or bias.data_ptr() & 15:
            bias = bias.clone(memory_format=torch.contiguous_format)
        bp = bias.data_ptr()
    if mul is not None:
        mul, ld_mul = _rows_operand(mul, rows, M, device, "mul")
        mp = mul.data_ptr()
    if residual is not None:
        residual, ld_res = _rows_operand(residual, rows, M, device, "residual")
        rp = residual.data_ptr()
    return UswEpilogue(bp, mp, rp, ld_mul, ld_res, code, 0), (bias, mul, residual)


def _activations(x, K, device):
    import torch
    if x.dtype != torch.float16 or x.dim() != 2 or x.shape[1] != K:
        raise ValueError("x must be [rows][K] float16")
    if x.device != device:
        raise ValueError("x is on another device than the weight")
    if not x.is_contiguous() or x.data_ptr() & 15:
        x = x.clone(memory_format=torch.contiguous_format)
    return x


def _output(y, shape, out_dtype, device, what="y"):
    import torch
    if y is None:
        return torch.empty(shape, dtype=out_dtype or torch.float16, device=device)
    if y.shape != shape or not y.is_contiguous() or y.device != device:
        raise ValueError(f"{what} must be a contiguous {list(shape)} tensor on the weight's device")
    if out_dtype is not None and y.dtype != out_dtype:
        raise ValueError(f"{what} is not of out_dtype")
    return y


@lru_cache(maxsize=4096)
def _fused_sizes(M, K, gt_m, gt_k, val_type, nnz, N, splits):
    """(workspace bytes, counter bytes): a function of the sizes alone."""
    f = UswFmt(M, K, gt_m, gt_k, val_type, 0, nnz, None, None, None, None)
    need, cb = ctypes.c_size_t(), ctypes.c_size_t()
    check(lib().usw_spmm_fused_workspace(ctypes.byref(f), N, splits, ctypes.byref(need), ctypes.byref(cb)),
          "usw_spmm_fused")
    return need.value, cb.value


def spmm_fused(enc, x, bias=None, act: str = "none", mul=None, residual=None, y=None, out_dtype=None,
               splits: int = 0, stream=None):
    """Y [N][M] = residual + mul * act(W_sp . X + bias) (usw_spmm_fused).

    x [N][K] fp16; bias [M], mul [N][M], residual [N][M] fp16, each optional;
    act "none", "relu", "gelu", "gelu_tanh" or "silu".  The sums and the
    epilogue are fp32 and Y (fp16, or ``out_dtype`` float32) is rounded once.
    ``y`` may be ``residual`` itself, and may overlap nothing else that the
    call reads.  mul and residual may be rows of a wider tensor.  Encodings
    have 64x64 GroupTiles and fp16 or INT4 values.
    """
    dev = enc.device

    def body(handle):
        xc = _activations(x, enc.K, dev)
        N, M = xc.shape[0], enc.M
        ep, keep = _epilogue(bias, act, mul, residual, N, M, (M,), dev)
        out = _output(y, (N, M), out_dtype, dev)
        yt = _out_type(out.dtype, "y")
        need, cb = _fused_sizes(M, enc.K, enc.gt_m, enc.gt_k, enc.val_type, enc.nnz, N, splits)
        args = ctypes.byref(enc.fmt()), xc.data_ptr(), out.data_ptr(), yt, N, ctypes.byref(ep), splits
        if need:
            with _LOCK:
                ws = _workspace(dev, handle, need, cb)
                check(lib().usw_spmm_fused(*args, ws.data_ptr(), need, handle), "usw_spmm_fused")
        else:
            check(lib().usw_spmm_fused(*args, None, 0, handle), "usw_spmm_fused")
        return out

    return _on(dev, stream, body)


def _index(t, shape, device, what):
    import torch
    if t.dtype != torch.int32 or t.shape != shape or t.device != device:
        raise ValueError(f"{what} must be {list(shape)} int32 on the same device")
    return t if t.is_contiguous() else t.contiguous()


@lru_cache(maxsize=4096)
def _expert_sizes(E, M, K, val_type, nnz, values_bytes, S):
    f = UswExpertFmt(E, M, K, val_type, 0, nnz, values_bytes, None, None, None, None, None)
    need, cb = ctypes.c_size_t(), ctypes.c_size_t()
    check(lib().usw_expert_spmm_workspace(ctypes.byref(f), S, ctypes.byref(need), ctypes.byref(cb)),
          "usw_expert_spmm")
    return need.value, cb.value


def expert_spmm(bank: ExpertBank, x, offsets, rows=None, bias=None, act: str = "none", mul=None, y=None,
                out_dtype=None, stream=None):
    """The product by expert (usw_expert_spmm): row s of Y [S][M] is
    mul * act(W_e . x + bias[e]) for the expert e whose run
    ``offsets[e] <= s < offsets[e+1]`` holds s.

    offsets int32 [E+1] stays on the GPU.  With ``rows`` (int32 [S]) slot s
    reads x[rows[s]]; without, x[s], and S is x's length.  bias is [E][M],
    mul [S][M].  Rows of Y from offsets[E] on are left as they were (in a Y
    made here: whatever the memory held)."""
    dev = bank.device

    def body(handle):
        xc = _activations(x, bank.K, dev)
        T, M = xc.shape[0], bank.M
        off = _index(offsets, (bank.E + 1,), dev, "offsets")
        S, at = T, None
        if rows is not None:
            if rows.dim() != 1:
                raise ValueError("rows must be [S] int32")
            S = rows.shape[0]
            at = _index(rows, (S,), dev, "rows")
        ep, keep = _epilogue(bias, act, mul, None, S, M, (bank.E, M), dev)
        out = _output(y, (S, M), out_dtype, dev)
        yt = _out_type(out.dtype, "y")
        need, cb = _expert_sizes(bank.E, M, bank.K, bank.val_type, bank.nnz, bank.values.numel(), S)
        args = (ctypes.byref(bank.fmt()), xc.data_ptr(), T, off.data_ptr(), at.data_ptr() if at is not None else None,
                S, out.data_ptr(), yt, ctypes.byref(ep))
        if need:
            with _LOCK:
                ws = _workspace(dev, handle, need, cb)
                check(lib().usw_expert_spmm(*args, ws.data_ptr(), need, handle), "usw_expert_spmm")
        else:
            check(lib().usw_expert_spmm(*args, None, 0, handle), "usw_expert_spmm")
        return out

    return _on(dev, stream, body)


@lru_cache(maxsize=4096)
def _route_size(T, E, k):
    need = ctypes.c_size_t()
    check(lib().usw_expert_route_workspace(T, E, k, ctypes.byref(need)), "usw_expert_route")
    return need.value


def expert_route(logits, k: int, renormalize: bool = True, stream=None) -> RoutePlan:
    """Routing of T tokens (usw_expert_route): logits [T][E] fp16 or fp32.

    Each token's k largest logits are chosen, of equal ones the lower expert;
    -inf and NaN never, so mask padding tokens and unavailable experts with
    -inf.  Weights are softmax values over the chosen experts, or over all
    with ``renormalize=False``.  The chosen pairs are the plan's slots, sorted
    by (expert, token); nothing is read back to the host."""
    import torch
    if logits.dim() != 2:
        raise ValueError("logits must be [T][E]")
    lt = _out_type(logits.dtype, "logits")
    dev = logits.device
    T, E = logits.shape

    def body(handle):
        need = _route_size(T, E, k)
        lg = logits
        ld, one = lg.stride()
        if (one != 1 and E > 1) or (ld < E and T > 1):
            lg, ld = lg.contiguous(), E
        n = T * k
        # One allocation: ids, pos, rows, offsets, and behind them the scratch counts.
        buf = torch.empty(3 * n + E + 1 + need // 4, dtype=torch.int32, device=dev)
        weights = torch.empty((T, k), dtype=torch.float32, device=dev)
        at, step = buf.data_ptr(), 4 * n
        check(lib().usw_expert_route(lg.data_ptr(), lt, ld if T > 1 else 0, T, E, k, renormalize, at,
                                     weights.data_ptr(), at + 3 * step, at + 2 * step, at + step,
                                     at + 3 * step + 4 * (E + 1) if need else None, need, handle), "usw_expert_route")
        two, by = (T, k), (k, 1)
        return RoutePlan(buf.as_strided(two, by), weights, buf.as_strided((E + 1,), (1,), 3 * n),
                         buf.as_strided((n,), (1,), 2 * n), buf.as_strided(two, by, n))

    return _on(dev, stream, body)


def expert_combine(y, pos, weights, residual=None, out=None, out_dtype=None, stream=None):
    """out [T][M] = residual + sum over j of weights[t][j] * y[pos[t][j]]
    (usw_expert_combine), in the order of j, fp32, rounded once.  y [S][M]
    fp16 or fp32, pos int32 [T][k], weights fp32 [T][k], residual [T][M] fp16.
    A slot outside [0, S) counts nothing.  ``out`` may be ``residual``."""
    import torch
    if y.dim() != 2 or pos.dim() != 2:
        raise ValueError("y must be [S][M] and pos [T][k]")
    yt = _out_type(y.dtype, "y")
    dev = y.device
    S, M = y.shape
    T, k = pos.shape

    def body(handle):
        yc = y if y.is_contiguous() and not y.data_ptr() & 15 else y.clone(memory_format=torch.contiguous_format)
        p = _index(pos, (T, k), dev, "pos")
        if weights.dtype != torch.float32 or weights.shape != pos.shape or weights.device != dev:
            raise ValueError("weights must be float32 of pos's shape on the same device")
        w = weights.contiguous()
        rp, ld = None, 0
        if residual is not None:
            res, ld = _rows_operand(residual, T, M, dev, "residual")
            rp = res.data_ptr()
        o = _output(out, (T, M), out_dtype, dev, "out")
        check(lib().usw_expert_combine(yc.data_ptr(), yt, S, M, p.data_ptr(), w.data_ptr(), T, k, rp, ld,
                                       o.data_ptr(), _out_type(o.dtype, "out"), handle), "usw_expert_combine")
        return o

    return _on(dev, stream, body)


def expert_ffn(x, logits, k: int, up: ExpertBank, down: ExpertBank, gate: ExpertBank = None, act: str = "silu",
               up_bias=None, gate_bias=None, down_bias=None, residual=None, renormalize: bool = True, out_dtype=None,
               stream=None):
    """A feed-forward block of experts: x [T][K] goes through the k experts
    of its logits [T][E] and their outputs are joined,

        out = residual + sum over the chosen e of w_e (down_e(h_e) + down_bias_e),
        h_e = act(gate_e x + gate_bias_e) * (up_e x + up_bias_e), or
        h_e = act(up_e x + up_bias_e) without a gate.
    """
    if logits.dim() != 2 or logits.shape[0] != x.shape[0] or logits.shape[1] != up.E:
        raise ValueError("logits must be [T][E]")
    if gate is not None and (gate.E, gate.M, gate.K) != (up.E, up.M, up.K):
        raise ValueError("gate and up must have one shape")
    if gate is None and gate_bias is not None:
        raise ValueError("gate_bias without a gate")
    if (down.E, down.K) != (up.E, up.M):
        raise ValueError("down must have up's experts and take its outputs")
    plan = expert_route(logits, k, renormalize, stream)
    if gate is None:
        h = expert_spmm(up, x, plan.offsets, plan.rows, up_bias, act, stream=stream)
    else:
        u = expert_spmm(up, x, plan.offsets, plan.rows, up_bias, stream=stream)
        h = expert_spmm(gate, x, plan.offsets, plan.rows, gate_bias, act, mul=u, stream=stream)
    y = expert_spmm(down, h, plan.offsets, bias=down_bias, stream=stream)
    return expert_combine(y, plan.pos, plan.weights, residual, out_dtype=out_dtype, stream=stream)
