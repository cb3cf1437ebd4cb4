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
own, in the graph's memory pool.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

from ._lib import (USW_ACT, USW_OUT_F16, USW_OUT_F32, USW_VAL_I4, UswEpilogue, UswExpertFmt, UswFmt,  # noqa: F401
                   check, lib)

__all__ = ["ExpertBank", "RoutePlan", "spmm_fused", "expert_bank", "expert_route", "expert_spmm", "expert_combine",
           "expert_ffn"]


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


class _On:
    """The stream of a call and, for the call's duration, its device (and the
    stream, when it is not the current one) as torch's current ones."""

    def __init__(self, device, stream):
        import torch
        if device.type != "cuda":
            raise ValueError("the tensors must be on a GPU")
        self.stream = torch.cuda.current_stream(device) if stream is None else stream
        if self.stream.device_index != device.index:
            raise ValueError("the stream is of another device than the tensors")
        self.handle = self.stream.cuda_stream
        self.guard = None
        if stream is not None:
            self.guard = torch.cuda.stream(stream)
        elif torch.cuda.current_device() != device.index:
            self.guard = torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            return self.guard.__exit__(*exc)
        return False

    def workspace(self, nbytes, counter_bytes):
        """The workspace of a call that needs nbytes > 0, its counter bytes
        zero.  Outside capture it is the binding's, one per stream; a captured
        call gets one from the graph's pool, because a graph may be replayed
        at the same time as other work of the stream it was captured on."""
        import torch
        if torch.cuda.is_current_stream_capturing():
            ws = torch.empty(nbytes, dtype=torch.uint8, device=self.stream.device)
            if counter_bytes:
                ws[:counter_bytes].zero_()
            return ws
        from . import _workspace
        return _workspace(self.stream, nbytes, counter_bytes)


def _rows_operand(t, rows, M, device, what):
    """An epilogue operand [rows][M] fp16; rows may be strided, columns not."""
    import torch
    if t.dtype != torch.float16 or t.shape != (rows, M):
        raise ValueError(f"{what} must be [{rows}][{M}] float16")
    if t.device != device:
        raise ValueError(f"{what} is on another device")
    if t.stride(1) != 1 or t.stride(0) % 8 or t.stride(0) < M or t.data_ptr() & 15:
        t = t.contiguous()
    return t


def _epilogue(bias, act, mul, residual, rows, M, bias_shape, device):
    """(usw_epilogue, the tensors it points to)."""
    import torch
    code = USW_ACT.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(USW_ACT)}")
    keep = []
    ep = UswEpilogue(None, None, None, 0, 0, code, 0)
    if bias is not None:
        if bias.dtype != torch.float16 or tuple(bias.shape) != bias_shape or bias.device != device:
            raise ValueError(f"bias must be {list(bias_shape)} float16 on the weight's device")
        if not bias.is_contiguous() or bias.data_ptr() & 15:
            bias = bias.clone(memory_format=torch.contiguous_format)
        keep.append(bias)
        ep.bias = bias.data_ptr()
    if mul is not None:
        mul = _rows_operand(mul, rows, M, device, "mul")
        keep.append(mul)
        ep.mul, ep.ld_mul = mul.data_ptr(), mul.stride(0) if rows > 1 else 0
    if residual is not None:
        residual = _rows_operand(residual, rows, M, device, "residual")
        keep.append(residual)
        ep.res, ep.ld_res = residual.data_ptr(), residual.stride(0) if rows > 1 else 0
    return ep, keep


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
    if tuple(y.shape) != shape or not y.is_contiguous() or y.device != device:
        raise ValueError(f"{what} must be a contiguous {list(shape)} tensor on the weight's device")
    if out_dtype is not None and y.dtype != out_dtype:
        raise ValueError(f"{what} is not of out_dtype")
    return y


def spmm_fused(enc, x, bias=None, act: str = "none", mul=None, residual=None, y=None, out_dtype=None,
               splits: int = 0, stream=None):
    """Y [N][M] = residual + mul * act(W_sp . X + bias) (usw_spmm_fused).

    x [N][K] fp16; bias [M], mul [N][M], residual [N][M] fp16, each optional;
    act "none", "relu", "gelu", "gelu_tanh" or "silu".  The sums and the
    epilogue are fp32 and Y (fp16, or ``out_dtype`` float32) is rounded once.
    ``y`` may be ``residual`` itself.  mul and residual may be rows of a wider
    tensor.  Encodings have 64x64 GroupTiles and fp16 or INT4 values.
    """
    dev = enc.device
    with _On(dev, stream) as on:
        x = _activations(x, enc.K, dev)
        N = x.shape[0]
        ep, keep = _epilogue(bias, act, mul, residual, N, enc.M, (enc.M,), dev)
        y = _output(y, (N, enc.M), out_dtype, dev)
        yt = _out_type(y.dtype, "y")
        f = enc.fmt()
        L = lib()
        need, cb = ctypes.c_size_t(), ctypes.c_size_t()
        check(L.usw_spmm_fused_workspace(ctypes.byref(f), N, splits, ctypes.byref(need), ctypes.byref(cb)),
              "usw_spmm_fused")
        ws = on.workspace(need.value, cb.value) if need.value else None
        check(L.usw_spmm_fused(ctypes.byref(f), x.data_ptr(), y.data_ptr(), yt, N, ctypes.byref(ep), splits,
                               ws.data_ptr() if ws is not None else None, need.value, on.handle), "usw_spmm_fused")
    return y


def _index(t, shape, device, what):
    import torch
    if t.dtype != torch.int32 or tuple(t.shape) != shape or t.device != device:
        raise ValueError(f"{what} must be {list(shape)} int32 on the same device")
    return t if t.is_contiguous() else t.contiguous()


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
    with _On(dev, stream) as on:
        x = _activations(x, bank.K, dev)
        T = x.shape[0]
        offsets = _index(offsets, (bank.E + 1,), dev, "offsets")
        S = T
        if rows is not None:
            if rows.dim() != 1:
                raise ValueError("rows must be [S] int32")
            S = rows.shape[0]
            rows = _index(rows, (S,), dev, "rows")
        ep, keep = _epilogue(bias, act, mul, None, S, bank.M, (bank.E, bank.M), dev)
        y = _output(y, (S, bank.M), out_dtype, dev)
        yt = _out_type(y.dtype, "y")
        f = bank.fmt()
        L = lib()
        need, cb = ctypes.c_size_t(), ctypes.c_size_t()
        check(L.usw_expert_spmm_workspace(ctypes.byref(f), S, ctypes.byref(need), ctypes.byref(cb)),
              "usw_expert_spmm")
        ws = on.workspace(need.value, cb.value) if need.value else None
        check(L.usw_expert_spmm(ctypes.byref(f), x.data_ptr(), T, offsets.data_ptr(),
                                rows.data_ptr() if rows is not None else None, S, y.data_ptr(), yt, ctypes.byref(ep),
                                ws.data_ptr() if ws is not None else None, need.value, on.handle), "usw_expert_spmm")
    return y


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
    with _On(dev, stream) as on:
        if T > 1 and (logits.stride(1) != 1 or logits.stride(0) < E) or (E > 1 and logits.stride(1) != 1):
            logits = logits.contiguous()
        L = lib()
        need = ctypes.c_size_t()
        check(L.usw_expert_route_workspace(T, E, k, ctypes.byref(need)), "usw_expert_route")
        ints = torch.empty(3 * T * k + E + 1, dtype=torch.int32, device=dev)
        ids, pos, rows = (ints[i * T * k:(i + 1) * T * k] for i in range(3))
        offsets = ints[3 * T * k:]
        weights = torch.empty((T, k), dtype=torch.float32, device=dev)
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev) if need.value else None
        check(L.usw_expert_route(logits.data_ptr(), lt, logits.stride(0) if T > 1 else 0, T, E, k, int(renormalize),
                                 ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(),
                                 pos.data_ptr(), ws.data_ptr() if ws is not None else None, need.value, on.handle),
              "usw_expert_route")
    return RoutePlan(ids.view(T, k), weights, offsets, rows, pos.view(T, k))


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
    with _On(dev, stream) as on:
        if not y.is_contiguous() or y.data_ptr() & 15:
            y = y.clone(memory_format=torch.contiguous_format)
        pos = _index(pos, (T, k), dev, "pos")
        if weights.dtype != torch.float32 or weights.shape != pos.shape or weights.device != dev:
            raise ValueError("weights must be float32 of pos's shape on the same device")
        weights = weights.contiguous()
        ld = 0
        if residual is not None:
            residual = _rows_operand(residual, T, M, dev, "residual")
            ld = residual.stride(0) if T > 1 else 0
        out = _output(out, (T, M), out_dtype, dev, "out")
        check(lib().usw_expert_combine(y.data_ptr(), yt, S, M, pos.data_ptr(), weights.data_ptr(), T, k,
                                       residual.data_ptr() if residual is not None else None, ld, out.data_ptr(),
                                       _out_type(out.dtype, "out"), on.handle), "usw_expert_combine")
    return out


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
