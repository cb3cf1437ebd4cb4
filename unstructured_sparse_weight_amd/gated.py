"""The gated feed-forward block in one product, and the gradients of the
sparse products.

    h = spmm_gated(gate, up, x)                                  # silu(Wg x) * (Wu x)
    h, g, u = spmm_gated(gate, up, x, save=True)                 # with what the backward pass needs
    y = spmm_fused(down, h, residual=x_in)

    d = spmm_backward(down, h, dy)                               # d.x [N][K], d.values [nnz]
    b = spmm_gated_backward(gate, up, x, g, u, d.x)              # b.x, b.gate, b.up
    kept(gate).add_(b.gate, alpha=-lr)                           # the mask is fixed: only kept values move

Argument marshalling only; the work runs in libusw's kernels (include/usw.h),
on torch's current stream or ``stream``, with the workspaces of fused.py.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from functools import lru_cache

from ._lib import (USW_ACT, USW_GRAD_BIAS, USW_GRAD_VALUES, USW_GRAD_X, USW_OUT_F16, USW_VAL_F16, UswFmt, UswGated,
                   UswGatedGrad, check, lib)
from .fused import _LOCK, _activations, _on, _out_type, _output, _workspace

__all__ = ["ProductGrads", "GatedGrads", "spmm_gated", "spmm_backward", "spmm_gated_backward", "kept"]


@dataclass
class ProductGrads:
    """Gradients of y = W_sp x + b: x [N][K], values [nnz] in the order of the
    encoding's values, bias fp32 [M]; None where not asked for."""
    x: "object" = None
    values: "object" = None
    bias: "object" = None


@dataclass
class GatedGrads:
    """Gradients of the gated block: x fp16 [N][K], gate and up fp16 [nnz] in
    the order of each encoding's values, gate_bias and up_bias fp32 [M]; None
    where not asked for."""
    x: "object" = None
    gate: "object" = None
    up: "object" = None
    gate_bias: "object" = None
    up_bias: "object" = None


def kept(enc):
    """The kept values of an fp16 encoding on a GPU, as the fp16 [nnz] view of
    its buffer that a gradient's ``values`` matches: update it in place."""
    import torch
    if enc.val_type != USW_VAL_F16:
        raise ValueError("INT4 values are frozen codes")
    return enc.values.view(torch.float16)[:enc.nnz]


def _pair(gate, up):
    if (gate.M, gate.K, gate.val_type) != (up.M, up.K, up.val_type):
        raise ValueError("gate and up must have one shape and one value type")
    if gate.device != up.device:
        raise ValueError("gate and up must be on one device")


def _bare(enc):
    return enc.M, enc.K, enc.gt_m, enc.gt_k, enc.val_type, 0, enc.nnz


def _sizes(query, *args):
    need, cb = ctypes.c_size_t(), ctypes.c_size_t()
    check(query(*args, ctypes.byref(need), ctypes.byref(cb)), query.__name__)
    return need.value, cb.value


def _fmt(bare):
    return ctypes.byref(UswFmt(*bare, None, None, None, None))


@lru_cache(maxsize=4096)
def _gated_sizes(gate, up, N):
    return _sizes(lib().usw_spmm_gated_workspace, _fmt(gate), _fmt(up), N)


@lru_cache(maxsize=4096)
def _backward_sizes(bare, N, out_type, grads):
    return _sizes(lib().usw_spmm_backward_workspace, _fmt(bare), N, out_type, grads)


@lru_cache(maxsize=4096)
def _gated_backward_sizes(gate, up, N, grads):
    return _sizes(lib().usw_spmm_gated_backward_workspace, _fmt(gate), _fmt(up), N, grads)


def _run(device, handle, need, cb, call, where):
    """call(workspace pointer, bytes) with a workspace of the stream's (none of these calls asks for 0 bytes)."""
    with _LOCK:
        check(call(_workspace(device, handle, need, cb).data_ptr(), need), where)


def _rows(t, N, M, device, what):
    import torch
    if t.dtype != torch.float16 or t.shape != (N, M):
        raise ValueError(f"{what} must be [{N}][{M}] float16")
    if t.device != device:
        raise ValueError(f"{what} is on another device")
    if not t.is_contiguous() or t.data_ptr() & 15:
        t = t.clone(memory_format=torch.contiguous_format)
    return t


def _bias(t, M, device, what):
    import torch
    if t is None:
        return None
    if t.dtype != torch.float16 or t.shape != (M,) or t.device != device:
        raise ValueError(f"{what} must be [{M}] float16 on the weights' device")
    if not t.is_contiguous() or t.data_ptr() & 15:
        t = t.clone(memory_format=torch.contiguous_format)
    return t


def _act(act):
    code = USW_ACT.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(USW_ACT)}")
    return code


def _ptr(t):
    return None if t is None else t.data_ptr()


def spmm_gated(gate, up, x, gate_bias=None, up_bias=None, act: str = "silu", save: bool = False, y=None, out_dtype=None,
               stream=None):
    """h [N][M] = act(Wg x + bg) * (Wu x + bu) (usw_spmm_gated).

    gate and up are TCA-BME encodings of one shape and value type (fp16 or
    INT4, 64x64 GroupTiles); x [N][K], the biases [M], fp16.  Sums, activation
    and product are fp32; h (fp16, or ``out_dtype`` float32) is rounded once.
    With ``save`` returns (h, g, u), the pre-activations g = Wg x + bg and
    u = Wu x + bu in fp16 for ``spmm_gated_backward``."""
    import torch
    _pair(gate, up)
    code = _act(act)
    dev = gate.device

    def body(handle):
        xc = _activations(x, gate.K, dev)
        N, M = xc.shape[0], gate.M
        bg, bu = _bias(gate_bias, M, dev, "gate_bias"), _bias(up_bias, M, dev, "up_bias")
        h = _output(y, (N, M), out_dtype, dev)
        yt = _out_type(h.dtype, "y")
        pre_g, pre_u = torch.empty((2, N, M), dtype=torch.float16, device=dev).unbind() if save else (None, None)
        need, cb = _gated_sizes(_bare(gate), _bare(up), N)
        opt = UswGated(_ptr(bg), _ptr(bu), _ptr(pre_g), _ptr(pre_u), code, 0)
        fg, fu = gate.fmt(), up.fmt()
        _run(dev, handle, need, cb,
             lambda ws, n: lib().usw_spmm_gated(ctypes.byref(fg), ctypes.byref(fu), xc.data_ptr(), h.data_ptr(), yt, N,
                                                ctypes.byref(opt), ws, n, handle), "usw_spmm_gated")
        return (h, pre_g, pre_u) if save else h

    return _on(dev, stream, body)


def spmm_backward(enc, x, dy, dx: bool = True, values: bool = None, bias: bool = False, out_dtype=None,
                  stream=None) -> ProductGrads:
    """Gradients of y = W_sp x + b from dy [N][M] fp16 (usw_spmm_backward): of
    x (``dx``), of the kept values (``values``, by default where the encoding
    has fp16 values; INT4 weights are frozen) and of b (``bias``).  x [N][K]
    fp16 is read for the values only and may be None without them.  Sums are
    fp32; dx and the values' gradient are fp16 or ``out_dtype`` float32, the
    bias's fp32.  The gradient of a residual is dy itself."""
    import torch
    values = enc.val_type == USW_VAL_F16 if values is None else values
    if values and enc.val_type != USW_VAL_F16:
        raise ValueError("INT4 values are frozen codes: they have no gradient")
    if values and x is None:
        raise ValueError("the values' gradient needs x")
    dev = enc.device
    dtype = out_dtype or torch.float16
    ot = _out_type(dtype, "out_dtype")

    def body(handle):
        if dy.dim() != 2:
            raise ValueError("dy must be [N][M] float16")
        N, M, K = dy.shape[0], enc.M, enc.K
        d = _rows(dy, N, M, dev, "dy")
        xc = _rows(x, N, K, dev, "x") if values else None
        r = ProductGrads(torch.empty((N, K), dtype=dtype, device=dev) if dx else None,
                         torch.empty(enc.nnz, dtype=dtype, device=dev) if values else None,
                         torch.empty(M, dtype=torch.float32, device=dev) if bias else None)
        grads = (USW_GRAD_X if dx else 0) | (USW_GRAD_VALUES if values and enc.nnz else 0) | (USW_GRAD_BIAS if bias else 0)
        need, cb = _backward_sizes(_bare(enc), N, ot, grads)
        f = enc.fmt()
        _run(dev, handle, need, cb,
             lambda ws, n: lib().usw_spmm_backward(ctypes.byref(f), _ptr(xc), d.data_ptr(), N, _ptr(r.x),
                                                   _ptr(r.values) if enc.nnz else None, _ptr(r.bias), ot, ws, n, handle),
             "usw_spmm_backward")
        return r

    return _on(dev, stream, body)


def spmm_gated_backward(gate, up, x, g, u, dy, act: str = "silu", dx: bool = True, values: bool = None,
                        bias: bool = False, stream=None) -> GatedGrads:
    """Gradients of the gated block from dy [N][M] (usw_spmm_gated_backward), with
    the g and u that ``spmm_gated(..., save=True)`` returned and its ``act``.
    x, g, u and dy are fp16; arguments otherwise as ``spmm_backward``, both
    weights and both biases together.  The products take dg = dy u act'(g) and
    du = dy act(g) in fp16 (up to 32 rows with the remainders of that rounding),
    so all but the biases' gradients (fp32) are fp16, and a loss is scaled as for
    any fp16 gradient."""
    import torch
    _pair(gate, up)
    code = _act(act)
    values = gate.val_type == USW_VAL_F16 if values is None else values
    if values and gate.val_type != USW_VAL_F16:
        raise ValueError("INT4 values are frozen codes: they have no gradient")
    if values and x is None:
        raise ValueError("the values' gradient needs x")
    dev = gate.device

    def body(handle):
        if dy.dim() != 2:
            raise ValueError("dy must be [N][M] float16")
        N, M, K = dy.shape[0], gate.M, gate.K
        d, gc, uc = _rows(dy, N, M, dev, "dy"), _rows(g, N, M, dev, "g"), _rows(u, N, M, dev, "u")
        xc = _rows(x, N, K, dev, "x") if values else None

        def out(wanted, shape, dtype=torch.float16):
            return torch.empty(shape, dtype=dtype, device=dev) if wanted else None

        r = GatedGrads(out(dx, (N, K)), out(values, gate.nnz), out(values, up.nnz), out(bias, M, torch.float32),
                       out(bias, M, torch.float32))
        some = values and (gate.nnz or up.nnz)
        grads = (USW_GRAD_X if dx else 0) | (USW_GRAD_VALUES if some else 0) | (USW_GRAD_BIAS if bias else 0)
        need, cb = _gated_backward_sizes(_bare(gate), _bare(up), N, grads)
        a = UswGatedGrad(d.data_ptr(), gc.data_ptr(), uc.data_ptr(), _ptr(r.x), _ptr(r.gate) if gate.nnz else None,
                         _ptr(r.up) if up.nnz else None, _ptr(r.gate_bias), _ptr(r.up_bias), code, 0)
        fg, fu = gate.fmt(), up.fmt()
        _run(dev, handle, need, cb,
             lambda ws, n: lib().usw_spmm_gated_backward(ctypes.byref(fg), ctypes.byref(fu), _ptr(xc), N, ctypes.byref(a),
                                                         ws, n, handle), "usw_spmm_gated_backward")
        return r

    return _on(dev, stream, body)
