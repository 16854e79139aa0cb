"""The layers around the products, for torch tensors on the GPU: the dense
layer with bias, activation and residual, the gated up-projection and layer
norm, each with its backward pass.  Argument checks and marshalling only: the
arithmetic is in the HIP kernels behind the C ABI of ``include/gemm.h``.

Rows may have any stride; weights are ``K x N`` views whose storage is
``K x N`` or ``N x K`` (a transposed view, as ``weight.t()`` of weights kept
outputs by inputs).  Leading dimensions of activations are folded into rows.
Outputs and workspaces are allocated when not given, on the call's stream; the
library itself allocates nothing.  A status other than GEMM_OK raises
``GemmError``, a tensor of the wrong shape, type or layout ``ValueError`` or
``TypeError`` before anything is launched.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import binding
from .binding import (ACTIVATIONS, GEMM_OK, GEMM_OP_N, GEMM_OP_T, GatedBackwardParams, GatedParams, GemmError,
                      LayerNormParams, LinearBackwardParams, LinearParams)

_KIND = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32"}
_functions = {}
_MAX_INT = 2 ** 31 - 1


def _function(stem, kind):
    """(entry point, workspace function or None) of a layer, looked up once."""
    f = _functions.get((stem, kind))
    if f is None:
        lib = binding.load()
        f = (getattr(lib, f"{stem}_{kind}"), getattr(lib, stem + "_workspace", None))
        _functions[stem, kind] = f
    return f


def _activation(name):
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"unknown activation {name!r}: one of {sorted(ACTIVATIONS)}") from None


def _kind16(t, name):
    if t.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"{name} must be float16 or bfloat16, not {t.dtype}")
    return _KIND[t.dtype]


def _rows(t, cols, name, like, rows=None, dtype=None):
    """(2-D form, row stride) of an activation-like tensor with ``cols``
    contiguous columns on ``like``'s device."""
    if t.device != like.device or not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU of the first argument")
    if t.dtype != (like.dtype if dtype is None else dtype):
        raise TypeError(f"{name} must be {like.dtype if dtype is None else dtype}, not {t.dtype}")
    if t.dim() != 2:
        if t.dim() == 0:
            raise ValueError(f"{name} needs at least one dimension")
        t = t.reshape(-1 if t.numel() else _count(t.shape[:-1]), t.shape[-1])
    r, c = t.shape
    if c != cols or (rows is not None and r != rows):
        raise ValueError(f"{name} is {r} x {c}, expected {rows if rows is not None else 'any'} x {cols}")
    s0, s1 = t.stride()
    if s1 != 1 and c > 1:
        raise ValueError(f"{name} must have contiguous rows (strides {t.stride()})")
    ld = s0 if r > 1 else max(cols, 1)
    if ld > _MAX_INT:
        raise ValueError(f"{name}'s row stride {ld} is out of range")
    return t, ld


def _count(shape):
    n = 1
    for s in shape:
        n *= s
    return n


def _weight(w, name, like):
    """(op, leading dimension) of a K x N weight view."""
    if w.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    if w.device != like.device:
        raise ValueError(f"{name} must be on the GPU of the first argument")
    if w.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, not {w.dtype}")
    op, ld = binding._layout(w, name)
    if ld > _MAX_INT:
        raise ValueError(f"{name}'s stride {ld} is out of range")
    return op, ld


def _vector(v, n, name, like, dtype=None):
    if v is None:
        return None
    if v.device != like.device:
        raise ValueError(f"{name} must be on the GPU of the first argument")
    if v.dtype != (like.dtype if dtype is None else dtype):
        raise TypeError(f"{name} must be {like.dtype if dtype is None else dtype}, not {v.dtype}")
    if v.dim() != 1 or v.shape[0] != n or (n > 1 and v.stride(0) != 1):
        raise ValueError(f"{name} must be {n} contiguous elements")
    return v.data_ptr() if n else None


def _out(t, shape, like, name, dtype=None):
    """An output of ``shape`` (allocated when not given), its row stride."""
    dtype = like.dtype if dtype is None else dtype
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=like.device)
        return t, max(shape[-1], 1)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} is {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dim() != 2 and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t, _rows(t, shape[-1], name, like, dtype=dtype)[1]


def _grad_like(w, op, given, name):
    """A gradient of weight w (K x N view), in w's kind of storage."""
    if given is not None:
        if given.shape != w.shape or given.dtype != w.dtype or given.device != w.device:
            raise ValueError(f"{name} must match its weight")
        op_g, ld = binding._layout(given, name)
        if op_g != op and min(given.shape) > 1:
            raise ValueError(f"{name} must be stored as its weight is")
        k, n = given.shape
        return given, max(ld, (k if op == GEMM_OP_T else n), 1)
    k, n = w.shape
    if op == GEMM_OP_T:
        return torch.empty((n, k), dtype=w.dtype, device=w.device).t(), max(k, 1)
    return torch.empty((k, n), dtype=w.dtype, device=w.device), max(n, 1)


def _ptr(t):
    return t.data_ptr() if t is not None and t.numel() else None


@contextlib.contextmanager
def _on(device, stream, tensors):
    """The call's device and stream as the current ones, so that what the call
    allocates belongs to that stream; yields the stream's handle.  Tensors of
    another stream are held for this one."""
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
            return
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        with torch.cuda.stream(stream):
            yield stream.cuda_stream
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _workspace(size_of, stem, params, given, device):
    """(address, bytes) of a call's workspace, and the tensor that holds it."""
    need = ctypes.c_size_t()
    rc = size_of(ctypes.byref(params), ctypes.byref(need))
    if rc != GEMM_OK:
        raise GemmError(rc, stem)
    if given is not None:
        if given.dtype != torch.uint8 or given.device != device or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the call's GPU")
        return given.data_ptr(), given.numel(), given
    if need.value == 0:
        return None, 0, None
    t = torch.empty(need.value, dtype=torch.uint8, device=device)
    return t.data_ptr(), need.value, t


def _gpu(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")


# ------------------------------------------------------------- dense layer --

def linear(x, w, bias=None, residual=None, activation="none", save_pre=False, out_dtype=None, y=None, pre=None,
           workspace=None, stream=None):
    """``act(x w + bias) + residual`` for float16 or bfloat16 x (..., K) and w
    (K x N), summed in FP32.  ``out_dtype`` is x's type (None) or
    torch.float32, also the residual's; ``activation`` none, relu, gelu (exact),
    gelu_tanh or silu.  With ``save_pre`` (or ``pre`` given) also returns the
    sums before the activation, in x's type, for ``linear_backward``.  ``y``
    may be the residual itself."""
    _gpu(x, "x")
    kind = _kind16(x, "x")
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    op, ldw = _weight(w, "w", x)
    K, N = w.shape
    x2, ldx = _rows(x, K, "x", x)
    M = x2.shape[0]
    act = _activation(activation)
    if out_dtype is None:
        out_dtype = x.dtype if y is None else y.dtype
    if out_dtype not in (x.dtype, torch.float32):
        raise TypeError(f"out_dtype must be {x.dtype} or float32")
    lead = tuple(x.shape[:-1])
    b = _vector(bias, N, "bias", x)
    r2 = None
    ldr = 0
    if residual is not None:
        if tuple(residual.shape) != lead + (N,):
            raise ValueError(f"residual is {tuple(residual.shape)}, expected {lead + (N,)}")
        r2, ldr = _rows(residual, N, "residual", x, M, out_dtype)
    with _on(x.device, stream, (x, w, bias, residual, y, pre, workspace)) as handle:
        y, ldy = _out(y, lead + (N,), x, "y", out_dtype)
        ldp = 0
        if save_pre or pre is not None:
            pre, ldp = _out(pre, lead + (N,), x, "pre")
        f, size_of = _function("gemm_linear", kind)
        params = LinearParams(M, N, K, op, ldx, ldw, ldy, ldr, ldp, act, out_dtype == torch.float32)
        ws, ws_bytes, held = _workspace(size_of, "gemm_linear", params, workspace, x.device)
        rc = f(ctypes.byref(params), _ptr(x2), _ptr(w), b, _ptr(r2), _ptr(y), _ptr(pre), ws, ws_bytes, handle)
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_linear")
    return y if pre is None else (y, pre)


def linear_backward(dy, x, w, pre=None, activation="none", need_input=True, need_weight=True, need_bias=True,
                    dx=None, dw=None, dbias=None, workspace=None, stream=None):
    """Gradients ``(dx, dw, dbias)`` of ``linear`` from that of its output (in
    x's type) and its saved ``pre`` (not needed without an activation); None
    for those not needed.  The residual's gradient is dy.  dw has w's shape and
    storage."""
    _gpu(dy, "dy")
    kind = _kind16(dy, "dy")
    op, ldw = _weight(w, "w", dy)
    K, N = w.shape
    act = _activation(activation)
    dy2, lddy = _rows(dy, N, "dy", dy)
    M = dy2.shape[0]
    x2, ldx = _rows(x, K, "x", dy, M)
    p2, ldp = None, 0
    if act:
        if pre is None:
            raise ValueError("the backward pass of an activation needs pre")
        p2, ldp = _rows(pre, N, "pre", dy, M)
    with _on(dy.device, stream, (dy, x, w, pre, dx, dw, dbias, workspace)) as handle:
        lddx = lddw = 0
        if need_input or dx is not None:
            dx, lddx = _out(dx, tuple(x.shape), x, "dx")
        if need_weight or dw is not None:
            dw, lddw = _grad_like(w, op, dw, "dw")
        if need_bias and dbias is None:
            dbias = torch.empty(N, dtype=dy.dtype, device=dy.device)
        db = _vector(dbias, N, "dbias", dy)
        f, size_of = _function("gemm_linear_backward", kind)
        params = LinearBackwardParams(M, N, K, op, lddy, ldx, ldw, ldp, lddx, lddw, act)
        ws, ws_bytes, held = _workspace(size_of, "gemm_linear_backward", params, workspace, dy.device)
        rc = f(ctypes.byref(params), _ptr(dy2), _ptr(x2), _ptr(w), _ptr(p2), _ptr(dx), _ptr(dw), db, ws, ws_bytes,
               handle)
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_linear_backward")
    return dx, dw, dbias


# ----------------------------------------------------- gated up-projection --

def gated(x, wg, wu, activation="silu", save_pre=False, h=None, workspace=None, stream=None):
    """``act(x wg) * (x wu)`` for float16 or bfloat16 x (..., K) and the
    K x F weights wg and wu (of one storage and stride: the halves of one
    K x 2F matrix will do), both products in one kernel.  With ``save_pre``
    returns ``(h, g, u)``, the products for ``gated_backward``."""
    _gpu(x, "x")
    kind = _kind16(x, "x")
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    op, ldw = _gate_weights(wg, wu, x)
    K, F = wg.shape
    x2, ldx = _rows(x, K, "x", x)
    act = _activation(activation)
    lead = tuple(x.shape[:-1])
    with _on(x.device, stream, (x, wg, wu, h, workspace)) as handle:
        h, ldh = _out(h, lead + (F,), x, "h")
        g = u = None
        if save_pre:
            g = torch.empty(lead + (F,), dtype=x.dtype, device=x.device)
            u = torch.empty_like(g)
        f, size_of = _function("gemm_gated", kind)
        params = GatedParams(x2.shape[0], F, K, op, ldx, ldw, ldh, max(F, 1), act)
        ws, ws_bytes, held = _workspace(size_of, "gemm_gated", params, workspace, x.device)
        rc = f(ctypes.byref(params), _ptr(x2), _ptr(wg), _ptr(wu), _ptr(h), _ptr(g), _ptr(u), ws, ws_bytes, handle)
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_gated")
    return (h, g, u) if save_pre else h


def _gate_weights(wg, wu, like):
    op, ld = _weight(wg, "wg", like)
    op_u, ld_u = _weight(wu, "wu", like)
    if wu.shape != wg.shape:
        raise ValueError(f"wg is {tuple(wg.shape)}, wu {tuple(wu.shape)}")
    if op != op_u or ld != ld_u:
        raise ValueError("wg and wu must have one storage order and stride")
    return op, ld


def gated_backward(dh, x, wg, wu, g, u, activation="silu", need_input=True, need_weight=True, dx=None, dwg=None,
                   dwu=None, workspace=None, stream=None):
    """Gradients ``(dx, dwg, dwu)`` of ``gated`` from that of its output and
    its saved products g and u; None for those not needed."""
    _gpu(dh, "dh")
    kind = _kind16(dh, "dh")
    op, ldw = _gate_weights(wg, wu, dh)
    K, F = wg.shape
    act = _activation(activation)
    dh2, lddh = _rows(dh, F, "dh", dh)
    M = dh2.shape[0]
    x2, ldx = _rows(x, K, "x", dh, M)
    g2, ldp = _rows(g, F, "g", dh, M)
    u2, ldu = _rows(u, F, "u", dh, M)
    if ldp != ldu:
        raise ValueError("g and u must have one row stride")
    if (dwg is None) != (dwu is None):
        raise ValueError("dwg and dwu are given together or not at all")
    with _on(dh.device, stream, (dh, x, wg, wu, g, u, dx, dwg, dwu, workspace)) as handle:
        lddx = lddw = 0
        if need_input or dx is not None:
            dx, lddx = _out(dx, tuple(x.shape), x, "dx")
        if need_weight or dwg is not None:
            dwg, lddw = _grad_like(wg, op, dwg, "dwg")
            dwu, lddu = _grad_like(wu, op, dwu, "dwu")
            if lddw != lddu:
                raise ValueError("dwg and dwu must have one stride")
        f, size_of = _function("gemm_gated_backward", kind)
        params = GatedBackwardParams(M, F, K, op, lddh, ldx, ldw, ldp, lddx, lddw, act)
        ws, ws_bytes, held = _workspace(size_of, "gemm_gated_backward", params, workspace, dh.device)
        rc = f(ctypes.byref(params), _ptr(dh2), _ptr(x2), _ptr(wg), _ptr(wu), _ptr(g2), _ptr(u2), _ptr(dx), _ptr(dwg),
               _ptr(dwu), ws, ws_bytes, handle)
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_gated_backward")
    return dx, dwg, dwu


# --------------------------------------------------------------- layer norm --

def _norm_weights(weight, bias, N, x):
    """(addresses, whether they are FP32) of layer norm's weight and bias."""
    dtype = next((t.dtype for t in (weight, bias) if t is not None), torch.float32)
    if dtype not in (x.dtype, torch.float32):
        raise TypeError(f"weight and bias must be {x.dtype} or float32, not {dtype}")
    return _vector(weight, N, "weight", x, dtype), _vector(bias, N, "bias", x, dtype), dtype


def layer_norm(x, weight=None, bias=None, eps=1e-5, save_stats=False, y=None, stream=None):
    """Layer norm over the last dimension of a float32, float16 or bfloat16
    tensor; weight and bias in x's type or float32.  With ``save_stats``
    returns ``(y, mean, rstd)``, the statistics of each row in float32 for
    ``layer_norm_backward``."""
    _gpu(x, "x")
    if x.dtype not in _KIND:
        raise TypeError(f"x must be float32, float16 or bfloat16, not {x.dtype}")
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    N = x.shape[-1]
    x2, ldx = _rows(x, N, "x", x)
    M = x2.shape[0]
    w, b, wt = _norm_weights(weight, bias, N, x)
    with _on(x.device, stream, (x, weight, bias, y)) as handle:
        y, ldy = _out(y, tuple(x.shape), x, "y")
        mean = rstd = None
        if save_stats:
            mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
            rstd = torch.empty_like(mean)
            if N == 0:
                mean.zero_(), rstd.zero_()
        f = _function("gemm_layer_norm", _KIND[x.dtype])[0]
        params = LayerNormParams(M, N, ldx, ldy, 0, wt == torch.float32, eps)
        rc = f(ctypes.byref(params), _ptr(x2), w, b, _ptr(y), _ptr(mean), _ptr(rstd), handle)
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_layer_norm")
    return (y, mean, rstd) if save_stats else y


def layer_norm_backward(dy, x, weight, mean, rstd, need_weight=True, dx=None, dweight=None, dbias=None,
                        workspace=None, stream=None):
    """Gradients ``(dx, dweight, dbias)`` of ``layer_norm`` from that of its
    output and its saved statistics; the last two in weight's type (float32
    without one), None unless ``need_weight``."""
    _gpu(dy, "dy")
    if dy.dtype not in _KIND:
        raise TypeError(f"dy must be float32, float16 or bfloat16, not {dy.dtype}")
    if dy.dim() < 1:
        raise ValueError("dy needs at least one dimension")
    N = dy.shape[-1]
    dy2, lddy = _rows(dy, N, "dy", dy)
    M = dy2.shape[0]
    x2, ldx = _rows(x, N, "x", dy, M)
    w, _, wt = _norm_weights(weight, None, N, dy)
    stats = []
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t.dtype != torch.float32 or t.device != dy.device or t.numel() != M or not t.is_contiguous():
            raise ValueError(f"{name} must be {M} contiguous float32 values on dy's GPU")
        stats.append(_ptr(t))
    with _on(dy.device, stream, (dy, x, weight, mean, rstd, dx, dweight, dbias, workspace)) as handle:
        dx, lddx = _out(dx, tuple(x.shape), x, "dx")
        if need_weight:
            dweight = torch.empty(N, dtype=wt, device=dy.device) if dweight is None else dweight
            dbias = torch.empty(N, dtype=wt, device=dy.device) if dbias is None else dbias
        dwp, dbp = _vector(dweight, N, "dweight", dy, wt), _vector(dbias, N, "dbias", dy, wt)
        f, size_of = _function("gemm_layer_norm_backward", _KIND[dy.dtype])
        params = LayerNormParams(M, N, ldx, lddy, lddx, wt == torch.float32, 0.0)
        ws, ws_bytes, held = (None, 0, None)
        if dwp or dbp:
            ws, ws_bytes, held = _workspace(size_of, "gemm_layer_norm_backward", params, workspace, dy.device)
        rc = f(ctypes.byref(params), _ptr(dy2), _ptr(x2), w, *stats, _ptr(dx), dwp, dbp, ws, ws_bytes, handle)
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_layer_norm_backward")
    return dx, dweight, dbias
