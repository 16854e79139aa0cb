"""The layers around the products, for torch tensors on the GPU: the dense
layer with bias, activation and residual, the gated up-projection and layer
norm, each with its backward pass; the first two on 8-bit codes with a scale for
each token and channel, and what makes such codes; and the orthogonalised update
of a weight from its gradient.  Argument checks and marshalling only: the
arithmetic is in the HIP kernels behind the C ABI of ``include/gemm.h``.

Rows may have any stride; weights are ``K x N`` views whose storage is
``K x N`` or ``N x K`` (a transposed view, as ``weight.t()`` of weights kept
outputs by inputs).  Leading dimensions of activations are folded into rows.
Outputs and workspaces are allocated when not given, on the call's stream; the
library itself allocates nothing.  A status other than GEMM_OK raises
``GemmError``, a tensor of the wrong shape, type or layout ``ValueError`` or
``TypeError`` before anything is launched.

The functions are the passes themselves and record nothing for autograd: a
tensor that requires grad is refused (``ValueError``) where torch records
gradients, since theirs would be lost.  Call them under ``torch.no_grad()``, in
the two halves of an autograd function, or on detached tensors.

A call's checks, C parameters and workspace size depend on its arguments'
shapes, strides, types and devices only, so they are made once for each such
form and kept (``_FORMS``, nothing of the tensors themselves): a repeated call
costs its allocations and its launches.
"""
from __future__ import annotations

import contextlib
import ctypes
import warnings

import torch

from . import binding
from .binding import (ACTIVATIONS, GEMM_ERR_INVALID_LAYOUT, GEMM_OK, GEMM_NO_INPUT_GRADIENT, GEMM_NO_WEIGHT_GRADIENT,
                      GEMM_ONLY_BF16, GEMM_ONLY_F16, GEMM_OP_N, GEMM_OP_T, GEMM_MAX_STEPS, GEMM_ROUND_GRADIENT, GatedBackwardParams,
                      GatedI8Params, GatedParams, GemmError, LayerNormParams, LinearBackwardParams, LinearI8Params,
                      LinearParams, OrthogonalizeParams, QuantizeParams)

_KIND = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32"}
_functions = {}
_FORMS = {}
_MAX_FORMS = 4096   # then the kept forms are dropped: a form is made in about 20 us
_MAX_INT = 2 ** 31 - 1
_NEED = ctypes.c_size_t


def _function(stem, kind):
    """(entry point, workspace function or None) of a layer, looked up once."""
    f = _functions.get((stem, kind))
    if f is None:
        lib = binding.load()
        f = (getattr(lib, f"{stem}_{kind}"), getattr(lib, stem + "_workspace", None))
        _functions[stem, kind] = f
    return f


class _Form:
    """What a call of one form needs besides its tensors."""
    __slots__ = ("device", "index", "entry", "stem", "params", "ref", "workspace", "sized", "shape", "dtype", "copies",
                 "extra")

    def __init__(self, like, stem, kind, params, shape=(), dtype=None, copies=(), extra=None):
        self.device, self.index, self.stem = like.device, like.device.index, stem
        self.entry, size_of = _function(stem, kind)
        self.params, self.ref = params, ctypes.byref(params)
        self.shape, self.dtype, self.extra = shape, dtype, extra
        self.copies = copies      # the tensors whose leading dimensions do not fold into rows
        self.workspace, self.sized = 0, size_of is not None
        if size_of is not None:
            need = _NEED()
            rc = size_of(self.ref, ctypes.byref(need))
            if rc != GEMM_OK:
                raise GemmError(rc, stem)
            self.workspace = need.value


def _keep(key, form):
    if len(_FORMS) >= _MAX_FORMS:
        _FORMS.clear()
    _FORMS[key] = form
    return form


def _sig(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _grad_unless_off():
    """Refuses a call on tensors that require grad, where torch would record it."""
    if torch.is_grad_enabled():
        raise ValueError("a tensor requires grad, which these functions do not record: call them under "
                         "torch.no_grad() or on detached tensors, and use the _backward functions")


def _activation(name):
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"unknown activation {name!r}: one of {sorted(ACTIVATIONS)}") from None


def _flagged(act, kind, need_input, need_weight, round_gradient):
    """The activation of a backward pass with what the call will be."""
    return (act | (GEMM_ROUND_GRADIENT if round_gradient else 0) | (GEMM_ONLY_F16 if kind == "f16" else GEMM_ONLY_BF16)
            | (0 if need_input else GEMM_NO_INPUT_GRADIENT) | (0 if need_weight else GEMM_NO_WEIGHT_GRADIENT))


def _kind16(t, name):
    if t.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"{name} must be float16 or bfloat16, not {t.dtype}")
    return _KIND[t.dtype]


def _fold(t):
    """The rows x columns view of a tensor, None where only a copy has one."""
    if t.dim() == 2:
        return t
    try:
        return t.view(_count(t.shape[:-1]), t.shape[-1])
    except RuntimeError:
        return None


def _rows(t, cols, name, like, rows=None, dtype=None):
    """(rows, row stride, whether only a copy has such rows) of an
    activation-like tensor of ``cols`` columns on ``like``'s device."""
    if t.device != like.device or not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU of the first argument")
    if t.dtype != (like.dtype if dtype is None else dtype):
        raise TypeError(f"{name} must be {like.dtype if dtype is None else dtype}, not {t.dtype}")
    if t.dim() == 0:
        raise ValueError(f"{name} needs at least one dimension")
    r, c = _count(t.shape[:-1]), t.shape[-1]
    if c != cols or (rows is not None and r != rows):
        raise ValueError(f"{name} is {r} x {c}, expected {rows if rows is not None else 'any'} x {cols}")
    v = _fold(t)
    if v is None:
        return r, max(cols, 1), True
    s0, s1 = v.stride()
    if s1 != 1 and c > 1:
        raise ValueError(f"{name} must have contiguous rows (strides {t.stride()})")
    ld = s0 if r > 1 else max(cols, 1)
    if ld > _MAX_INT:
        raise ValueError(f"{name}'s row stride {ld} is out of range")
    return r, ld, False


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
        return
    if v.device != like.device:
        raise ValueError(f"{name} must be on the GPU of the first argument")
    if v.dtype != (like.dtype if dtype is None else dtype):
        raise TypeError(f"{name} must be {like.dtype if dtype is None else dtype}, not {v.dtype}")
    if v.dim() != 1 or v.shape[0] != n or (n > 1 and v.stride(0) != 1):
        raise ValueError(f"{name} must be {n} contiguous elements")


def _out(t, shape, like, name, dtype=None):
    """Row stride of an output of ``shape`` (None: one that the call allocates)."""
    if t is None:
        return max(shape[-1], 1)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} is {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dim() != 2 and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _rows(t, shape[-1], name, like, dtype=like.dtype if dtype is None else dtype)[1]


def _grad_stride(w, op, given, name):
    """Row stride of a gradient of weight w (K x N view), in w's kind of storage."""
    k, n = w.shape
    if given is None:
        return max(k if op == GEMM_OP_T else n, 1)
    if given.shape != w.shape or given.dtype != w.dtype or given.device != w.device:
        raise ValueError(f"{name} must match its weight")
    # the weight's storage, also where a single row or column could be either
    unit, stride, inner, outer = (0, 1, k, n) if op == GEMM_OP_T else (1, 0, n, k)
    ld = given.stride(stride) if outer > 1 else max(inner, 1)
    if (inner > 1 and given.stride(unit) != 1) or ld > _MAX_INT:
        raise ValueError(f"{name} must be stored as its weight is")
    return ld


def _grad_like(w, op):
    return w.new_empty((w.shape[1], w.shape[0])).t() if op == GEMM_OP_T else w.new_empty(w.shape)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _in(t, name, form):
    """An input as the kernels take it: the tensor, or a copy (made on the
    call's stream) where its leading dimensions do not fold into rows."""
    return t.reshape(-1, t.shape[-1]) if name in form.copies else t


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


def _run(form, stream, tensors, go):
    """go(handle of the call's stream), with the device and stream current."""
    if stream is None and form.index == torch._C._cuda_getDevice():   # (there are GPU tensors: torch has its GPU)
        return go(torch._C._cuda_getCurrentRawStream(form.index))
    with _on(form.device, stream, tensors) as handle:
        return go(handle)


def _workspace(form, given, like):
    """The tensor of a call's workspace (None where it needs none)."""
    if given is not None:
        if given.dtype != torch.uint8 or given.device != form.device or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the call's GPU")
        return given
    return like.new_empty(form.workspace, dtype=torch.uint8) if form.workspace else None


def _size(ws):
    return 0 if ws is None else ws.numel()


def _done(rc, form):
    if rc != GEMM_OK:
        raise GemmError(rc, form.stem)


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
    save_pre = bool(save_pre) or pre is not None
    if x.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad) or \
            (residual is not None and residual.requires_grad):
        _grad_unless_off()
    key = ("linear", x.shape, x.stride(), x.dtype, x.device, w.shape, w.stride(), w.dtype, w.device, _sig(bias),
           _sig(residual), activation, save_pre, out_dtype, _sig(y), _sig(pre))
    form = _FORMS.get(key) or _keep(key, _linear_form(x, w, bias, residual, activation, save_pre, out_dtype, y, pre))

    def go(handle):
        xs, rs = (_in(x, "x", form), _in(residual, "residual", form)) if form.copies else (x, residual)
        out = x.new_empty(form.shape, dtype=form.dtype) if y is None else y
        saved = x.new_empty(form.shape) if save_pre and pre is None else pre
        ws = _workspace(form, workspace, x)
        _done(form.entry(form.ref, xs.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(rs), out.data_ptr(), _ptr(saved),
                         _ptr(ws), _size(ws), handle), form)
        return (out, saved) if save_pre else out
    return _run(form, stream, (x, w, bias, residual, y, pre, workspace), go)


def _linear_form(x, w, bias, residual, activation, save_pre, out_dtype, y, pre):
    _gpu(x, "x")
    kind = _kind16(x, "x")
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    op, ldw = _weight(w, "w", x)
    K, N = w.shape
    M, ldx, copy_x = _rows(x, K, "x", x)
    act = _activation(activation)
    if out_dtype is None:
        out_dtype = x.dtype if y is None else y.dtype
    if out_dtype not in (x.dtype, torch.float32):
        raise TypeError(f"out_dtype must be {x.dtype} or float32")
    shape = tuple(x.shape[:-1]) + (N,)
    _vector(bias, N, "bias", x)
    ldr, copy_r = 0, False
    if residual is not None:
        if tuple(residual.shape) != shape:
            raise ValueError(f"residual is {tuple(residual.shape)}, expected {shape}")
        _, ldr, copy_r = _rows(residual, N, "residual", x, M, out_dtype)
    ldy = _out(y, shape, x, "y", out_dtype)
    ldp = _out(pre, shape, x, "pre") if save_pre else 0
    params = LinearParams(M, N, K, op, ldx, ldw, ldy, ldr, ldp, act, out_dtype == torch.float32)
    copies = [n for n, c in (("x", copy_x), ("residual", copy_r)) if c]
    return _Form(x, "gemm_linear", kind, params, shape, out_dtype, copies)


def linear_backward(dy, x, w, pre=None, activation="none", need_input=True, need_weight=True, need_bias=True,
                    dx=None, dw=None, dbias=None, workspace=None, stream=None, round_gradient=False):
    """Gradients ``(dx, dw, dbias)`` of ``linear`` from that of its output (in
    x's type) and its saved ``pre`` (not needed without an activation); None
    for those not needed.  The residual's gradient is dy.  dw has w's shape and
    storage.

    The gradient of the pre-activation is held to 2^-17 of its values and with the
    range of FP32, as two terms, which takes two products' work for dx and dw
    each, three in float16.  With ``round_gradient`` it is rounded to x's type and
    takes one: dx and dw are off by about 1.4 times their own rounding, and in
    float16 a gradient past 65504 becomes infinite, one below 2^-25 zero.  (none
    and relu need no rounding.)"""
    if dy.requires_grad or x.requires_grad or w.requires_grad or (pre is not None and pre.requires_grad):
        _grad_unless_off()
    need_input, need_weight, need_bias = (bool(need_input) or dx is not None, bool(need_weight) or dw is not None,
                                          bool(need_bias) or dbias is not None)
    key = ("linear_backward", dy.shape, dy.stride(), dy.dtype, dy.device, x.shape, x.stride(), x.dtype, x.device,
           w.shape, w.stride(), w.dtype, w.device, _sig(pre), activation, need_input, need_weight, need_bias,
           _sig(dx), _sig(dw), _sig(dbias), bool(round_gradient))
    form = _FORMS.get(key) or _keep(key, _linear_backward_form(dy, x, w, pre, activation, need_input, need_weight,
                                                               need_bias, dx, dw, dbias, round_gradient))

    def go(handle):
        dys, xs, pres = dy, x, pre
        if form.copies:
            dys, xs, pres = (_in(t, n, form) for t, n in ((dy, "dy"), (x, "x"), (pre, "pre")))
        gx = x.new_empty(x.shape) if need_input and dx is None else dx
        gw = _grad_like(w, form.extra) if need_weight and dw is None else dw
        gb = dy.new_empty(w.shape[1]) if need_bias and dbias is None else dbias
        ws = _workspace(form, workspace, dy)
        _done(form.entry(form.ref, dys.data_ptr(), xs.data_ptr(), w.data_ptr(), _ptr(pres), _ptr(gx), _ptr(gw),
                         _ptr(gb), _ptr(ws), _size(ws), handle), form)
        return gx, gw, gb
    return _run(form, stream, (dy, x, w, pre, dx, dw, dbias, workspace), go)


def _linear_backward_form(dy, x, w, pre, activation, need_input, need_weight, need_bias, dx, dw, dbias,
                          round_gradient):
    _gpu(dy, "dy")
    kind = _kind16(dy, "dy")
    op, ldw = _weight(w, "w", dy)
    K, N = w.shape
    act = _activation(activation)
    M, lddy, copy_dy = _rows(dy, N, "dy", dy)
    _, ldx, copy_x = _rows(x, K, "x", dy, M)
    ldp, copy_p = 0, False
    if act:
        if pre is None:
            raise ValueError("the backward pass of an activation needs pre")
        _, ldp, copy_p = _rows(pre, N, "pre", dy, M)
    lddx = _out(dx, tuple(x.shape), x, "dx") if need_input else 0
    lddw = _grad_stride(w, op, dw, "dw") if need_weight else 0
    _vector(dbias, N, "dbias", dy)
    params = LinearBackwardParams(M, N, K, op, lddy, ldx, ldw, ldp, lddx, lddw,
                                  _flagged(act, kind, need_input, need_weight, round_gradient))
    copies = [n for n, c in (("dy", copy_dy), ("x", copy_x), ("pre", copy_p)) if c]
    return _Form(dy, "gemm_linear_backward", kind, params, copies=copies, extra=op)


# ----------------------------------------------------- gated up-projection --

def gated(x, wg, wu, activation="silu", save_pre=False, h=None, workspace=None, stream=None):
    """``act(x wg) * (x wu)`` for float16 or bfloat16 x (..., K) and the
    K x F weights wg and wu (of one storage and stride: the halves of one
    K x 2F matrix will do), both products in one kernel.  With ``save_pre``
    returns ``(h, g, u)``, the products for ``gated_backward``."""
    save_pre = bool(save_pre)
    if x.requires_grad or wg.requires_grad or wu.requires_grad:
        _grad_unless_off()
    key = ("gated", x.shape, x.stride(), x.dtype, x.device, wg.shape, wg.stride(), wg.dtype, wg.device, wu.shape,
           wu.stride(), wu.dtype, wu.device, activation, save_pre, _sig(h))
    form = _FORMS.get(key) or _keep(key, _gated_form(x, wg, wu, activation, h))

    def go(handle):
        xs = _in(x, "x", form) if form.copies else x
        out = x.new_empty(form.shape) if h is None else h
        g, u = (x.new_empty(form.shape), x.new_empty(form.shape)) if save_pre else (None, None)
        ws = _workspace(form, workspace, x)
        _done(form.entry(form.ref, xs.data_ptr(), wg.data_ptr(), wu.data_ptr(), out.data_ptr(), _ptr(g), _ptr(u),
                         _ptr(ws), _size(ws), handle), form)
        return (out, g, u) if save_pre else out
    return _run(form, stream, (x, wg, wu, h, workspace), go)


def _gated_form(x, wg, wu, activation, h):
    _gpu(x, "x")
    kind = _kind16(x, "x")
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    op, ldw = _gate_weights(wg, wu, x)
    K, F = wg.shape
    M, ldx, copy_x = _rows(x, K, "x", x)
    act = _activation(activation)
    shape = tuple(x.shape[:-1]) + (F,)
    ldh = _out(h, shape, x, "h")
    return _Form(x, "gemm_gated", kind, GatedParams(M, F, K, op, ldx, ldw, ldh, max(F, 1), act), shape,
                 copies=["x"] if copy_x else ())


def _gate_weights(wg, wu, like):
    op, ld = _weight(wg, "wg", like)
    op_u, ld_u = _weight(wu, "wu", like)
    if wu.shape != wg.shape:
        raise ValueError(f"wg is {tuple(wg.shape)}, wu {tuple(wu.shape)}")
    if op != op_u or ld != ld_u:
        raise ValueError("wg and wu must have one storage order and stride")
    return op, ld


def gated_backward(dh, x, wg, wu, g, u, activation="silu", need_input=True, need_weight=True, dx=None, dwg=None,
                   dwu=None, workspace=None, stream=None, round_gradient=False):
    """Gradients ``(dx, dwg, dwu)`` of ``gated`` from that of its output and
    its saved products g and u; None for those not needed.  The gradients of g
    and u are held as ``linear_backward`` holds that of its pre-activation (here
    under every activation), or rounded with ``round_gradient``."""
    if (dwg is None) != (dwu is None):
        raise ValueError("dwg and dwu are given together or not at all")
    if dh.requires_grad or x.requires_grad or wg.requires_grad or wu.requires_grad or g.requires_grad or \
            u.requires_grad:
        _grad_unless_off()
    need_input, need_weight = bool(need_input) or dx is not None, bool(need_weight) or dwg is not None
    key = ("gated_backward", dh.shape, dh.stride(), dh.dtype, dh.device, x.shape, x.stride(), x.dtype, x.device,
           wg.shape, wg.stride(), wg.dtype, wg.device, wu.shape, wu.stride(), wu.dtype, wu.device, _sig(g), _sig(u),
           activation, need_input, need_weight, _sig(dx), _sig(dwg), _sig(dwu), bool(round_gradient))
    form = _FORMS.get(key) or _keep(key, _gated_backward_form(dh, x, wg, wu, g, u, activation, need_input,
                                                              need_weight, dx, dwg, dwu, round_gradient))

    def go(handle):
        dhs, xs, gs, us = dh, x, g, u
        if form.copies:
            dhs, xs, gs, us = (_in(t, n, form) for t, n in ((dh, "dh"), (x, "x"), (g, "g"), (u, "u")))
        gx = x.new_empty(x.shape) if need_input and dx is None else dx
        a, b = (_grad_like(wg, form.extra), _grad_like(wg, form.extra)) if need_weight and dwg is None else (dwg, dwu)
        ws = _workspace(form, workspace, dh)
        _done(form.entry(form.ref, dhs.data_ptr(), xs.data_ptr(), wg.data_ptr(), wu.data_ptr(), gs.data_ptr(),
                         us.data_ptr(), _ptr(gx), _ptr(a), _ptr(b), _ptr(ws), _size(ws), handle), form)
        return gx, a, b
    return _run(form, stream, (dh, x, wg, wu, g, u, dx, dwg, dwu, workspace), go)


def _gated_backward_form(dh, x, wg, wu, g, u, activation, need_input, need_weight, dx, dwg, dwu, round_gradient):
    _gpu(dh, "dh")
    kind = _kind16(dh, "dh")
    op, ldw = _gate_weights(wg, wu, dh)
    K, F = wg.shape
    act = _activation(activation)
    M, lddh, copy_dh = _rows(dh, F, "dh", dh)
    _, ldx, copy_x = _rows(x, K, "x", dh, M)
    _, ldp, copy_g = _rows(g, F, "g", dh, M)
    _, ldu, copy_u = _rows(u, F, "u", dh, M)
    if ldp != ldu:
        raise ValueError("g and u must have one row stride")
    lddx = _out(dx, tuple(x.shape), x, "dx") if need_input else 0
    lddw = 0
    if need_weight:
        lddw = _grad_stride(wg, op, dwg, "dwg")
        if _grad_stride(wu, op, dwu, "dwu") != lddw:
            raise ValueError("dwg and dwu must have one stride")
    params = GatedBackwardParams(M, F, K, op, lddh, ldx, ldw, ldp, lddx, lddw,
                                 _flagged(act, kind, need_input, need_weight, round_gradient))
    copies = [n for n, c in (("dh", copy_dh), ("x", copy_x), ("g", copy_g), ("u", copy_u)) if c]
    return _Form(dh, "gemm_gated_backward", kind, params, copies=copies, extra=op)


# --------------------------------------------------------------- layer norm --

def _norm_weights(weight, bias, N, x):
    """Type of layer norm's weight and bias."""
    dtype = next((t.dtype for t in (weight, bias) if t is not None), torch.float32)
    if dtype not in (x.dtype, torch.float32):
        raise TypeError(f"weight and bias must be {x.dtype} or float32, not {dtype}")
    _vector(weight, N, "weight", x, dtype)
    _vector(bias, N, "bias", x, dtype)
    return dtype


def layer_norm(x, weight=None, bias=None, eps=1e-5, save_stats=False, y=None, stream=None):
    """Layer norm over the last dimension of a float32, float16 or bfloat16
    tensor; weight and bias in x's type or float32.  With ``save_stats``
    returns ``(y, mean, rstd)``, the statistics of each row in float32 for
    ``layer_norm_backward``."""
    if x.requires_grad or (weight is not None and weight.requires_grad) or (bias is not None and bias.requires_grad):
        _grad_unless_off()
    key = ("layer_norm", x.shape, x.stride(), x.dtype, x.device, _sig(weight), _sig(bias), eps, _sig(y))
    form = _FORMS.get(key) or _keep(key, _layer_norm_form(x, weight, bias, eps, y))

    def go(handle):
        xs = _in(x, "x", form) if form.copies else x
        out = x.new_empty(x.shape) if y is None else y
        mean = rstd = None
        if save_stats:
            mean = x.new_empty(form.shape, dtype=torch.float32)
            rstd = x.new_empty(form.shape, dtype=torch.float32)
            if x.shape[-1] == 0:
                mean.zero_(), rstd.zero_()
        _done(form.entry(form.ref, xs.data_ptr(), _ptr(weight), _ptr(bias), out.data_ptr(), _ptr(mean), _ptr(rstd),
                         handle), form)
        return (out, mean, rstd) if save_stats else out
    return _run(form, stream, (x, weight, bias, y), go)


def _layer_norm_form(x, weight, bias, eps, y):
    _gpu(x, "x")
    if x.dtype not in _KIND:
        raise TypeError(f"x must be float32, float16 or bfloat16, not {x.dtype}")
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    N = x.shape[-1]
    M, ldx, copy_x = _rows(x, N, "x", x)
    wt = _norm_weights(weight, bias, N, x)
    ldy = _out(y, tuple(x.shape), x, "y")
    return _Form(x, "gemm_layer_norm", _KIND[x.dtype], LayerNormParams(M, N, ldx, ldy, 0, wt == torch.float32, eps),
                 tuple(x.shape[:-1]), copies=["x"] if copy_x else ())


def layer_norm_backward(dy, x, weight, mean, rstd, need_weight=True, dx=None, dweight=None, dbias=None,
                        workspace=None, stream=None):
    """Gradients ``(dx, dweight, dbias)`` of ``layer_norm`` from that of its
    output and its saved statistics; the last two in weight's type (float32
    without one), None unless ``need_weight``."""
    need_weight = bool(need_weight)
    if dy.requires_grad or x.requires_grad or (weight is not None and weight.requires_grad) or mean.requires_grad or \
            rstd.requires_grad:
        _grad_unless_off()
    key = ("layer_norm_backward", dy.shape, dy.stride(), dy.dtype, dy.device, x.shape, x.stride(), x.dtype, x.device,
           _sig(weight), _sig(mean), _sig(rstd), need_weight, _sig(dx), _sig(dweight), _sig(dbias))
    form = _FORMS.get(key) or _keep(key, _layer_norm_backward_form(dy, x, weight, mean, rstd, need_weight, dx, dweight,
                                                                   dbias))

    def go(handle):
        dys, xs = (_in(dy, "dy", form), _in(x, "x", form)) if form.copies else (dy, x)
        gx = x.new_empty(x.shape) if dx is None else dx
        gw = dy.new_empty(dy.shape[-1], dtype=form.dtype) if need_weight and dweight is None else dweight
        gb = dy.new_empty(dy.shape[-1], dtype=form.dtype) if need_weight and dbias is None else dbias
        ws = _workspace(form, workspace, dy) if gw is not None or gb is not None else None
        _done(form.entry(form.ref, dys.data_ptr(), xs.data_ptr(), _ptr(weight), mean.data_ptr(), rstd.data_ptr(),
                         gx.data_ptr(), _ptr(gw), _ptr(gb), _ptr(ws), _size(ws), handle), form)
        return gx, gw, gb
    return _run(form, stream, (dy, x, weight, mean, rstd, dx, dweight, dbias, workspace), go)


def _layer_norm_backward_form(dy, x, weight, mean, rstd, need_weight, dx, dweight, dbias):
    _gpu(dy, "dy")
    if dy.dtype not in _KIND:
        raise TypeError(f"dy must be float32, float16 or bfloat16, not {dy.dtype}")
    if dy.dim() < 1:
        raise ValueError("dy needs at least one dimension")
    N = dy.shape[-1]
    M, lddy, copy_dy = _rows(dy, N, "dy", dy)
    _, ldx, copy_x = _rows(x, N, "x", dy, M)
    wt = _norm_weights(weight, None, N, dy)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t.dtype != torch.float32 or t.device != dy.device or t.numel() != M or not t.is_contiguous():
            raise ValueError(f"{name} must be {M} contiguous float32 values on dy's GPU")
    lddx = _out(dx, tuple(x.shape), x, "dx")
    _vector(dweight, N, "dweight", dy, wt)
    _vector(dbias, N, "dbias", dy, wt)
    params = LayerNormParams(M, N, ldx, lddy, lddx, wt == torch.float32, 0.0)
    copies = [n for n, c in (("dy", copy_dy), ("x", copy_x)) if c]
    return _Form(dy, "gemm_layer_norm_backward", _KIND[dy.dtype], params, dtype=wt, copies=copies)


# --------------------------------------------- calls of forms seen before --
#
# The kernels of a few rows on 8-bit operands take 3 to 5 us, less than a call's
# checks, allocations and marshalling in Python (7 to 8 us with the launch): the
# extension module does these for a form that a call in Python has made and kept.

_marshal = None   # the module; False where there is none
_QUANTIZE_I8, _LINEAR_I8, _GATED_I8 = range(3)
_TYPES = {None: 0, torch.float32: 1, torch.float16: 2, torch.bfloat16: 3}


def _again(op, stem, tensors, extra):
    """The result of a call whose form is known to the extension module; None
    where it is not, where the call is not one on the current device, and without the
    module."""
    if not tensors[0].is_cuda or -1 in extra:
        return None
    global _marshal
    if _marshal is None:
        try:
            from . import _marshal as module
        except ImportError as e:
            module = False
            warnings.warn(f"calls of quantize_i8, linear_i8 and gated_i8 take about 3 us longer without the extension "
                          f"module _marshal.so ({e}): `python -m dense_gemm_optimisation_row_amd.build` makes it",
                          RuntimeWarning)
        _marshal = module
    if not _marshal:
        return None
    index = torch._C._cuda_getDevice()
    out = _marshal.run(op, tensors, extra, index, torch._C._cuda_getCurrentRawStream(index))
    if type(out) is int:
        raise GemmError(out, stem)
    return out


def _remember(op, tensors, extra, form, slots, outputs):
    """Makes a form known to the extension module.  slots: the entry point's
    pointers, each the index of a tensor or -1 - that of an output; outputs: the
    index of a given tensor, or (shape, dtype)."""
    if _marshal and not form.copies and -1 not in extra and form.index == torch._C._cuda_getDevice():
        _marshal.keep(op, tensors, extra, form.index, ctypes.cast(form.entry, ctypes.c_void_p).value,
                      bytes(form.params), slots, outputs, form.workspace if form.sized else -1)


# ---------------------------------------------------- 8-bit dense layers --

def _kind_of(dtype, name):
    if dtype not in _KIND:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, not {dtype}")
    return _KIND[dtype]


def _scales(t, n, name, like):
    """Scales of n rows or columns: n float32 values one after another."""
    if t.device != like.device:
        raise ValueError(f"{name} must be on the GPU of the first argument")
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, not {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous values, not {tuple(t.shape)}")


def quantize_i8(x, q=None, scale=None, stream=None):
    """``(q, scale)``: the rows of a float32, float16 or bfloat16 x (..., K) as
    int8 codes of x's shape and one float32 scale each, of shape (...): the
    largest |x| of the row times float32(1 / 127), at least 2^-126, and x / scale to the
    nearest whole number, ties to even.  A row that holds a NaN or an infinity gets the
    scale NaN and zeros.  Weights are quantised as outputs by inputs:
    ``q, s = quantize_i8(weight)``, and ``q.t()`` with ``s`` goes into
    ``linear_i8``."""
    tensors = (x, q, scale)
    if stream is None:
        done = _again(_QUANTIZE_I8, "gemm_quantize_i8", tensors, ())
        if done is not None:
            return done
    if x.requires_grad:
        _grad_unless_off()
    key = ("quantize_i8", x.shape, x.stride(), x.dtype, x.device, _sig(q), _sig(scale))
    form = _FORMS.get(key) or _keep(key, _quantize_form(x, q, scale))

    def go(handle):
        xs = _in(x, "x", form) if form.copies else x
        codes = x.new_empty(x.shape, dtype=torch.int8) if q is None else q
        steps = x.new_empty(form.shape, dtype=torch.float32) if scale is None else scale
        _done(form.entry(form.ref, xs.data_ptr(), codes.data_ptr(), steps.data_ptr(), handle), form)
        return codes, steps
    done = _run(form, stream, tensors, go)
    if stream is None:
        _remember(_QUANTIZE_I8, tensors, (), form, (0, -1, -2),
                  ((tuple(x.shape), torch.int8) if q is None else 1,
                   (form.shape, torch.float32) if scale is None else 2))
    return done


def _quantize_form(x, q, scale):
    _gpu(x, "x")
    kind = _kind_of(x.dtype, "x")
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    K = x.shape[-1]
    M, ldx, copy_x = _rows(x, K, "x", x)
    ldq = _out(q, tuple(x.shape), x, "q", torch.int8)
    shape = tuple(x.shape[:-1])
    if scale is not None:
        if tuple(scale.shape) != shape:
            raise ValueError(f"scale is {tuple(scale.shape)}, expected {shape}")
        _scales(scale, M, "scale", x)
    return _Form(x, "gemm_quantize_i8", kind, QuantizeParams(M, K, ldx, ldq), shape, copies=["x"] if copy_x else ())


def _off_units(*tensors):
    return any(t.data_ptr() & 15 for t in tensors)


def _codes(x, name):
    _gpu(x, name)
    if x.dtype != torch.int8:
        raise TypeError(f"{name} must be int8, not {x.dtype}")


def linear_i8(x, x_scale, w, w_scale, bias=None, residual=None, activation="none", out_dtype=None, y=None,
              workspace=None, stream=None):
    """``act(x_scale w_scale (x w) + bias) + residual`` for int8 x (..., K) with
    a float32 scale for each of its rows and int8 w (K x N) with one for each of
    its columns (``quantize_i8``).  The sums are exact (K up to 131071), the rest
    is float32; ``bias`` is float32, the residual and the result ``out_dtype``:
    float32, float16 or bfloat16; by default y's or the residual's type, else
    bfloat16.  w is fastest stored outputs by inputs (a transposed view) with K a multiple of 16:
    other weights are copied into that form in each call.  ``y`` may be the
    residual itself."""
    tensors = (x, x_scale, w, w_scale, bias, residual, y)
    extra = (ACTIVATIONS.get(activation, -1), _TYPES.get(out_dtype, -1))
    if stream is None and workspace is None:
        done = _again(_LINEAR_I8, "gemm_linear_i8", tensors, extra)
        if done is not None:
            return done
    if (bias is not None and bias.requires_grad) or (residual is not None and residual.requires_grad) or \
            x_scale.requires_grad or w_scale.requires_grad:
        _grad_unless_off()
    off = _off_units(x, w)
    key = ("linear_i8", x.shape, x.stride(), x.dtype, x.device, _sig(x_scale), w.shape, w.stride(), w.dtype, w.device,
           _sig(w_scale), _sig(bias), _sig(residual), activation, out_dtype, _sig(y), off)
    form = _FORMS.get(key) or _keep(key, _linear_i8_form(x, x_scale, w, w_scale, bias, residual, activation, out_dtype,
                                                         y, off))

    def go(handle):
        xs, rs = (_in(x, "x", form), _in(residual, "residual", form)) if form.copies else (x, residual)
        out = x.new_empty(form.shape, dtype=form.dtype) if y is None else y
        ws = _workspace(form, workspace, x)
        _done(form.entry(form.ref, xs.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), _ptr(bias),
                         _ptr(rs), out.data_ptr(), _ptr(ws), _size(ws), handle), form)
        return out
    done = _run(form, stream, tensors + (workspace,), go)
    if stream is None and workspace is None:
        _remember(_LINEAR_I8, tensors, extra, form, (0, 1, 2, 3, 4, 5, -1),
                  ((form.shape, form.dtype) if y is None else 6,))
    return done


def _linear_i8_form(x, x_scale, w, w_scale, bias, residual, activation, out_dtype, y, off):
    _codes(x, "x")
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    op, ldw = _weight(w, "w", x)
    K, N = w.shape
    M, ldx, copy_x = _rows(x, K, "x", x)
    _scales(x_scale, M, "x_scale", x)
    _scales(w_scale, N, "w_scale", x)
    act = _activation(activation)
    if out_dtype is None:
        out_dtype = next((t.dtype for t in (y, residual) if t is not None), torch.bfloat16)
    kind = _kind_of(out_dtype, "out_dtype")
    shape = tuple(x.shape[:-1]) + (N,)
    _vector(bias, N, "bias", x, torch.float32)
    ldr, copy_r = 0, False
    if residual is not None:
        if tuple(residual.shape) != shape:
            raise ValueError(f"residual is {tuple(residual.shape)}, expected {shape}")
        _, ldr, copy_r = _rows(residual, N, "residual", x, M, out_dtype)
    ldy = _out(y, shape, x, "y", out_dtype)
    # (a copy of x is on 16 bytes; that it is then copied once more costs little beside it)
    params = LinearI8Params(M, N, K, op, ldx, ldw, ldy, ldr, act, off)
    copies = [n for n, c in (("x", copy_x), ("residual", copy_r)) if c]
    return _Form(x, "gemm_linear_i8", kind, params, shape, out_dtype, copies)


def gated_i8(x, x_scale, wg, wg_scale, wu, wu_scale, activation="silu", out_dtype=None, h=None, workspace=None,
             stream=None):
    """``act(x wg) * (x wu)`` for int8 x (..., K) and K x F weights (of one
    storage and stride), each product scaled as in ``linear_i8``; the result is
    ``out_dtype``: float32, float16 or bfloat16, by default h's type or
    bfloat16."""
    tensors = (x, x_scale, wg, wg_scale, wu, wu_scale, h)
    extra = (ACTIVATIONS.get(activation, -1), _TYPES.get(out_dtype, -1))
    if stream is None and workspace is None:
        done = _again(_GATED_I8, "gemm_gated_i8", tensors, extra)
        if done is not None:
            return done
    if x_scale.requires_grad or wg_scale.requires_grad or wu_scale.requires_grad:
        _grad_unless_off()
    off = _off_units(x, wg, wu)
    key = ("gated_i8", x.shape, x.stride(), x.dtype, x.device, _sig(x_scale), wg.shape, wg.stride(), wg.dtype,
           wg.device, _sig(wg_scale), _sig(wu), _sig(wu_scale), activation, out_dtype, _sig(h), off)
    form = _FORMS.get(key) or _keep(key, _gated_i8_form(x, x_scale, wg, wg_scale, wu, wu_scale, activation, out_dtype,
                                                        h, off))

    def go(handle):
        xs = _in(x, "x", form) if form.copies else x
        out = x.new_empty(form.shape, dtype=form.dtype) if h is None else h
        ws = _workspace(form, workspace, x)
        _done(form.entry(form.ref, xs.data_ptr(), x_scale.data_ptr(), wg.data_ptr(), wg_scale.data_ptr(),
                         wu.data_ptr(), wu_scale.data_ptr(), out.data_ptr(), _ptr(ws), _size(ws), handle), form)
        return out
    done = _run(form, stream, tensors + (workspace,), go)
    if stream is None and workspace is None:
        _remember(_GATED_I8, tensors, extra, form, (0, 1, 2, 3, 4, 5, -1),
                  ((form.shape, form.dtype) if h is None else 6,))
    return done


def _gated_i8_form(x, x_scale, wg, wg_scale, wu, wu_scale, activation, out_dtype, h, off):
    _codes(x, "x")
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    op, ldw = _gate_weights(wg, wu, x)
    K, F = wg.shape
    M, ldx, copy_x = _rows(x, K, "x", x)
    _scales(x_scale, M, "x_scale", x)
    _scales(wg_scale, F, "wg_scale", x)
    _scales(wu_scale, F, "wu_scale", x)
    act = _activation(activation)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if h is None else h.dtype
    kind = _kind_of(out_dtype, "out_dtype")
    shape = tuple(x.shape[:-1]) + (F,)
    ldh = _out(h, shape, x, "h", out_dtype)
    return _Form(x, "gemm_gated_i8", kind, GatedI8Params(M, F, K, op, ldx, ldw, ldh, act, off), shape, out_dtype,
                 copies=["x"] if copy_x else ())


# --------------------------------------------------- orthogonalised update --

def _matrices(t, name):
    """(batch, op, row stride, stride between matrices) of a matrix or a stack
    of them (..., M, N), each stored by rows or by columns."""
    rows, cols = t.shape[-2:]
    batch = _count(t.shape[:-2])
    lead = t.shape[:-2]
    stride = 0
    if batch > 1:
        # the leading dimensions must be one stride apart: last to first
        expect = None
        for n, s in zip(reversed(lead), reversed(t.stride()[:-2])):
            if n == 1:
                continue
            if expect is None:
                stride = s
            elif s != expect:
                raise ValueError(f"{name}'s leading dimensions must be one stride apart (strides {t.stride()})")
            expect = s * n
    s0, s1 = t.stride()[-2:]
    if s1 == 1 or cols <= 1:
        op, ld = GEMM_OP_N, s0 if rows > 1 else max(cols, 1)
    elif s0 == 1 or rows <= 1:
        op, ld = GEMM_OP_T, s1 if cols > 1 else max(rows, 1)
    else:
        raise ValueError(f"{name} needs a unit stride in one dimension (strides {t.stride()})")
    if ld > _MAX_INT:
        raise ValueError(f"{name}'s stride {ld} is out of range")
    if ld < (rows if op == GEMM_OP_T else cols):
        raise ValueError(f"{name}'s rows overlap (strides {t.stride()})")
    return batch, op, ld, stride


def _step_coefficients(coefficients, steps):
    """a, b, c of every step, one after another."""
    if not 1 <= steps <= GEMM_MAX_STEPS:
        raise ValueError(f"steps must be 1 to {GEMM_MAX_STEPS}, not {steps}")
    triples = list(coefficients)
    if triples and not hasattr(triples[0], "__len__"):
        triples = [tuple(triples)] * steps
    if len(triples) != steps or any(len(t) != 3 for t in triples):
        raise ValueError(f"coefficients are a, b, c, or {steps} such triples")
    return tuple(float(v) for t in triples for v in t)


def orthogonalize(g, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, scale=1.0, out=None, workspace=None,
                  stream=None):
    """The orthogonalised update of a gradient g (M x N) or of each of a stack
    (..., M, N), float32, float16 or bfloat16: with X = g / (|g| + eps), |g| the
    root of its sum of squares, ``steps`` Newton-Schulz steps
    X = a X + (b A + c A A) X, A = X X^T, then ``scale`` X, in g's type and
    storage.  ``coefficients`` are a, b, c, or such a triple for each step; they must not let
    a singular value of at most 1, nor what multiplies it, grow past 256, nor hold all
    of them below 2^-35.
    Products are computed from two float16 terms of each operand, to 2^-23 of
    its values.  g may be a transposed view (a weight gradient of
    ``linear_backward``) and a stack's matrices may lie between each other's rows
    (``w.view(d, heads, -1).transpose(0, 1)``); ``out`` likewise, and it may be g itself."""
    if g.requires_grad:
        _grad_unless_off()
    values = _step_coefficients(coefficients, steps)
    # (eps and scale, which a schedule changes from call to call, are not of the form)
    key = ("orthogonalize", g.shape, g.stride(), g.dtype, g.device, steps, values, _sig(out))
    form = _FORMS.get(key) or _keep(key, _orthogonalize_form(g, steps, values, eps, scale, out))

    def go(handle):
        o = out
        if o is None:
            o = g.new_empty(form.shape)
            if form.extra:
                o = o.mT
        ws = _workspace(form, workspace, g)
        params = OrthogonalizeParams.from_buffer_copy(form.params)   # the call's own
        params.eps, params.scale = eps, scale
        rc = form.entry(ctypes.byref(params), g.data_ptr(), o.data_ptr(), _ptr(ws), _size(ws), handle)
        if rc == GEMM_ERR_INVALID_LAYOUT:   # the rest of the layout has been checked
            raise ValueError(f"out's matrices overlap (strides {o.stride()})")
        _done(rc, form)
        return o
    return _run(form, stream, (g, out, workspace), go)


def _orthogonalize_form(g, steps, values, eps, scale, out):
    _gpu(g, "g")
    kind = _kind_of(g.dtype, "g")
    if g.dim() < 2:
        raise ValueError("g must be a matrix or a stack of them")
    M, N = g.shape[-2:]
    batch, op_g, ldg, stride_g = _matrices(g, "g")
    if out is None:
        op_o, ldo, stride_o = op_g, max(M if op_g == GEMM_OP_T else N, 1), M * N
    else:
        if out.shape != g.shape or out.dtype != g.dtype or out.device != g.device:
            raise ValueError("out must match g")
        _, op_o, ldo, stride_o = _matrices(out, "out")
    params = OrthogonalizeParams(batch, M, N, op_g, op_o, ldg, ldo, steps, stride_g, stride_o, eps, scale)
    params.coefficients[:len(values)] = values
    turned = op_g == GEMM_OP_T
    shape = tuple(g.shape[:-2]) + ((N, M) if turned else (M, N))
    return _Form(g, "gemm_orthogonalize", kind, params, shape, extra=turned and out is None)
