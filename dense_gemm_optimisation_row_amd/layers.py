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

import torch

from . import binding
from .binding import (ACTIVATIONS, GEMM_OK, GEMM_NO_INPUT_GRADIENT, GEMM_NO_WEIGHT_GRADIENT, GEMM_ONLY_BF16,
                      GEMM_ONLY_F16, GEMM_OP_N, GEMM_OP_T, GEMM_ROUND_GRADIENT, GatedBackwardParams, GatedParams,
                      GemmError, LayerNormParams, LinearBackwardParams, LinearParams)

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
    __slots__ = ("device", "index", "entry", "stem", "params", "ref", "workspace", "shape", "dtype", "copies", "extra")

    def __init__(self, like, stem, kind, params, shape=(), dtype=None, copies=(), extra=None):
        self.device, self.index, self.stem = like.device, like.device.index, stem
        self.entry, size_of = _function(stem, kind)
        self.params, self.ref = params, ctypes.byref(params)
        self.shape, self.dtype, self.extra = shape, dtype, extra
        self.copies = copies      # the tensors whose leading dimensions do not fold into rows
        self.workspace = 0
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
