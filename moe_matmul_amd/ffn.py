"""The feed-forward block in 16 bits beside the NVFP4 layer, and its training, on PyTorch tensors.

Norm with the residual, products with an epilogue, the gated projections, their gradients, and rows kept in 8
bits: dense (a shared expert), or with a ``moe.plan`` by the rows of every expert. Each function checks its
tensors, allocates the outputs that are not given and enqueues operators of ``include/nvfp4_ffn.h`` (which states
the mathematics, the limits and what happens at the edges) on ``stream``, by default torch's current stream.
Streams, memory, graphs and strides are as in ``moe_matmul_amd.moe``: nothing is synchronised or read from the
device, rows may lie apart but not overlap, and their elements are adjacent.

A block with its gradients, ``p`` a plan for the experts or None for a shared one::

    norm = rmsnorm(x, weight, residual=stream, rows8=True)
    h, kept = gated(norm.y, w1, plan=p, save="rows8")
    y = linear(h, w2, plan=p)                      # rows sorted by expert: moe.combine(y, weights, p)
    ...
    dh, dw2, _ = linear_backward(dy, h, w2, plan=p)
    dnorm, dw1 = gated_backward(dh, norm.y8, w1, kept, plan=p)
    dx, dweight = rmsnorm_backward(dnorm, norm.sum, weight, norm.rstd, dsum=dstream)

Gradients have their parameter's type unless an fp32 tensor is given for them.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _ffn_binding as c
from . import moe
from .moe import _at, _current_device, _enqueue, _gpu, _like, _on_stream, _out, _rows, _type

_ACTIVATIONS = {None: c.NVFP4_FFN_NONE, "relu": c.NVFP4_FFN_RELU, "silu": c.NVFP4_FFN_SILU, "gelu": c.NVFP4_FFN_GELU}
_16 = (torch.float16, torch.bfloat16)


def _activation(name, gated=False) -> int:
    if name not in _ACTIVATIONS or (gated and name is None):
        known = ", ".join(repr(n) for n in _ACTIVATIONS if n is not None or not gated)
        raise ValueError(f"activation must be one of {known}, not {name!r}")
    return _ACTIVATIONS[name]


def _type16(t, what) -> int:
    if t.dtype not in _16:
        raise ValueError(f"{what} must be fp16 or bf16, not {t.dtype}")
    return _type(t, what)


def _same(t, what, shape, like) -> int:
    """Row stride of a 2-d tensor of that shape, of the type and on the device of ``like``."""
    if t.shape != shape or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{what} must be a {like.dtype} tensor of shape {tuple(shape)} on {like.device}, not {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return _rows(t, what)


def _param(t, what, shape, like) -> int:
    """Whether a parameter is fp32 (else of the type of ``like``); contiguous, on its device."""
    f32 = t.dtype == torch.float32
    _like(t, what, shape, torch.float32 if f32 else like.dtype, like.device)
    return int(f32)


def _weights(w, plan, device, dtype):
    """(experts or 0, n, k) of checked weights."""
    if w.dim() != (2 if plan is None else 3):
        raise ValueError(f"w must have shape {'[n, k]' if plan is None else '[experts, n, k]'}, not {tuple(w.shape)}")
    _like(w, "w", w.shape, dtype, device)
    if plan is not None and (w.shape[0] != plan.experts or plan.device != device):
        raise ValueError(f"w must have the plan's {plan.experts} experts, on its device")
    return (0 if plan is None else plan.experts, *w.shape[-2:])


def _plan(plan):
    """The plan's argument, or None."""
    if plan is None:
        return None
    entry = getattr(plan, "_ffn_entry", None)
    if entry is None:
        entry = plan._ffn_entry = c.nvfp4_ffn_plan(plan.experts, plan.topk, plan.addresses[0], plan.addresses[3])
    return ctypes.byref(entry)


def _need(size, device, *args) -> int:
    """Bytes of a workspace on that device."""
    if device.index == _current_device():
        return size(*args, device.index)
    with torch.cuda.device(device):
        return size(*args, device.index)


def _room(need, device):
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


# ---- rows in 8 bits ---------------------------------------------------------------

class Rows8(NamedTuple):
    """Rows in 8 bits: ``codes`` uint8 [rows, n] (E4M3) and ``scales`` uint8 [rows, n / 32], one for 32 elements: the
    least power of two 2^(byte - 127) under which the largest is at most 448."""
    codes: torch.Tensor
    scales: torch.Tensor

    @property
    def shape(self):
        return self.codes.shape

    @property
    def device(self):
        return self.codes.device


def _rows8(t, what, shape, device) -> Rows8:
    if len(shape) != 2 or shape[1] % 32:
        raise ValueError(f"{what} must have shape [rows, n], n a multiple of 32, not {tuple(shape)}")
    _like(t.codes, what + ".codes", shape, torch.uint8, device)
    _like(t.scales, what + ".scales", (shape[0], shape[1] // 32), torch.uint8, device)
    return t


def _out8(t, what, shape, device) -> Rows8:
    if t is not None:
        return _rows8(t, what, shape, device)
    if shape[1] % 32:
        raise ValueError(f"rows in 8 bits must have a multiple of 32 elements, not {shape[1]}")
    return Rows8(_out(None, what, shape, torch.uint8, device), _out(None, what, (shape[0], shape[1] // 32), torch.uint8, device))


@_on_stream
def quantize8(x, *, out=None, stream=None) -> Rows8:
    """``x`` [rows, n] (fp32, fp16 or bf16) in 8 bits, each code rounded once, to nearest, ties to even. A block of 32
    that holds an infinity or NaN becomes NaN."""
    device = _gpu(x, "x")
    stride = _rows(x, "x")
    out = _out8(out, "out", x.shape, device)
    _enqueue(c.nvfp4_ffn_quantize8, device, x.data_ptr(), _type(x, "x"), x.shape[0], x.shape[1], stride,
             out.codes.data_ptr(), out.scales.data_ptr())
    return out


@_on_stream
def dequantize8(x, *, dtype=torch.bfloat16, out=None, stream=None):
    """The values that ``x`` (a Rows8) stands for, rounded to ``dtype`` (that of ``out`` where it is given)."""
    device = _gpu(x.codes, "x")
    _rows8(x, "x", x.shape, device)
    if out is None:
        out = _out(None, "out", x.shape, dtype, device)
    elif out.shape != x.shape or out.device != device:
        raise ValueError(f"out must have shape {tuple(x.shape)}, on {device}")
    _enqueue(c.nvfp4_ffn_dequantize8, device, x.codes.data_ptr(), x.scales.data_ptr(), *x.shape, out.data_ptr(),
             _type(out, "out"), _rows(out, "out"))
    return out


# ---- the norm ------------------------------------------------------------------------

class Norm(NamedTuple):
    """What ``rmsnorm`` gives: the normed rows in x's type and in 8 bits (None where not asked for), the sum that was
    normed (x itself without a residual), and 1 / its root mean square, fp32 [rows], for the gradient."""
    y: Optional[torch.Tensor]
    y8: Optional[Rows8]
    sum: torch.Tensor
    rstd: torch.Tensor


@_on_stream
def rmsnorm(x, weight=None, *, residual=None, eps=1e-6, rows=True, rows8=False, stream=None) -> Norm:
    """``s = x + residual`` (rounded to x's type), ``y = s / sqrt(mean(s^2) + eps) * weight`` of rows x [rows, n] (fp32,
    fp16 or bf16). ``weight`` [n]: fp32 or x's type, None for 1. ``rows``: y in x's type; ``rows8``: in 8 bits."""
    device = _gpu(x, "x")
    kind, stride, shape = _type(x, "x"), _rows(x, "x"), x.shape
    if not rows and not rows8:
        raise ValueError("rows or rows8 must be asked for")
    f32 = 0 if weight is None else _param(weight, "weight", shape[1:], x)
    total, residual_stride = x, 0
    if residual is not None:
        residual_stride = _same(residual, "residual", shape, x)
        total = _out(None, "sum", shape, x.dtype, device)
    y = _out(None, "y", shape, x.dtype, device) if rows else None
    y8 = _out8(None, "y8", shape, device) if rows8 else None
    rstd = torch.empty_strided(shape[:1], (1,), dtype=torch.float32, device=device)
    _enqueue(c.nvfp4_ffn_rmsnorm, device, x.data_ptr(), kind, *shape, stride, _at(residual), residual_stride,
             _at(weight), f32, eps, 0 if residual is None else total.data_ptr(), _at(y), _at(y8 and y8.codes),
             _at(y8 and y8.scales), rstd.data_ptr())
    return Norm(y, y8, total, rstd)


@_on_stream
def rmsnorm_backward(dy, sum, weight, rstd, *, dsum=None, stream=None):
    """(dx, dweight) of ``rmsnorm`` from its ``sum`` and ``rstd``: dx [rows, n] is the gradient of x and of the residual,
    ``dsum`` (what reaches the sum otherwise) added; dweight has the weight's type, None without a weight."""
    device = _gpu(sum, "sum")
    kind, stride = _type(sum, "sum"), _rows(sum, "sum")
    rows, n = sum.shape
    dy_stride = _same(dy, "dy", sum.shape, sum)
    dsum_stride = 0 if dsum is None else _same(dsum, "dsum", sum.shape, sum)
    f32 = 0 if weight is None else _param(weight, "weight", (n,), sum)
    _like(rstd, "rstd", (rows,), torch.float32, device)
    dx = _out(None, "dx", sum.shape, sum.dtype, device)
    dweight, need = None, 0
    if weight is not None:
        dweight = torch.empty(n, dtype=weight.dtype, device=device)
        need = _need(c.nvfp4_ffn_rmsnorm_workspace_bytes, device, rows, n)
    room = _room(need, device)
    _enqueue(c.nvfp4_ffn_rmsnorm_backward, device, dy.data_ptr(), dy_stride, sum.data_ptr(), stride, kind, rows, n,
             _at(weight), f32, rstd.data_ptr(), _at(dsum), dsum_stride, dx.data_ptr(), _at(dweight), _at(room), need)
    return dx, dweight


# ---- products --------------------------------------------------------------------------

def _kept(shape, like, cleared):
    """What is kept beside an output: where that is given, and keeps its rows of no expert, cleared."""
    make = torch.zeros if cleared else torch.empty
    return make(shape, dtype=like.dtype, device=like.device)


@_on_stream
def linear(x, w, *, bias=None, activation=None, residual=None, plan=None, save=False, out=None, stream=None):
    """``y = act(x w^T + bias) + residual`` in one product; with ``save`` (y, z), z the activation's argument as
    ``linear_backward`` needs it, rounded to x's type.

    ``x`` [rows, k] (fp16 or bf16), ``w`` [n, k], ``bias`` [n] (fp32 or x's type), ``residual`` [rows, n];
    ``activation``: None, "relu", "silu" or "gelu". With a ``plan``: rows sorted by expert, ``w`` [experts, n, k],
    ``bias`` [experts, n]; rows of no expert are 0 (in an ``out`` that is given they stay as they were)."""
    device = _gpu(x, "x")
    kind, act = _type16(x, "x"), _activation(activation)
    experts, n, k = _weights(w, plan, device, x.dtype)
    stride = _rows(x, "x", k)
    rows = x.shape[0]
    if plan is not None and rows != plan.rows:
        raise ValueError(f"x must have the plan's {plan.rows} rows, not {rows}")
    f32 = 0 if bias is None else _param(bias, "bias", w.shape[:-1], x)
    residual_stride = 0 if residual is None else _same(residual, "residual", (rows, n), x)
    clear = out is None
    out = _out(out, "out", (rows, n), x.dtype, device)
    z = _kept((rows, n), x, plan is not None and not clear) if save else None
    need = _need(c.nvfp4_ffn_product_workspace_bytes, device, rows, n, k, experts)
    room = _room(need, device)
    _enqueue(c.nvfp4_ffn_linear, device, x.data_ptr(), stride, w.data_ptr(), _at(bias), f32, act, _at(residual),
             residual_stride, _at(z), out.data_ptr(), kind, rows, n, k, _plan(plan), clear, _at(room), need)
    return (out, z) if save else out


def _dw(dw, w, dtype):
    """(dw, whether it is fp32): allocated like w where it is not given."""
    if dw is None:
        return torch.empty_like(w), 0
    return dw, _param(dw, "dw", w.shape, w)


def _products_back(dz, dz_stride, x, x_stride, w, plan, kind, experts, dw, dx_f32=False):
    """(dz w, dz^T x) over rows [rows, n] and [rows, k], sorted by expert with a plan; dz w in fp32 or dz's type."""
    device, (rows, n), k = dz.device, dz.shape, w.shape[-1]
    dw, f32 = _dw(dw, w, dz.dtype)
    dx = _out(None, "dx", (rows, k), torch.float32 if dx_f32 else dz.dtype, device)
    need = _need(c.nvfp4_ffn_product_workspace_bytes, device, rows, k, n, experts)
    need_dw = _need(c.nvfp4_ffn_dw_workspace_bytes, device, rows, n, k, experts)
    room = _room(max(need, need_dw), device)
    _enqueue(c.nvfp4_ffn_linear_dx_ex, device, dz.data_ptr(), dz_stride, w.data_ptr(), dx.data_ptr(), dx_f32, kind, rows, n, k,
             _plan(plan), 1, _at(room), need)
    _enqueue(c.nvfp4_ffn_linear_dw, device, dz.data_ptr(), dz_stride, x.data_ptr(), x_stride, dw.data_ptr(), f32, kind, rows,
             n, k, _plan(plan), _at(room), need_dw)
    return dx, dw


@_on_stream
def linear_backward(dy, x, w, *, bias=None, z=None, activation=None, plan=None, dw=None, stream=None):
    """(dx, dw, dbias) of ``linear``; the residual's gradient is dy.

    ``z`` as ``linear(..., save=True)`` gave it, with an activation; ``bias`` as it was given there (dbias has its
    type; None without one); ``dw``: a tensor to take w's gradient, of w's type or fp32. The slope is that of the kept
    z; dz = dy act'(z) is rounded to 16 bits for the products, not for dbias. With a ``plan``: rows sorted by expert;
    rows of no expert have dx 0, experts without rows gradients of 0. ``x`` may be a Rows8."""
    device = _gpu(dy, "dy")
    kind, act = _type16(dy, "dy"), _activation(activation)
    experts, n, k = _weights(w, plan, device, dy.dtype)
    stride = _rows(dy, "dy", n)
    rows = dy.shape[0]
    if plan is not None and rows != plan.rows:
        raise ValueError(f"dy must have the plan's {plan.rows} rows, not {rows}")
    if isinstance(x, Rows8):
        _rows8(x, "x", (rows, k), device)
        x = dequantize8(x, dtype=dy.dtype)
    x_stride = _same(x, "x", (rows, k), dy)
    dz, dz_stride = dy, stride
    if act != c.NVFP4_FFN_NONE:
        if z is None:
            raise ValueError("the gradient of an activation needs z: linear(..., save=True)")
        _like(z, "z", (rows, n), dy.dtype, device)
        dz, dz_stride = _out(None, "dz", (rows, n), dy.dtype, device), n
    dbias, f32, need = None, 0, 0
    if bias is not None:
        f32 = _param(bias, "bias", w.shape[:-1], dy)
        dbias = torch.empty(w.shape[:-1], dtype=bias.dtype, device=device)
        need = _need(c.nvfp4_ffn_dz_workspace_bytes, device, rows, n, experts)
    if dz is not dy or dbias is not None:
        room = _room(need, device)
        _enqueue(c.nvfp4_ffn_linear_dz, device, dy.data_ptr(), stride, _at(z) if act else 0, act,
                 0 if dz is dy else dz.data_ptr(), _at(dbias), f32, kind, rows, n, _plan(plan), _at(room), need)
    dx, dw = _products_back(dz, dz_stride, x, x_stride, w, plan, kind, experts, dw)
    return dx, dw, dbias


# ---- the gated projections -----------------------------------------------------------------

@_on_stream
def gated(x, w, *, activation="silu", plan=None, save=None, out=None, stream=None):
    """``h = act(x wg^T) * (x wu^T)``, both projections, the activation and the product in one kernel.

    ``x`` [tokens, k] (fp16 or bf16), ``w`` [2 * inner, k]: the gate's rows, then the other's; h [tokens, inner]. With a
    ``plan``: ``w`` [experts, 2 * inner, k], and h [tokens * topk, inner] has the rows of every slot sorted by expert,
    each from its token's row; rows of no expert are 0 (in an ``out`` that is given they stay as they were).
    ``save``: "rows" or "rows8" gives (h, kept), both projections [rows, 2 * inner] in 16 bits or as a Rows8, for
    ``gated_backward``."""
    device = _gpu(x, "x")
    kind, act = _type16(x, "x"), _activation(activation, gated=True)
    experts, n, k = _weights(w, plan, device, x.dtype)
    stride = _rows(x, "x", k)
    if n % 2:
        raise ValueError(f"w must have as many rows for the gate as for the other projection, not {n} in all")
    if plan is not None and x.shape[0] != plan.tokens:
        raise ValueError(f"x must have the plan's {plan.tokens} tokens, not {x.shape[0]}")
    if save not in (None, "rows", "rows8"):
        raise ValueError(f"save must be None, 'rows' or 'rows8', not {save!r}")
    rows = x.shape[0] if plan is None else plan.rows
    clear = out is None
    h = _out(out, "out", (rows, n // 2), x.dtype, device)
    kept = _kept((rows, n), x, plan is not None and not clear) if save == "rows" else None
    if save == "rows8" and n % 64:
        raise ValueError(f"projections in 8 bits must have a multiple of 32 columns each, not {n // 2}")
    kept8 = _out8(None, "kept", (rows, n), device) if save == "rows8" else None
    if kept8 is not None and plan is not None and not clear:
        kept8.codes.zero_()
        kept8.scales.zero_()
    need = _need(c.nvfp4_ffn_product_workspace_bytes, device, rows, n, k, experts)
    room = _room(need, device)
    _enqueue(c.nvfp4_ffn_gated, device, x.data_ptr(), stride, w.data_ptr(), act, h.data_ptr(), _at(kept),
             _at(kept8 and kept8.codes), _at(kept8 and kept8.scales), kind, rows, n // 2, k, _plan(plan), clear, _at(room), need)
    return h if save is None else (h, kept if kept8 is None else kept8)


@_on_stream
def gated_backward(dh, x, w, kept=None, *, activation="silu", plan=None, dw=None, stream=None):
    """(dx, dw) of ``gated``: dx [tokens, k] (with a plan the sum over each token's slots), dw like w.

    ``x``: the rows as they were given, or a Rows8 of them (of the norm, or by ``quantize8``); ``kept``: what
    ``gated(..., save=)`` gave, or None: both projections are computed again from x, and not rounded. ``dw``: a tensor to take w's
    gradient, of w's type or fp32. The projections' gradients are rounded to 16 bits for the products."""
    device = _gpu(dh, "dh")
    kind, act = _type16(dh, "dh"), _activation(activation, gated=True)
    experts, n, k = _weights(w, plan, device, dh.dtype)
    if n % 2:
        raise ValueError(f"w must have as many rows for the gate as for the other projection, not {n} in all")
    inner = n // 2
    stride = _rows(dh, "dh", inner)
    rows = dh.shape[0]
    if plan is not None and rows != plan.rows:
        raise ValueError(f"dh must have the plan's {plan.rows} rows, not {rows}")
    tokens = rows if plan is None else plan.tokens
    if isinstance(x, Rows8):
        _rows8(x, "x", (tokens, k), device)
    else:
        x_stride = _same(x, "x", (tokens, k), dh)
    if isinstance(kept, Rows8):
        _rows8(kept, "kept", (rows, n), device)
    elif kept is not None:
        _like(kept, "kept", (rows, n), dh.dtype, device)
    # x as rows of 16 bits, with a plan those of every slot
    if plan is not None:
        xs = torch.empty((rows, k), dtype=dh.dtype, device=device)
        eight = isinstance(x, Rows8)
        _enqueue(c.nvfp4_ffn_gather, device, 0 if eight else x.data_ptr(), 0 if eight else x_stride,
                 x.codes.data_ptr() if eight else 0, x.scales.data_ptr() if eight else 0, kind, tokens, k, _plan(plan),
                 xs.data_ptr())
    elif isinstance(x, Rows8):
        xs = dequantize8(x, dtype=dh.dtype)
    if plan is not None or isinstance(x, Rows8):
        rows_x, rows_stride = xs, k
    else:
        rows_x, rows_stride = x, x_stride
    dz = torch.empty((rows, n), dtype=dh.dtype, device=device)
    if kept is None:
        if plan is not None and isinstance(x, Rows8):
            x = dequantize8(x, dtype=dh.dtype)
        again, again_stride = (rows_x, rows_stride) if plan is None else (x, _rows(x, "x"))
        need = _need(c.nvfp4_ffn_product_workspace_bytes, device, rows, n, k, experts)
        room = _room(need, device)
        _enqueue(c.nvfp4_ffn_gated_again, device, dh.data_ptr(), stride, again.data_ptr(), again_stride, w.data_ptr(), act,
                 dz.data_ptr(), kind, rows, inner, k, _plan(plan), _at(room), need)
    else:
        eight = isinstance(kept, Rows8)
        _enqueue(c.nvfp4_ffn_gated_dz, device, dh.data_ptr(), stride, 0 if eight else kept.data_ptr(),
                 kept.codes.data_ptr() if eight else 0, kept.scales.data_ptr() if eight else 0, act, dz.data_ptr(), kind,
                 rows, inner, _plan(plan))
    # a token's dx is one sum over its slots: their parts of it stay in fp32
    dx, dw = _products_back(dz, n, rows_x, rows_stride, w, plan, kind, experts, dw, plan is not None and plan.topk > 1)
    return (dx if plan is None else moe.combine(dx, None, plan, dtype=dh.dtype)), dw
