"""Operators around the recurrence, the router and the loss of a model trained on
packed batches, over the C ABI of ``include/nstrain.h``.

``embed`` takes a table's rows at the batch's tokens, ``layer_norm`` normalises
every position, ``dispatch`` sorts tokens by the experts that ``route`` chose and
``combine`` brings the experts' rows back.  Padding (document ids below 0, no
expert) has rows of 0 and no part in a gradient.  As in ``operators``: each has a
form that PyTorch differentiates, in reverse mode, and the explicit passes behind it;
the work is queued on the current stream of the inputs' device; all sums run in a
fixed order.
"""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib as L
from .operators import (_DTYPES, _floats, _optional, _reverse_only, _shape, _stream,
                        _wants_grad)
from .packer import _refuse


def _row_step(t: torch.Tensor, name: str) -> int:
    """Elements between the rows of a [..., D] tensor, taken as rows in their order."""
    shape = t.shape
    if t.is_contiguous():
        return shape[-1]
    stride = t.stride()
    if shape[-1] > 1 and stride[-1] != 1:
        _refuse(f"{name}: strides {stride}, the last dimension has to be contiguous")
    step = None  # of the rows, from the last dimension with more than one on
    for size, s in zip(shape[-2::-1], stride[-2::-1]):
        if size == 1:
            continue
        if step is None:
            step, rows = s, size
        elif s != step * rows:
            _refuse(f"{name}: strides {stride}, expected rows at even distances")
        else:
            rows *= size
    return shape[-1] if step is None else step


def _even(t: torch.Tensor) -> torch.Tensor:
    """A gradient as rows at even distances; a copy where it is laid out otherwise."""
    if t.is_contiguous():
        return t
    try:
        return t if _row_step(t, "") >= t.shape[-1] else t.contiguous()
    except L.NsPackError:
        return t.contiguous()


# ---- rows of a table -----------------------------------------------------------------
def _embed_inputs(tokens, V, D, table_code, code, scale, doc) -> bytes:
    dtype = tokens.dtype
    if dtype != torch.int32 and dtype != torch.int64:
        _refuse(f"tokens: dtype {dtype}, expected int32 or int64")
    if not tokens.is_contiguous():
        _refuse("tokens: not contiguous")
    if not math.isfinite(scale):
        _refuse(f"scale: {scale}, expected a finite number")
    if doc is not None:
        doc = _optional(doc, "doc", torch.int32, tokens.shape, tokens.device)
    return L.pack_embed(tokens.data_ptr(), doc or 0, tokens.numel(), V, D, table_code, code,
                        dtype == torch.int64, scale)


# Its number; torch.cuda.current_device takes twice as long.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _code(dtype, name: str) -> int:
    if dtype not in _DTYPES:
        _refuse(f"{name}: {dtype}, expected float32, bfloat16 or float16")
    return _DTYPES[dtype]


def _embed(weight, tokens, scale, doc, dtype):
    code = _floats(weight, "weight")
    shape = weight.shape
    if len(shape) != 2:
        _refuse(f"weight: shape {tuple(shape)}, expected [V, D]")
    device = weight.device
    if not isinstance(tokens, torch.Tensor) or tokens.device != device:
        _refuse("tokens: expected a tensor on the weight's device")
    index = device.index
    if index != _current_device():
        with torch.cuda.device(device):
            return _embed(weight, tokens, scale, doc, dtype)
    V, D = shape
    if dtype is None:
        dtype, out_code = weight.dtype, code
    else:
        out_code = _code(dtype, "dtype")
    inputs = _embed_inputs(tokens, V, D, code, out_code, scale, doc)
    y = torch.empty((*tokens.shape, D), dtype=dtype, device=device)
    L.ns_embed_forward(inputs, weight.data_ptr(), _row_step(weight, "weight"), y.data_ptr(),
                       _stream(index))
    return y


def embed_backward(dy: torch.Tensor, tokens: torch.Tensor, vocab: int, *, scale: float = 1.0,
                   doc: Optional[torch.Tensor] = None,
                   dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Gradient of ``embed``'s table, [vocab, D] of ``dtype`` (dy's if None), from that
    of its rows ([..., D], rows at even distances)."""
    code = _floats(dy, "dy")
    if not isinstance(vocab, int) or vocab < 0 or vocab >= 1 << 31:
        _refuse(f"vocab: {vocab!r}, expected a number of tokens below 2**31")
    device = dy.device
    if not isinstance(tokens, torch.Tensor) or tokens.device != device:
        _refuse("tokens: expected a tensor on dy's device")
    if device.index != _current_device():
        with torch.cuda.device(device):
            return embed_backward(dy, tokens, vocab, scale=scale, doc=doc, dtype=dtype)
    if dy.dim() < 1 or dy.shape[:-1] != tokens.shape:
        _refuse(f"dy: shape {tuple(dy.shape)}, expected {(*tokens.shape, 'D')}")
    D = dy.shape[-1]
    if dtype is None:
        dtype, out_code = dy.dtype, code
    else:
        out_code = _code(dtype, "dtype")
    inputs = _embed_inputs(tokens, vocab, D, out_code, code, scale, doc)
    step = _row_step(dy, "dy")
    dweight = torch.empty((vocab, D), dtype=dtype, device=device)
    work = torch.empty(L.ns_embed_workspace(tokens.numel(), vocab, D), dtype=torch.uint8,
                       device=device)
    L.ns_embed_backward(inputs, dy.data_ptr(), step, dweight.data_ptr(), work.data_ptr(),
                        _stream(device.index))
    return dweight


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, tokens, scale, doc, dtype):
        y = _embed(weight, tokens, scale, doc, dtype)
        ctx.save_for_backward(tokens, doc)
        ctx.table = weight.shape[0], weight.dtype
        ctx.scale = scale
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        _reverse_only(dy)
        tokens, doc = ctx.saved_tensors
        vocab, dtype = ctx.table
        return (embed_backward(_even(dy), tokens, vocab, scale=ctx.scale, doc=doc, dtype=dtype),
                None, None, None, None)


def embed(weight: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0,
          doc: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Rows of a table at tokens, times ``scale``: [*tokens.shape, D].

    ``weight`` [V, D] is float32, bfloat16 or float16 (rows at any distance from D on), ``tokens``
    int32 or int64 of any shape, contiguous, ``doc`` int32 of that shape.  Positions
    whose ``doc`` is below 0, and tokens outside [0, V), have rows of 0 and no part in
    the gradient.  The rows are of ``dtype``, or the weight's.

    PyTorch differentiates it with respect to ``weight``: positions are sorted by token,
    each row of the gradient is summed in 32 bits in a fixed order and rounded once.
    """
    _reverse_only(weight)
    if _wants_grad(weight):
        return _Embed.apply(weight, tokens, scale, doc, dtype)
    return _embed(weight, tokens, scale, doc, dtype)


# ---- layer norm ------------------------------------------------------------------------
def _norm_inputs(x, weight, bias, eps, doc) -> bytes:
    code = _floats(x, "x")
    shape, device = x.shape, x.device
    D = shape[-1] if shape else 0
    if D < 1:
        _refuse(f"x: shape {tuple(shape)}, expected [..., D]")
    given = weight if weight is not None else bias
    weight_code, weight_ptr, bias_ptr, doc_ptr = code, 0, 0, 0
    if given is not None:
        weight_code = _floats(given, "weight" if weight is not None else "bias")
        if weight_code != L.NS_F32 and weight_code != code:
            _refuse(f"weight, bias: dtype {given.dtype}, expected float32 or {x.dtype}")
        if weight is not None:
            weight_ptr = _optional(weight, "weight", given.dtype, (D,), device)
        if bias is not None:
            bias_ptr = _optional(bias, "bias", given.dtype, (D,), device)
    if doc is not None:
        doc_ptr = _optional(doc, "doc", torch.int32, shape[:-1], device)
    if not (eps >= 0.0 and math.isfinite(eps)):
        _refuse(f"eps: {eps}, expected 0 or a positive number")
    return L.pack_norm(x.data_ptr(), _row_step(x, "x"), weight_ptr, bias_ptr, doc_ptr,
                       x.numel() // D, D, code, weight_code, eps)


def _norm(x, weight, bias, eps, doc, keep: bool):
    inputs = _norm_inputs(x, weight, bias, eps, doc)
    device = x.device
    index = device.index
    if index != _current_device():
        with torch.cuda.device(device):
            return _norm(x, weight, bias, eps, doc, keep)
    shape = x.shape
    y = torch.empty(shape, dtype=x.dtype, device=device)
    if not keep:
        L.ns_norm_forward(inputs, y.data_ptr(), None, None, _stream(index))
        return y, None, None
    mean = torch.empty(shape[:-1], dtype=torch.float32, device=device)
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=device)
    L.ns_norm_forward(inputs, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _stream(index))
    return y, mean, rstd


def layer_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
                       doc: Optional[torch.Tensor] = None):
    """``layer_norm`` without autograd: (y, mean, rstd), the last two float32 [...], for
    ``layer_norm_backward``."""
    return _norm(x, weight, bias, eps, doc, True)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor],
                        bias: Optional[torch.Tensor], mean: torch.Tensor, rstd: torch.Tensor, *,
                        doc: Optional[torch.Tensor] = None):
    """Gradients (dx, dweight, dbias) from that of ``y`` ([..., D], rows at even
    distances), with the forward pass's inputs and what it returned; dweight and dbias
    are None where ``weight`` and ``bias`` are."""
    return _norm_backward(dy, x, weight, bias, mean, rstd, doc, weight is not None,
                          bias is not None)


def _norm_backward(dy, x, weight, bias, mean, rstd, doc, to_weight: bool, to_bias: bool):
    inputs = _norm_inputs(x, weight, bias, 0.0, doc)
    shape, device = x.shape, x.device
    if device.index != _current_device():
        with torch.cuda.device(device):
            return _norm_backward(dy, x, weight, bias, mean, rstd, doc, to_weight, to_bias)
    if not isinstance(dy, torch.Tensor) or dy.dtype != x.dtype or dy.device != device:
        _refuse("dy: expected a tensor of x's dtype on x's device")
    _shape(dy, "dy", shape)
    if mean is None or rstd is None:
        _refuse("mean, rstd: expected what layer_norm_forward returned")
    mean_ptr = _optional(mean, "mean", torch.float32, shape[:-1], device)
    rstd_ptr = _optional(rstd, "rstd", torch.float32, shape[:-1], device)
    dx = torch.empty(shape, dtype=x.dtype, device=device)
    dweight = dbias = work = None
    if to_weight:
        dweight = torch.empty(shape[-1], dtype=weight.dtype, device=device)
    if to_bias:
        dbias = torch.empty(shape[-1], dtype=bias.dtype, device=device)
    if dweight is not None or dbias is not None:
        D = shape[-1]
        work = torch.empty(L.ns_norm_workspace(x.numel() // D, D) // 4, dtype=torch.float32,
                           device=device)
    L.ns_norm_backward(inputs, mean_ptr, rstd_ptr, dy.data_ptr(), _row_step(dy, "dy"),
                       dx.data_ptr(), None if dweight is None else dweight.data_ptr(),
                       None if dbias is None else dbias.data_ptr(),
                       None if work is None else work.data_ptr(), _stream(device.index))
    return dx, dweight, dbias


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, doc):
        y, mean, rstd = _norm(x, weight, bias, eps, doc, True)
        ctx.save_for_backward(x, weight, bias, doc, mean, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        _reverse_only(dy)
        x, weight, bias, doc, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dweight, dbias = _norm_backward(_even(dy), x, weight, bias, mean, rstd, doc,
                                            need[1], need[2])
        return dx if need[0] else None, dweight, dbias, None, None


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
               doc: Optional[torch.Tensor] = None) -> torch.Tensor:
    """(x - mean) / sqrt(variance + eps) * weight + bias over the last dimension.

    ``x`` [..., D] is float32, bfloat16 or float16, its rows at even distances from D on; ``weight``
    and ``bias`` [D] are float32 or of x's dtype, 1 and 0 if None; ``doc`` is int32 [...].
    Rows whose ``doc`` is below 0 are not read: they are 0, and have no part in a
    gradient.  Statistics and sums have 32 bits, the variance is that of the values less
    their mean.  PyTorch differentiates it with respect to x, weight and bias.
    """
    _reverse_only(x, weight, bias)
    if _wants_grad(x, weight, bias):
        return _LayerNorm.apply(x, weight, bias, eps, doc)
    return _norm(x, weight, bias, eps, doc, False)[0]


# ---- tokens by expert, and back ------------------------------------------------------------
class ExpertOrder(NamedTuple):
    """Where ``dispatch`` put the choices of experts."""
    place: torch.Tensor    # int32 [N, k], each choice's row; from offsets[E] on: no expert
    slots: torch.Tensor    # int32 [N * k], the choice of each row: token slots // k
    offsets: torch.Tensor  # int32 [E + 1], expert e has the rows offsets[e] to offsets[e + 1]


def _dispatch(x, ids, experts):
    code = _floats(x, "x")
    shape = x.shape
    if len(shape) != 2:
        _refuse(f"x: shape {tuple(shape)}, expected [N, D]")
    if not isinstance(experts, int) or not 1 <= experts <= L.NS_DISPATCH_MAX_EXPERTS:
        _refuse(f"experts: {experts!r}, expected 1 to {L.NS_DISPATCH_MAX_EXPERTS}")
    device = x.device
    index = device.index
    if index != _current_device():
        with torch.cuda.device(device):
            return _dispatch(x, ids, experts)
    N, D = shape
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        _refuse("ids: expected a tensor [N, k]")
    k = ids.shape[1]
    sizes = L.pack_experts(N, k, experts, D, code)
    ids_ptr = _optional(ids, "ids", torch.int32, (N, k), device)
    step = _row_step(x, "x")
    place = torch.empty((N, k), dtype=torch.int32, device=device)
    slots = torch.empty(N * k, dtype=torch.int32, device=device)
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=device)
    rows = torch.empty((N * k, D), dtype=x.dtype, device=device)
    size = L.ns_dispatch_workspace(N, k, experts)
    work = torch.empty(size // 4, dtype=torch.int32, device=device) if size else None
    L.ns_dispatch(sizes, ids_ptr, x.data_ptr(), step, place.data_ptr(), slots.data_ptr(),
                  offsets.data_ptr(), rows.data_ptr(), work.data_ptr() if size else None,
                  _stream(index))
    return rows, ExpertOrder(place, slots, offsets)


def _order(order, rows, name: str):
    """Sizes and addresses of an order whose rows are `rows`."""
    if not isinstance(order, tuple) or len(order) != 3:
        _refuse("order: expected what dispatch returned")
    place, _, offsets = order
    code = _floats(rows, name)
    if not isinstance(place, torch.Tensor) or place.dim() != 2:
        _refuse("order.place: expected [N, k]")
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1:
        _refuse("order.offsets: expected [E + 1]")
    N, k = place.shape
    E = offsets.shape[0] - 1
    shape, device = rows.shape, rows.device
    if len(shape) != 2 or shape[0] != N * k:
        _refuse(f"{name}: shape {tuple(shape)}, expected [{N * k}, D]")
    return (code, N, k, E, _optional(place, "order.place", torch.int32, (N, k), device),
            _optional(offsets, "order.offsets", torch.int32, (E + 1,), device))


def _combine(rows, order, weights):
    code, N, k, E, place, offsets = _order(order, rows, "rows")
    D, device = rows.shape[1], rows.device
    index = device.index
    if index != _current_device():
        with torch.cuda.device(device):
            return _combine(rows, order, weights)
    if weights is not None:
        weights = _optional(weights, "weights", torch.float32, (N, k), device)
    out = torch.empty((N, D), dtype=rows.dtype, device=device)
    L.ns_combine(L.pack_experts(N, k, E, D, code), place, offsets, weights, rows.data_ptr(),
                 _row_step(rows, "rows"), out.data_ptr(), _stream(index))
    return out


def dispatch_backward(d_rows: torch.Tensor, order: ExpertOrder) -> torch.Tensor:
    """Gradient of ``dispatch``'s x [N, D] from that of its rows: for each token the sum
    of its choices' rows."""
    return _combine(d_rows, order, None)


def combine_backward(d_out: torch.Tensor, rows: torch.Tensor, order: ExpertOrder,
                     weights: Optional[torch.Tensor] = None):
    """Gradients (d_rows, d_weights) of ``combine`` from that of its output [N, D], with
    its inputs; d_weights is None where ``weights`` is."""
    return _combine_backward(d_out, rows, order, weights, weights is not None)


def _combine_backward(d_out, rows, order, weights, to_weights: bool):
    code, N, k, E, place, offsets = _order(order, rows, "rows")
    D, device = rows.shape[1], rows.device
    if device.index != _current_device():
        with torch.cuda.device(device):
            return _combine_backward(d_out, rows, order, weights, to_weights)
    if not isinstance(d_out, torch.Tensor) or d_out.dtype != rows.dtype or d_out.device != device:
        _refuse("d_out: expected a tensor of the rows' dtype on their device")
    _shape(d_out, "d_out", (N, D))
    sizes = L.pack_experts(N, k, E, D, code)
    weights_ptr = _optional(weights, "weights", torch.float32, (N, k), device)
    d_rows = torch.empty((N * k, D), dtype=rows.dtype, device=device)
    d_weights = None
    if to_weights:
        d_weights = torch.empty((N, k), dtype=torch.float32, device=device)
    L.ns_combine_backward(sizes, place, offsets, weights_ptr, rows.data_ptr(),
                          _row_step(rows, "rows"), d_out.data_ptr(), _row_step(d_out, "d_out"),
                          d_rows.data_ptr(), None if d_weights is None else d_weights.data_ptr(),
                          _stream(device.index))
    return d_rows, d_weights


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, ids, experts):
        rows, order = _dispatch(x, ids, experts)
        ctx.save_for_backward(*order)
        ctx.mark_non_differentiable(*order)
        ctx.set_materialize_grads(False)
        return rows, *order

    @staticmethod
    @once_differentiable
    def backward(ctx, d_rows, *_):
        _reverse_only(d_rows)
        if d_rows is None:
            return None, None, None
        return dispatch_backward(_even(d_rows), ExpertOrder(*ctx.saved_tensors)), None, None


def dispatch(x: torch.Tensor, ids: torch.Tensor, experts: int):
    """Tokens sorted by expert: (rows [N * k, D], order).

    ``ids`` (int32 [N, k], as ``route`` returns them; outside [0, experts): none) are the
    experts of each row of ``x`` ([N, D], float32, bfloat16 or float16, rows at any
    distance from D on).  Expert e's rows are ``rows[order.offsets[e]:order.offsets[e + 1]]``, in
    the tokens' order; ``rows[order.place[n, j]]`` is ``x[n]``.  Rows from
    ``order.offsets[experts]`` on, as many as choices without an expert, are 0.

    PyTorch differentiates ``rows`` with respect to ``x``.
    """
    _reverse_only(x)
    if _wants_grad(x):
        rows, *order = _Dispatch.apply(x, ids, experts)
        return rows, ExpertOrder(*order)
    return _dispatch(x, ids, experts)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, place, slots, offsets):
        out = _combine(rows, (place, slots, offsets), weights)
        ctx.save_for_backward(rows, weights, place, slots, offsets)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        _reverse_only(d_out)
        rows, weights, *order = ctx.saved_tensors
        need = ctx.needs_input_grad
        d_rows, d_weights = _combine_backward(_even(d_out), rows, ExpertOrder(*order), weights,
                                             need[1])
        return d_rows if need[0] else None, d_weights, None, None, None


def combine(rows: torch.Tensor, order: ExpertOrder,
            weights: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The experts' rows brought back to their tokens: [N, D], the sum over a token's
    choices of ``weights`` (float32 [N, k], 1 if None) times ``rows[order.place]``.

    ``rows`` [N * k, D] are in the order that ``dispatch`` returned; those from
    ``order.offsets[-1]`` on are not read.  Sums have 32 bits and are rounded once.
    PyTorch differentiates it with respect to ``rows`` and ``weights``.
    """
    _reverse_only(rows, weights)
    if _wants_grad(rows, weights) and isinstance(order, tuple) and len(order) == 3:
        return _Combine.apply(rows, weights, *order)
    return _combine(rows, order, weights)
