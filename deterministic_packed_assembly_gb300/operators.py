"""Operators of a model trained on packed batches, over the C ABI of
``include/nstrain.h``.

``gated_scan`` mixes a row's positions over time, ``route`` chooses experts and
``distill_loss`` compares the model's logits with a teacher's.  They take the
packed batch's position ids (0 starts a document), document ids (below 0 is
padding) and loss mask as ``Packer.step`` writes them.  Each has a form that
PyTorch differentiates, in reverse mode, and the explicit passes behind it.  The work is queued on
the current stream of the inputs' device; outputs and workspaces come from
PyTorch's caching allocator there.  All sums run in a fixed order: the same
inputs give the same bits.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib as L
from .packer import _need, _refuse

_DTYPES = {torch.float32: L.NS_F32, torch.bfloat16: L.NS_BF16, torch.float16: L.NS_F16}


def _floats(t, name: str) -> int:
    """The library's code of a CUDA tensor's floating type."""
    if not isinstance(t, torch.Tensor):
        _refuse(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.dtype not in _DTYPES:
        _refuse(f"{name}: dtype {t.dtype}, expected float32, bfloat16 or float16")
    if not t.is_cuda:
        _refuse(f"{name}: on {t.device}, expected a CUDA device")
    return _DTYPES[t.dtype]


def _shape(t: torch.Tensor, name: str, shape: tuple) -> None:
    if tuple(t.shape) != tuple(shape):
        _refuse(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _optional(t, name: str, dtype: torch.dtype, shape: tuple, device) -> Optional[int]:
    """The address of an optional contiguous tensor."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device
            and t.shape == shape and t.is_contiguous()):
        _need(t, name, dtype, device)  # says which of them it is
        _shape(t, name, shape)
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str) -> None:
    """Refuse a tensor whose last dimension is not contiguous."""
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        _refuse(f"{name}: strides {t.stride()}, the last dimension has to be contiguous")


def _elsewhere(t) -> bool:
    """Whether a CUDA tensor is on another device than the current one."""
    return t.device.index != torch.cuda.current_device()


# The current stream's handle; building a torch.cuda.Stream for it takes 3 us.
_stream = torch._C._cuda_getCurrentRawStream


def _wants_grad(*tensors) -> bool:
    if torch.is_grad_enabled():
        for t in tensors:
            if isinstance(t, torch.Tensor) and t.requires_grad:
                return True
    return False


def _reverse_only(*tensors) -> None:
    """Forward-mode derivatives are not there: an error, where outputs without a tangent
    would be a derivative of 0."""
    if forward_ad._current_level < 0:  # no dual level: 1 us a call saved
        return
    for t in tensors:
        if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError("the operators have no forward-mode derivative")


# ---- gated linear recurrence ---------------------------------------------------
def _scan_inputs(z, f, bias, pos, doc) -> L.ns_scan_inputs:
    code = _floats(z, "z")
    shape = z.shape
    if len(shape) != 3:
        _refuse(f"z: shape {tuple(shape)}, expected [B, T, D]")
    device = z.device
    if not isinstance(f, torch.Tensor) or f.dtype != z.dtype or f.device != device:
        _refuse("f: expected a tensor of z's dtype on z's device")
    if f.shape != shape:
        _shape(f, "f", shape)
    B, T, D = shape
    zs, fs = z.stride(), f.stride()
    if (zs[2] != 1 or fs[2] != 1) and D > 1:
        _rows(z, "z")
        _rows(f, "f")
    return L.ns_scan_inputs(
        z.data_ptr(), f.data_ptr(), zs[0], zs[1], fs[0], fs[1],
        _optional(bias, "bias", torch.float32, (D,), device),
        _optional(pos, "pos", torch.int32, (B, T), device),
        _optional(doc, "doc", torch.int32, (B, T), device), B, T, D, code)


def _scan(z, f, bias, pos, doc, h0, keep: bool):
    inputs = _scan_inputs(z, f, bias, pos, doc)
    if _elsewhere(z):
        with torch.cuda.device(z.device):
            return _scan(z, f, bias, pos, doc, h0, keep)
    B, T, D = shape = z.shape
    device = z.device
    h0_ptr = _optional(h0, "h0", torch.float32, (B, D), device)
    y = torch.empty(shape, dtype=z.dtype, device=device)
    h_last = torch.empty((B, D), dtype=torch.float32, device=device)
    states = None
    if keep:
        states = torch.empty((B, -(-T // L.NS_SCAN_TILE), D), dtype=torch.float32, device=device)
    L.ns_scan_forward(inputs, h0_ptr, y.data_ptr(), h_last.data_ptr(),
                      states.data_ptr() if keep else None, _stream(device.index))
    return y, h_last, states


def gated_scan_forward(z: torch.Tensor, f: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                       pos: Optional[torch.Tensor] = None, doc: Optional[torch.Tensor] = None,
                       h0: Optional[torch.Tensor] = None):
    """``gated_scan`` without autograd: (y, h_last, states), where ``states``
    (the state before every NS_SCAN_TILE steps) is for ``gated_scan_backward``."""
    return _scan(z, f, bias, pos, doc, h0, True)


def gated_scan_backward(dy: torch.Tensor, dh_last: Optional[torch.Tensor], z: torch.Tensor,
                        f: torch.Tensor, bias: Optional[torch.Tensor], states: torch.Tensor, *,
                        pos: Optional[torch.Tensor] = None, doc: Optional[torch.Tensor] = None):
    """Gradients (dz, df, dbias, dh0) from those of ``y`` and of ``h_last`` (or
    None), with the forward pass's inputs and ``states``; dbias is None where
    ``bias`` is."""
    inputs = _scan_inputs(z, f, bias, pos, doc)
    if _elsewhere(z):
        with torch.cuda.device(z.device):
            return gated_scan_backward(dy, dh_last, z, f, bias, states, pos=pos, doc=doc)
    B, T, D = shape = z.shape
    device = z.device
    if not isinstance(dy, torch.Tensor) or dy.dtype != z.dtype or dy.device != device:
        _refuse("dy: expected a tensor of z's dtype on z's device")
    _shape(dy, "dy", shape)
    _rows(dy, "dy")
    dh_ptr = _optional(dh_last, "dh_last", torch.float32, (B, D), device)
    if states is None:
        _refuse("states: expected what gated_scan_forward returned")
    states_ptr = _optional(states, "states", torch.float32, (B, -(-T // L.NS_SCAN_TILE), D), device)
    dz = torch.empty(shape, dtype=z.dtype, device=device)
    df = torch.empty(shape, dtype=z.dtype, device=device)
    dh0 = torch.empty((B, D), dtype=torch.float32, device=device)
    dbias = work = None
    if bias is not None:
        dbias = torch.empty(D, dtype=torch.float32, device=device)
        work = torch.empty(L.ns_scan_workspace(B, T, D) // 4, dtype=torch.float32, device=device)
    dys = dy.stride()
    L.ns_scan_backward(inputs, states_ptr, dy.data_ptr(), dys[0], dys[1], dh_ptr, dz.data_ptr(),
                       df.data_ptr(), None if dbias is None else dbias.data_ptr(), dh0.data_ptr(),
                       None if work is None else work.data_ptr(), _stream(device.index))
    return dz, df, dbias, dh0


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, f, bias, h0, pos, doc):
        y, h_last, states = _scan(z, f, bias, pos, doc, h0, True)
        ctx.save_for_backward(z, f, bias, pos, doc, states)
        ctx.set_materialize_grads(False)
        return y, h_last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh_last):
        _reverse_only(dy, dh_last)
        z, f, bias, pos, doc, states = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros(z.shape, dtype=z.dtype, device=z.device)
        elif dy.shape[-1] > 1 and dy.stride(-1) != 1:
            dy = dy.contiguous()
        if dh_last is not None:
            dh_last = dh_last.contiguous()
        need = ctx.needs_input_grad
        dz, df, dbias, dh0 = gated_scan_backward(dy, dh_last, z, f, bias, states, pos=pos, doc=doc)
        return (dz if need[0] else None, df if need[1] else None, dbias if need[2] else None,
                dh0 if need[3] else None, None, None)


def gated_scan(z: torch.Tensor, f: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
               pos: Optional[torch.Tensor] = None, doc: Optional[torch.Tensor] = None,
               h0: Optional[torch.Tensor] = None):
    """A gated linear recurrence over packed rows: (y, h_last).

    With a_t = sigmoid(f_t + bias), h_t = a_t h_{t-1} + (1 - a_t) z_t per row and
    channel, and y_t = h_t.  Where ``pos`` is 0 the state before is taken as 0;
    at padding (``doc`` below 0) the state stays and y is 0.  The state before
    the first step is ``h0``, or 0; ``h_last`` is the one after the last step,
    to go on from (one token at a time: T = 1).

    ``z`` and ``f`` are [B, T, D] of one dtype (float32, bfloat16, float16), any
    strides over rows and time (such as the halves of one projection); ``bias``
    [D], ``h0`` and ``h_last`` [B, D] are float32, ``pos`` and ``doc`` [B, T]
    int32.  PyTorch differentiates it with respect to z, f, bias and h0.
    """
    _reverse_only(z, f, bias, h0)
    if _wants_grad(z, f, bias, h0):
        return _GatedScan.apply(z, f, bias, h0, pos, doc)
    return _scan(z, f, bias, pos, doc, h0, False)[:2]


# ---- distillation from a teacher's top logits ------------------------------------
def _distill(logits, top_logits, top_ids, mask, temperature, teacher_lse, weight, out, grad: bool):
    code = _floats(logits, "logits")
    if logits.dim() != 2:
        _refuse(f"logits: shape {tuple(logits.shape)}, expected [N, V]")
    if _elsewhere(logits):
        with torch.cuda.device(logits.device):
            return _distill(logits, top_logits, top_ids, mask, temperature, teacher_lse, weight,
                            out, grad)
    N, V = logits.shape
    row, column = logits.stride()
    if column != 1:
        _rows(logits, "logits")
    device = logits.device
    top_code = _floats(top_logits, "top_logits")
    shape = top_logits.shape
    if len(shape) != 2 or shape[0] != N:
        _refuse(f"top_logits: shape {tuple(shape)}, expected [{N}, K]")
    ids_64 = isinstance(top_ids, torch.Tensor) and top_ids.dtype == torch.int64
    if top_ids is None:
        _refuse("top_ids: expected a tensor")
    if isinstance(mask, torch.Tensor) and mask.dtype == torch.bool:
        mask = mask.view(torch.uint8)
    inputs = L.ns_distill_inputs(
        logits.data_ptr(), row if N > 1 else max(row, V),
        _optional(top_logits, "top_logits", top_logits.dtype, shape, device),
        _optional(top_ids, "top_ids", torch.int64 if ids_64 else torch.int32, shape, device),
        _optional(teacher_lse, "teacher_lse", torch.float32, (N,), device),
        _optional(mask, "mask", torch.uint8, (N,), device),
        _optional(weight, "weight", torch.float32, (N,), device),
        N, V, shape[1], code, top_code, ids_64, float(temperature))
    loss = torch.empty(N, dtype=torch.float32, device=device)
    if not grad:
        L.ns_distill(inputs, loss.data_ptr(), None, 0, _stream(device.index))
        return loss, None
    if out is None:
        out = torch.empty((N, V), dtype=logits.dtype, device=device)
    elif not isinstance(out, torch.Tensor) or out.dtype != logits.dtype or out.device != device:
        _refuse("out: expected a tensor of the logits' dtype on their device")
    _shape(out, "out", (N, V))
    _rows(out, "out")
    out_row = out.stride(0)
    L.ns_distill(inputs, loss.data_ptr(), out.data_ptr(), out_row if N > 1 else max(out_row, V),
                 _stream(device.index))
    return loss, out


def distill_grad(logits: torch.Tensor, top_logits: torch.Tensor, top_ids: torch.Tensor, *,
                 mask: Optional[torch.Tensor] = None, temperature: float = 1.0,
                 teacher_lse: Optional[torch.Tensor] = None,
                 weight: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """``distill_loss`` and its gradient in one pass over the logits: (loss [N],
    dlogits [N, V]).  ``weight`` (float32 [N], 1 if None) is the gradient of what
    is minimised with respect to each row's loss, such as 1 / learned positions;
    ``out`` receives dlogits and may be ``logits`` itself."""
    return _distill(logits, top_logits, top_ids, mask, temperature, teacher_lse, weight, out, True)


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_logits, top_ids, mask, temperature, teacher_lse):
        loss, _ = _distill(logits, top_logits, top_ids, mask, temperature, teacher_lse, None, None,
                           False)
        ctx.save_for_backward(logits, top_logits, top_ids, mask, teacher_lse)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, d_loss):
        _reverse_only(d_loss)
        logits, top_logits, top_ids, mask, teacher_lse = ctx.saved_tensors
        _, dlogits = _distill(logits, top_logits, top_ids, mask, ctx.temperature, teacher_lse,
                              d_loss.contiguous(), None, True)
        return dlogits, None, None, None, None, None


def distill_loss(logits: torch.Tensor, top_logits: torch.Tensor, top_ids: torch.Tensor, *,
                 mask: Optional[torch.Tensor] = None, temperature: float = 1.0,
                 teacher_lse: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Divergence of every row from a teacher's top logits (float32 [N]).

    With p the softmax of ``top_logits / temperature`` over the row's K entries
    (or, given ``teacher_lse`` [N], exp(top_logits / temperature - teacher_lse):
    the teacher's own probabilities) and q the softmax of ``logits / temperature``
    over V, loss = temperature**2 * sum_k p_k (log p_k - log q_{top_ids_k}).  Rows
    whose ``mask`` (uint8 or bool [N]) is 0 are not read and have loss 0; entries
    whose id is outside [0, V) are absent.  (Where a row's loss is that of the next
    token, its mask is the next position's, 0 where that starts a document.)

    ``logits`` [N, V] and ``top_logits`` [N, K] are float32, bfloat16 or float16,
    ``top_ids`` int32 or int64.  PyTorch differentiates it with respect to
    ``logits`` (reading them a second time; ``distill_grad`` needs only one pass).
    """
    _reverse_only(logits, top_logits, teacher_lse)
    if _wants_grad(logits):
        return _DistillLoss.apply(logits, top_logits, top_ids, mask, temperature, teacher_lse)
    return _distill(logits, top_logits, top_ids, mask, temperature, teacher_lse, None, None,
                    False)[0]


# ---- router --------------------------------------------------------------------------
class Routing(NamedTuple):
    """What ``route`` returns."""
    ids: torch.Tensor      # int32 [N, k], -1: none
    weights: torch.Tensor  # float32 [N, k]
    counts: torch.Tensor   # int32 [E], tokens that chose each expert
    tokens: torch.Tensor   # int32 [], tokens that count
    loss: torch.Tensor     # float32 [], the balance loss


def _route_inputs(logits, k, doc, normalize) -> L.ns_route_inputs:
    code = _floats(logits, "logits")
    if logits.dim() != 2:
        _refuse(f"logits: shape {tuple(logits.shape)}, expected [N, E]")
    N, E = logits.shape
    row, column = logits.stride()
    if column != 1:
        _rows(logits, "logits")
    return L.ns_route_inputs(
        logits.data_ptr(), row if N > 1 else max(row, E),
        _optional(doc, "doc", torch.int32, (N,), logits.device), N, E, int(k), code,
        1 if normalize else 0)


def _route(logits, k, doc, normalize) -> Routing:
    if not isinstance(k, int) or k < 1:
        _refuse(f"k: {k!r}, expected a positive integer")
    inputs = _route_inputs(logits, k, doc, normalize)
    if _elsewhere(logits):
        with torch.cuda.device(logits.device):
            return _route(logits, k, doc, normalize)
    N, E = logits.shape
    device = logits.device
    ids = torch.empty((N, k), dtype=torch.int32, device=device)
    weights = torch.empty((N, k), dtype=torch.float32, device=device)
    counts = torch.empty(E, dtype=torch.int32, device=device)
    tokens = torch.empty((), dtype=torch.int32, device=device)
    loss = torch.empty((), dtype=torch.float32, device=device)
    size = L.ns_route_workspace(N, E)
    work = torch.empty(size // 4, dtype=torch.int32, device=device) if size else None
    L.ns_route_forward(inputs, ids.data_ptr(), weights.data_ptr(), counts.data_ptr(),
                       tokens.data_ptr(), loss.data_ptr(), work.data_ptr() if size else None,
                       _stream(device.index))
    return Routing(ids, weights, counts, tokens, loss)


def route_backward(logits: torch.Tensor, routing: Routing, d_weights: Optional[torch.Tensor] = None,
                   d_loss: Optional[torch.Tensor] = None, *,
                   doc: Optional[torch.Tensor] = None, normalize: bool = True) -> torch.Tensor:
    """Gradient of the logits [N, E] from those of the weights ([N, k]) and of
    the balance loss (a tensor of one element), either or both, with what
    ``route`` was given and returned."""
    if not isinstance(routing, tuple) or len(routing) != 5:
        _refuse("routing: expected what route returned")
    ids, weights, counts, tokens, _ = routing
    dev = logits.device if isinstance(logits, torch.Tensor) else None
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        _refuse("routing.ids: expected [N, k]")
    inputs = _route_inputs(logits, ids.shape[1], doc, normalize)
    if _elsewhere(logits):
        with torch.cuda.device(dev):
            return route_backward(logits, routing, d_weights, d_loss, doc=doc, normalize=normalize)
    N, E = logits.shape
    shape = ids.shape
    pointers = [_optional(ids, "routing.ids", torch.int32, (N, shape[1]), dev),
                _optional(weights, "routing.weights", torch.float32, shape, dev),
                _optional(counts, "routing.counts", torch.int32, (E,), dev),
                _optional(tokens, "routing.tokens", torch.int32, (), dev),
                _optional(d_weights, "d_weights", torch.float32, shape, dev)]
    if d_loss is not None:
        _need(d_loss, "d_loss", torch.float32, dev)
        if d_loss.numel() != 1:
            _refuse(f"d_loss: shape {tuple(d_loss.shape)}, expected one element")
    dlogits = torch.empty((N, E), dtype=logits.dtype, device=dev)
    L.ns_route_backward(inputs, *pointers, None if d_loss is None else d_loss.data_ptr(),
                        dlogits.data_ptr(), _stream(dev.index))
    return dlogits


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, doc, normalize):
        r = _route(logits, k, doc, normalize)
        ctx.save_for_backward(logits, doc, *r)
        ctx.normalize = normalize
        ctx.mark_non_differentiable(r.ids, r.counts, r.tokens)
        ctx.set_materialize_grads(False)
        return tuple(r)

    @staticmethod
    @once_differentiable
    def backward(ctx, _ids, d_weights, _counts, _tokens, d_loss):
        _reverse_only(d_weights, d_loss)
        logits, doc, *r = ctx.saved_tensors
        if d_weights is not None:
            d_weights = d_weights.contiguous()
        return (route_backward(logits, Routing(*r), d_weights, d_loss, doc=doc,
                               normalize=ctx.normalize), None, None, None)


def route(logits: torch.Tensor, k: int, *, doc: Optional[torch.Tensor] = None,
          normalize: bool = True) -> Routing:
    """Choose ``k`` experts a token and measure how evenly they are used.

    With p the softmax of ``logits`` [N, E] (float32, bfloat16 or float16), a
    token's experts are its k largest logits (of equal ones the lowest index
    first); an expert whose logit is -inf is never chosen (id -1, weight 0).
    The weights are p there, with ``normalize`` divided by their sum.  Tokens
    with ``doc`` (int32 [N]) below 0, and tokens whose logits are all -inf,
    choose none and count for nothing.  ``counts`` has each expert's tokens and
    ``loss`` is the balance loss E / (k M**2) * sum_e counts_e sum_n p_ne over the
    M tokens that count, 1 when the experts are used evenly.

    PyTorch differentiates ``weights`` and ``loss`` with respect to ``logits``.
    """
    _reverse_only(logits)
    if _wants_grad(logits):
        return Routing(*_Route.apply(logits, k, doc, normalize))
    return _route(logits, k, doc, normalize)
