"""The gated feed-forward block of the encoder and its gradient.

Binding of ``ersj_gated`` and ``ersj_gated_grad`` (``include/ersj_encoder.h``),
in the manner of ``encoder``: types, rows, ``out`` and ``stream`` are as there.
``gated`` takes part in autograd.
"""
import torch

from .encoder import (_TYPES, PackedRows, _apply, _as_rows, _check, _elsewhere, _given, _library, _on, _packed,
                      _raw_stream, _rows, _run_elsewhere, _type, _written, pack_rows)

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}  # ERSJ_SILU, ERSJ_GELU, ERSJ_GELU_TANH


def _activation(activation):
    code = ACTIVATIONS.get(activation)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}")
    return code


def _weights(w_gate, w_up, dim, row_type, device):
    """(hidden, spacing of w_gate, of w_up)."""
    spaced = []
    for what, w in (("w_gate", w_gate), ("w_up", w_up)):
        if _type(w, what) != row_type:
            raise TypeError(f"{what} must have the type of x")
        if w.dim() != 2 or w.shape != w_gate.shape:
            raise ValueError("w_gate and w_up must have one shape, [hidden, dim]")
        _on(device, w, what)
        spaced.append(_rows(w, what, dim)[1])
    if not w_gate.shape[0]:
        raise ValueError("w_gate and w_up must have rows")
    return w_gate.shape[0], spaced[0], spaced[1]


def gated(x, w_gate, w_up, activation="silu", pack=False, out=None, stream=None):
    """``ersj_gated``: ``act(x @ w_gate.T) * (x @ w_up.T)``, of shape
    ``x.shape[:-1] + [hidden]``.

    ``w_gate``, ``w_up``: [hidden, dim], of x's type.  ``activation``: "silu",
    "gelu" (with the normal distribution itself) or "gelu_tanh".  Differentiable
    with respect to x and both weights (``gated_grad``); the backward pass keeps
    x alone, with ``pack`` in 8 bits (``PackedRows``).  In float32 an infinity
    among the inputs counts as NaN."""
    if (x.requires_grad or w_gate.requires_grad or w_up.requires_grad) and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out cannot be given where a gradient is wanted")
        return _apply(x.device, stream, (x, w_gate, w_up), lambda: _Gated.apply(x, w_gate, w_up, activation, pack))
    return _gated(x, w_gate, w_up, activation, out, stream)


def _gated(x, w_gate, w_up, activation, out, stream):
    xt = _type(x, "x")
    device = x.device
    if _elsewhere(device, stream):
        return _run_elsewhere(device, stream, (x, w_gate, w_up, out),
                              lambda: _gated(x, w_gate, w_up, activation, out, None))
    act = _activation(activation)
    n, ldx = _rows(x, "x")
    dim = x.shape[-1]
    hidden, ldg, ldu = _weights(w_gate, w_up, dim, xt, device)
    shape = x.shape[:-1] + (hidden,)
    given = out is not None
    if given:
        ldo = _given(out, "out", shape, x.dtype, device)
    else:
        out, ldo = torch.empty(shape, dtype=x.dtype, device=device), hidden
    L = _library()
    args = (x.data_ptr(), xt, n, dim, ldx, w_gate.data_ptr(), ldg, w_up.data_ptr(), ldu, hidden)
    need = L.ersj_gated_work(*args)
    work = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _check(L.ersj_gated(*args, act, out.data_ptr(), ldo, work.data_ptr() if need else None, need,
                        _raw_stream(device.index)))
    if given:
        _written(out)
    return out


def gated_grad(grad, x, w_gate, w_up, activation="silu", want_x=True, want_gate=True, want_up=True, stream=None):
    """``ersj_gated_grad``: (grad of x, of w_gate, of w_up) from ``grad``, the
    gradient of ``gated``'s result.  ``x``: the rows, or ``PackedRows`` of them.
    What is not wanted comes back as None.  The gradients of both projections are
    rounded to the 16-bit type that they are multiplied in (in small products held
    to twice its bits, in float32 to all): 16-bit results of large products are off
    by 1.4 times what their own rounding makes."""
    packed = type(x) is PackedRows
    xt = _TYPES[x.dtype] if packed else _type(x, "x")
    if _type(grad, "grad") != xt:
        raise TypeError("grad must have the type of x")
    device = x.device
    if _elsewhere(device, stream):
        kept = (x.codes, x.scales) if packed else (x,)
        return _run_elsewhere(device, stream, (grad, *kept, w_gate, w_up),
                              lambda: gated_grad(grad, x, w_gate, w_up, activation, want_x, want_gate, want_up))
    act = _activation(activation)
    shape = x.shape
    n, ldx = _rows(x.codes if packed else x, "x")
    dim = shape[-1]
    hidden, ldg, ldu = _weights(w_gate, w_up, dim, xt, device)
    if grad.shape != shape[:-1] + (hidden,):
        raise ValueError(f"grad has the shape {list(grad.shape)}, {list(shape[:-1] + (hidden,))} is expected")
    _on(device, grad, "grad")
    gx, gg, gu = (torch.empty(s, dtype=x.dtype, device=device) if want else None
                  for s, want in ((shape, want_x), (w_gate.shape, want_gate), (w_up.shape, want_up)))
    L = _library()
    weights = (w_gate.data_ptr(), ldg, w_up.data_ptr(), ldu, hidden)
    rows = None if packed else x.data_ptr()
    need = L.ersj_gated_grad_work(rows, xt, n, dim, ldx, *weights, 1 if want_x else 0, 1 if want_gate else 0,
                                  1 if want_up else 0)
    work = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _check(L.ersj_gated_grad(grad.data_ptr(), _rows(grad, "grad")[1], rows, ldx, x.codes.data_ptr() if packed else None,
                             x.scales.data_ptr() if packed else None, xt, n, dim, *weights, act,
                             gx.data_ptr() if want_x else None, dim, gg.data_ptr() if want_gate else None, dim,
                             gu.data_ptr() if want_up else None, dim, work.data_ptr() if need else None, need,
                             _raw_stream(device.index)))
    return gx, gg, gu


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, activation, pack):
        h = _gated(x, w_gate, w_up, activation, None, None)
        ctx.activation, ctx.packed = activation, x.dtype if pack else None
        if pack:
            kept = pack_rows(x)
            ctx.save_for_backward(kept.codes, kept.scales, w_gate, w_up)
        else:
            ctx.save_for_backward(x, w_gate, w_up)
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        *kept, w_gate, w_up = ctx.saved_tensors
        x = kept[0] if ctx.packed is None else _packed(*kept, ctx.packed)
        return *gated_grad(_as_rows(grad), x, w_gate, w_up, ctx.activation, *ctx.needs_input_grad[:3]), None, None
