"""Operators of the encoder whose vectors the join compares: token embedding,
layer norm, their gradients, rows held in 8 bits for a backward pass, and
clipping by the global gradient norm (``feedforward`` has the gated block).

Binding of ``include/ersj_encoder.h``.  The functions carry the C names
without the ``ersj_`` prefix, check and marshal their arguments, and take
output and working memory from torch; all arithmetic runs in the library's
HIP kernels.  ``embed`` and ``layer_norm`` take part in autograd.

Tensors are float32, float16 or bfloat16 on the GPU.  A tensor of rows may
have any leading shape as long as its rows are contiguous and equally spaced.
``stream`` (a torch stream or a raw handle; None: the current one) is where
the work is enqueued; outputs belong to that stream, and a backward pass through
them runs on it.  A tensor given as ``out`` must not require a gradient (unless
gradients are off) nor overlap an input, unless the function says so; what is
written counts for autograd as written in place.
"""
import ctypes

import torch
from torch.autograd import forward_ad

_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}  # ERSJ_F32, ERSJ_F16, ERSJ_BF16
_ID_TYPES = {torch.int32: 0, torch.int64: 1}                      # ERSJ_I32, ERSJ_I64
GRADS_WORK = 16384                                                # ERSJ_GRADS_WORK

ENCODER_SYMBOLS = ("ersj_embed", "ersj_embed_grad", "ersj_embed_grad_work", "ersj_layer_norm",
                   "ersj_layer_norm_grad", "ersj_layer_norm_grad_work", "ersj_grads_create", "ersj_grads_clip",
                   "ersj_grads_free", "ersj_clip_tensors", "ersj_clip_tensors_work", "ersj_pack_rows",
                   "ersj_unpack_rows", "ersj_layer_norm_pack", "ersj_layer_norm_grad_packed",
                   "ersj_layer_norm_grad_packed_work", "ersj_gated", "ersj_gated_work", "ersj_gated_grad",
                   "ersj_gated_grad_work")
PACK_BLOCK = 32                                                   # ERSJ_PACK_BLOCK


def declare(L):
    """Argument types of the entry points on the loaded library."""
    global _lib
    vp, i32, i64, u64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float
    L.ersj_embed.argtypes = [vp, i32, i64, i32, i64, vp, i32, i64, f32, i64, vp, i32, i64, vp]
    L.ersj_embed_grad.argtypes = [vp, i32, i64, vp, i32, i64, f32, i64, vp, i32, i64, i32, i64, i32, vp, u64, vp]
    L.ersj_embed_grad_work.argtypes = [i64, i64, i32]
    L.ersj_embed_grad_work.restype = u64
    L.ersj_layer_norm.argtypes = [vp, i32, i64, i32, i64, vp, vp, i32, f32, vp, i64, vp, vp, vp]
    L.ersj_layer_norm_grad.argtypes = [vp, i64, vp, i64, i32, i64, i32, vp, vp, vp, i32, vp, i64, vp, vp, vp, u64, vp]
    L.ersj_layer_norm_grad_work.argtypes = [i64, i32]
    L.ersj_layer_norm_grad_work.restype = u64
    L.ersj_grads_create.argtypes = [i32, vp, vp, vp, vp, vp, ctypes.POINTER(vp)]
    L.ersj_grads_clip.argtypes = [vp, f32, vp, vp, u64, vp]
    L.ersj_clip_tensors.argtypes = [i32, vp, vp, vp, vp, f32, vp, vp, u64, vp]
    L.ersj_clip_tensors_work.argtypes = [i32, vp, vp]
    L.ersj_clip_tensors_work.restype = u64
    L.ersj_pack_rows.argtypes = [vp, i32, i64, i32, i64, vp, vp, vp]
    L.ersj_unpack_rows.argtypes = [vp, vp, i64, i32, vp, i32, i64, vp]
    L.ersj_layer_norm_pack.argtypes = [vp, i32, i64, i32, i64, vp, vp, i32, f32, vp, i64, vp, vp, vp, vp, vp]
    L.ersj_layer_norm_grad_packed.argtypes = [vp, i64, vp, vp, i32, i64, i32, vp, vp, vp, i32, vp, i64, vp, vp, vp,
                                              u64, vp]
    L.ersj_layer_norm_grad_packed_work.argtypes = [i32, i64, i32]
    L.ersj_layer_norm_grad_packed_work.restype = u64
    weights = [vp, i64, vp, i64, i32]
    L.ersj_gated.argtypes = [vp, i32, i64, i32, i64, *weights, i32, vp, i64, vp, u64, vp]
    L.ersj_gated_work.argtypes = [vp, i32, i64, i32, i64, *weights]
    L.ersj_gated_work.restype = u64
    L.ersj_gated_grad.argtypes = [vp, i64, vp, i64, vp, vp, i32, i64, i32, *weights, i32, vp, i64, vp, i64, vp, i64,
                                  vp, u64, vp]
    L.ersj_gated_grad_work.argtypes = [vp, i32, i64, i32, i64, *weights, i32, i32, i32]
    L.ersj_gated_grad_work.restype = u64
    L.ersj_grads_free.argtypes = [vp]
    L.ersj_grads_free.restype = None
    _lib = L


_lib = None  # the loaded library, set by declare
# the current stream's handle without a Stream object, where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)

_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _library():
    if _lib is None:
        from . import lib
        lib()
    return _lib


def _check(rc):
    if rc:
        from . import _check
        _check(rc)


def _elsewhere(device, stream):
    """Whether a call for tensors on ``device`` has to change the current device
    or stream first (``_run_elsewhere`` does)."""
    if device.type != "cuda":
        raise TypeError("the tensors must live on the GPU")
    return stream is not None or device.index != _current_device()


def _run_elsewhere(device, stream, tensors, call):
    """``call()`` with the device and the stream current, so that torch
    allocates there; the tensors are kept until the stream's work is done."""
    with torch.cuda.device(device):
        if stream is None:
            return call()
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        elif stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.stream(stream):
            result = call()
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return result


def _apply(device, stream, tensors, call):
    """``call()``, which makes an autograd node, with the stream current: autograd
    runs the node's backward pass on the stream that was current when it was
    made, and that has to be the one to whose memory pool the tensors that the
    forward pass saves belong."""
    return _run_elsewhere(device, stream, tensors, call) if _elsewhere(device, stream) else call()


def _type(t, what):
    if isinstance(t, torch.Tensor):
        code = _TYPES.get(t.dtype)
        if code is not None:
            # the forward-mode level that is open, -1: none (torch tells it without a look at a tensor)
            if getattr(forward_ad, "_current_level", 0) >= 0 and forward_ad.unpack_dual(t).tangent is not None:
                raise NotImplementedError(f"{what} has a forward-mode tangent, for which there is no rule")
            return code
    raise TypeError(f"{what} must be a float32, float16 or bfloat16 tensor")


def _rows(t, what, dim=None):
    """(rows, spacing) of a tensor of rows along its last dimension."""
    shape = t.shape
    if not shape:
        raise ValueError(f"{what} must have at least one dimension")
    d = shape[-1]
    if dim is not None and d != dim:
        raise ValueError(f"{what} has rows of {d}, {dim} are expected")
    n = t.numel() // d if d else 0
    if t.is_contiguous():
        return n, d
    if d > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} rows must be contiguous (stride(-1) == 1)")
    if n == 1:
        return n, d
    ld = None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld = step = stride
        elif stride != step:
            raise ValueError(f"{what} rows must be equally spaced")
        step = stride * size
    if ld < d:
        raise ValueError(f"{what} rows overlap (spacing {ld}, length {d})")
    return n, ld


def _as_rows(t):
    """``t`` itself where its rows are ones that the kernels take, else a copy."""
    if t.is_contiguous():
        return t
    try:
        _rows(t, "grad")
    except ValueError:
        return t.contiguous()
    return t


def _on(device, t, what):
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")


def _empty_rows(x):
    """Contiguous rows of the shape and type of ``x``."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _param(t, what, dim, row_type, device):
    """Type code of a weight or bias vector."""
    code = _type(t, what)
    if t.shape != (dim,):
        raise ValueError(f"{what} must have the shape [{dim}]")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if code and code != row_type:
        raise TypeError(f"{what} must have the rows' type or float32")
    _on(device, t, what)
    return code


def _ids(ids, device):
    if not isinstance(ids, torch.Tensor) or ids.dtype not in _ID_TYPES:
        raise TypeError("ids must be an int32 or int64 tensor")
    if ids.device != device:
        raise ValueError(f"ids is on {ids.device}, expected {device}")
    return ids if ids.is_contiguous() else ids.contiguous()


def _padding(padding_idx):
    if padding_idx is None:
        return -1
    if padding_idx < 0:
        raise ValueError("padding_idx must be an id (not negative) or None")
    return int(padding_idx)


def _given(out, what, shape, dtype, device):
    """Row spacing of an output that the caller gave."""
    if not isinstance(out, torch.Tensor) or out.dtype != dtype or out.shape != shape:
        raise ValueError(f"{what} must be a {dtype} tensor of shape {list(shape)}")
    _on(device, out, what)
    if out.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what} must not require a gradient")
    return _rows(out, what)[1]


# Tells autograd that a tensor, or each of several, was written, so that a
# backward pass that saved it is refused instead of using the new values.
_written = torch.autograd.graph.increment_version


def embed(weight, ids, scale=1.0, padding_idx=None, dtype=None, out=None, stream=None):
    """``ersj_embed``: ``scale * weight[ids]``, of shape ``ids.shape + [dim]``.

    ``weight``: [rows, dim].  ``dtype``: the result's type, the weight's own by
    default; a float32 weight gives any.  Places that hold ``padding_idx`` get
    zeros; any other id outside the table gets NaN.  Differentiable with
    respect to ``weight`` (the gradient is ``embed_grad``'s)."""
    if weight.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out cannot be given where a gradient is wanted")
        return _apply(weight.device, stream, (weight, ids),
                      lambda: _Embed.apply(weight, ids, scale, padding_idx, dtype))
    return _embed(weight, ids, scale, padding_idx, dtype, out, stream)


def _embed(weight, ids, scale, padding_idx, dtype, out, stream):
    wt = _type(weight, "weight")
    device = weight.device
    if _elsewhere(device, stream):
        return _run_elsewhere(device, stream, (weight, ids, out),
                              lambda: _embed(weight, ids, scale, padding_idx, dtype, out, None))
    if weight.dim() != 2:
        raise ValueError("weight must have two dimensions")
    rows, dim = weight.shape
    dtype = weight.dtype if dtype is None else dtype
    if dtype not in _TYPES:
        raise TypeError("dtype must be float32, float16 or bfloat16")
    ids = _ids(ids, device)
    shape = ids.shape + (dim,)
    given = out is not None
    if given:
        ldo = _given(out, "out", shape, dtype, device)
    else:
        out, ldo = torch.empty(shape, dtype=dtype, device=device), dim
    _check(_library().ersj_embed(weight.data_ptr(), wt, rows, dim, _rows(weight, "weight")[1], ids.data_ptr(),
                                 _ID_TYPES[ids.dtype], ids.numel(), scale, _padding(padding_idx), out.data_ptr(),
                                 _TYPES[dtype], ldo, _raw_stream(device.index)))
    if given:
        _written(out)
    return out


def embed_grad(grad, ids, rows, scale=1.0, padding_idx=None, dtype=None, out=None, accumulate=False, stream=None):
    """``ersj_embed_grad``: the gradient [rows, dim] of an embedding's table
    from ``grad``, of shape ``ids.shape + [dim]``.  ``dtype``: grad's type (the
    default) or float32.  With ``accumulate`` it is added to ``out``."""
    gt = _type(grad, "grad")
    device = grad.device
    if _elsewhere(device, stream):
        return _run_elsewhere(device, stream, (grad, ids, out),
                              lambda: embed_grad(grad, ids, rows, scale, padding_idx, dtype, out, accumulate))
    dtype = dtype or (grad.dtype if out is None else out.dtype)
    if dtype not in _TYPES:
        raise TypeError("dtype must be float32, float16 or bfloat16")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    ids = _ids(ids, device)
    if grad.shape[:-1] != ids.shape:
        raise ValueError(f"grad has the leading shape {list(grad.shape[:-1])}, ids {list(ids.shape)}")
    n, dim = ids.numel(), grad.shape[-1]
    L = _library()
    need = L.ersj_embed_grad_work(n, rows, dim)
    work = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    given = out is not None
    if given:
        ldo = _given(out, "out", (rows, dim), dtype, device)
    else:
        out, ldo = torch.empty((rows, dim), dtype=dtype, device=device), dim
    _check(L.ersj_embed_grad(grad.data_ptr(), gt, _rows(grad, "grad")[1], ids.data_ptr(), _ID_TYPES[ids.dtype], n,
                             scale, _padding(padding_idx), out.data_ptr(), _TYPES[dtype], rows, dim, ldo,
                             1 if accumulate else 0, work.data_ptr() if need else None, need, _raw_stream(device.index)))
    if given:
        _written(out)
    return out


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, padding_idx, dtype):
        ctx.save_for_backward(ids)
        ctx.args = (weight.shape[0], weight.dtype, scale, padding_idx)
        return _embed(weight, ids, scale, padding_idx, dtype, None, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        rows, dtype, scale, padding_idx = ctx.args
        return embed_grad(_as_rows(grad), ctx.saved_tensors[0], rows, scale, padding_idx, dtype), None, None, None, None


class PackedRows:
    """Rows held in 8 bits (``ersj_pack_rows``): ``codes``, int8 of the rows'
    ``shape``, ``scales``, uint8 with one for each run of 32 along a row, and
    ``dtype``, the rows' type."""

    __slots__ = ("codes", "scales", "dtype")

    def __init__(self, codes, scales, dtype):
        if dtype not in _TYPES:
            raise TypeError("dtype must be float32, float16 or bfloat16")
        for what, t, kind in (("codes", codes, torch.int8), ("scales", scales, torch.uint8)):
            if not isinstance(t, torch.Tensor) or t.dtype != kind or not t.is_contiguous():
                raise ValueError(f"{what} must be a contiguous {kind} tensor")
        if not codes.dim() or not codes.shape[-1]:
            raise ValueError("codes must have rows")
        shape = codes.shape[:-1] + (-(-codes.shape[-1] // PACK_BLOCK),)
        if scales.shape != shape:
            raise ValueError(f"scales must have the shape {list(shape)}")
        _on(codes.device, scales, "scales")
        self.codes, self.scales, self.dtype = codes, scales, dtype

    @property
    def shape(self):
        return self.codes.shape

    @property
    def device(self):
        return self.codes.device


def _empty_packed(shape, dtype, device):
    codes = torch.empty(shape, dtype=torch.int8, device=device)
    scales = torch.empty(shape[:-1] + (-(-shape[-1] // PACK_BLOCK),), dtype=torch.uint8, device=device)
    return _packed(codes, scales, dtype)


def _packed(codes, scales, dtype):
    """PackedRows of tensors made here, which need no checks."""
    kept = object.__new__(PackedRows)
    kept.codes, kept.scales, kept.dtype = codes, scales, dtype
    return kept


def pack_rows(x, stream=None):
    """``ersj_pack_rows``: the rows of ``x`` in 8 bits, as ``PackedRows``: whole
    multiples of a power of two for each run of 32 along a row, off by less than
    1/127 of the largest of the run (by up to 1/64 in runs that reach 63.5 * 2^10 in
    float16 or 63.5 * 2^122 in the others, by up to 2^-127 in runs below 2^-120).
    Not differentiable; ``layer_norm`` and
    ``gated`` keep their input so with ``pack=True``."""
    xt = _type(x, "x")
    device = x.device
    if _elsewhere(device, stream):
        return _run_elsewhere(device, stream, (x,), lambda: pack_rows(x))
    n, ldx = _rows(x, "x")
    kept = _empty_packed(x.shape, x.dtype, device)
    _check(_library().ersj_pack_rows(x.data_ptr(), xt, n, x.shape[-1], ldx, kept.codes.data_ptr(),
                                     kept.scales.data_ptr(), _raw_stream(device.index)))
    return kept


def unpack_rows(packed, out=None, stream=None):
    """``ersj_unpack_rows``: the values that the rows stand for, in their type."""
    if not isinstance(packed, PackedRows):
        raise TypeError("packed must be PackedRows")
    device = packed.device
    if _elsewhere(device, stream):
        return _run_elsewhere(device, stream, (packed.codes, packed.scales, out), lambda: unpack_rows(packed, out))
    shape = packed.shape
    dim = shape[-1]
    given = out is not None
    if given:
        ldo = _given(out, "out", shape, packed.dtype, device)
    else:
        out, ldo = torch.empty(shape, dtype=packed.dtype, device=device), dim
    _check(_library().ersj_unpack_rows(packed.codes.data_ptr(), packed.scales.data_ptr(), packed.codes.numel() // dim,
                                       dim, out.data_ptr(), _TYPES[packed.dtype], ldo, _raw_stream(device.index)))
    if given:
        _written(out)
    return out


def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, stream=None, pack=False):
    """``ersj_layer_norm`` over the last dimension: (y, mean, rstd), mean and
    rstd float32 of shape ``x.shape[:-1]``.  ``weight`` and ``bias``: [dim], of
    x's type or float32 (both of one type), or None.  ``out`` may be ``x``.
    Differentiable with respect to x, weight and bias (``layer_norm_grad``); with
    ``pack`` the backward pass keeps x in 8 bits (``PackedRows``)."""
    if ((x.requires_grad or (weight is not None and weight.requires_grad) or (bias is not None and bias.requires_grad))
            and torch.is_grad_enabled()):
        if out is not None:
            raise ValueError("out cannot be given where a gradient is wanted")
        node = _LayerNormPacked if pack else _LayerNorm
        return _apply(x.device, stream, (x, weight, bias), lambda: node.apply(x, weight, bias, eps))
    return _layer_norm(x, weight, bias, eps, out, stream)


def layer_norm_pack(x, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """``ersj_layer_norm_pack``: ``layer_norm`` and ``pack_rows`` of x in one pass,
    (y, mean, rstd, PackedRows), for ``layer_norm_grad``.  Not differentiable."""
    return _layer_norm(x, weight, bias, eps, out, stream, True)


def _layer_norm(x, weight, bias, eps, out, stream, pack=False):
    xt = _type(x, "x")
    device = x.device
    if _elsewhere(device, stream):
        return _run_elsewhere(device, stream, (x, weight, bias, out),
                              lambda: _layer_norm(x, weight, bias, eps, out, None, pack))
    n, ldx = _rows(x, "x")
    shape = x.shape
    dim = shape[-1]
    pt, w, b = 0, None, None
    if weight is not None:
        pt = _param(weight, "weight", dim, xt, device)
        w = weight.data_ptr()
    if bias is not None:
        bt = _param(bias, "bias", dim, xt, device)
        if w is not None and bt != pt:
            raise TypeError("weight and bias must have one type")
        pt, b = bt, bias.data_ptr()
    given = out is not None
    if given:
        ldy = _given(out, "out", shape, x.dtype, device)
    else:
        out, ldy = _empty_rows(x), dim
    mean = torch.empty(shape[:-1], dtype=torch.float32, device=device)
    rstd = torch.empty_like(mean)
    if pack:
        kept = _empty_packed(shape, x.dtype, device)
        _check(_library().ersj_layer_norm_pack(x.data_ptr(), xt, n, dim, ldx, w, b, pt, eps, out.data_ptr(), ldy,
                                               mean.data_ptr(), rstd.data_ptr(), kept.codes.data_ptr(),
                                               kept.scales.data_ptr(), _raw_stream(device.index)))
        if given:
            _written(out)
        return out, mean, rstd, kept
    _check(_library().ersj_layer_norm(x.data_ptr(), xt, n, dim, ldx, w, b, pt, eps, out.data_ptr(), ldy,
                                      mean.data_ptr(), rstd.data_ptr(), _raw_stream(device.index)))
    if given:
        _written(out)
    return out, mean, rstd


def layer_norm_grad(grad, x, mean, rstd, weight=None, dtype=None, want_x=True, want_params=True, stream=None):
    """``ersj_layer_norm_grad``: (grad of x, of weight, of bias) from ``grad``,
    the gradient of y, and what ``layer_norm`` returned.  ``x``: the rows, or
    ``PackedRows`` of them (``ersj_layer_norm_grad_packed``).  The last two have
    ``dtype``: the weight's type (the default; float32 without one), x's, or float32.
    What is not wanted comes back as None."""
    if type(x) is PackedRows:
        return _layer_norm_grad_packed(grad, x, mean, rstd, weight, dtype, want_x, want_params, stream)
    xt = _type(x, "x")
    if _type(grad, "grad") != xt:
        raise TypeError("grad must have the type of x")
    device = x.device
    if _elsewhere(device, stream):
        return _run_elsewhere(device, stream, (grad, x, mean, rstd, weight),
                              lambda: layer_norm_grad(grad, x, mean, rstd, weight, dtype, want_x, want_params))
    n, ldx = _rows(x, "x")
    dim, pt, w, dtype = _norm_grad_args(grad, x, mean, rstd, weight, dtype, xt, device)
    L = _library()
    gx = _empty_rows(x) if want_x else None
    gw = gb = work = None
    need = 0
    if want_params:
        gw = torch.empty(dim, dtype=dtype, device=device)
        gb = torch.empty_like(gw)
        need = L.ersj_layer_norm_grad_work(n, dim)
        if need:
            work = torch.empty(need, dtype=torch.uint8, device=device)
    _check(L.ersj_layer_norm_grad(grad.data_ptr(), _rows(grad, "grad")[1], x.data_ptr(), ldx, xt, n, dim,
                                  mean.data_ptr(), rstd.data_ptr(), w, pt, gx.data_ptr() if want_x else None, dim,
                                  gw.data_ptr() if want_params else None, gb.data_ptr() if want_params else None,
                                  work.data_ptr() if need else None, need, _raw_stream(device.index)))
    return gx, gw, gb


def _norm_grad_args(grad, x, mean, rstd, weight, dtype, xt, device):
    """(dim, type code and address of the weight, type of its gradient) of checked arguments."""
    shape = x.shape
    if grad.shape != shape:
        raise ValueError(f"grad has the shape {list(grad.shape)}, x {list(shape)}")
    _on(device, grad, "grad")
    dim = shape[-1]
    for what, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != torch.float32 or t.shape != shape[:-1] or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous float32 tensor of shape {list(shape[:-1])}")
        _on(device, t, what)
    if weight is None:
        dtype = dtype or torch.float32
        pt, w = _TYPES.get(dtype), None
        if pt is None or (pt and pt != xt):
            raise TypeError("dtype must be the type of x or float32")
    else:
        pt, w = _param(weight, "weight", dim, xt, device), weight.data_ptr()
        if dtype is None:
            dtype = weight.dtype
        elif dtype != weight.dtype:
            raise TypeError("the gradients of weight and bias have the weight's type")
    return dim, pt, w, dtype


def _layer_norm_grad_packed(grad, x, mean, rstd, weight, dtype, want_x, want_params, stream):
    xt = _TYPES[x.dtype]
    if _type(grad, "grad") != xt:
        raise TypeError("grad must have the type of x")
    device = x.device
    if _elsewhere(device, stream):
        return _run_elsewhere(device, stream, (grad, x.codes, x.scales, mean, rstd, weight),
                              lambda: layer_norm_grad(grad, x, mean, rstd, weight, dtype, want_x, want_params))
    dim, pt, w, dtype = _norm_grad_args(grad, x, mean, rstd, weight, dtype, xt, device)
    n = x.codes.numel() // dim
    L = _library()
    gx = torch.empty(x.shape, dtype=x.dtype, device=device) if want_x else None
    gw = gb = None
    if want_params:
        gw = torch.empty(dim, dtype=dtype, device=device)
        gb = torch.empty_like(gw)
    need = L.ersj_layer_norm_grad_packed_work(xt, n, dim)
    work = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _check(L.ersj_layer_norm_grad_packed(grad.data_ptr(), _rows(grad, "grad")[1], x.codes.data_ptr(),
                                         x.scales.data_ptr(), xt, n, dim, mean.data_ptr(), rstd.data_ptr(), w, pt,
                                         gx.data_ptr() if want_x else None, dim, gw.data_ptr() if want_params else None,
                                         gb.data_ptr() if want_params else None, work.data_ptr() if need else None,
                                         need, _raw_stream(device.index)))
    return gx, gw, gb


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = _layer_norm(x, weight, bias, eps, None, None)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        ctx.mark_non_differentiable(mean, rstd)
        return y, mean, rstd

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, _mean, _rstd):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        params = need[1] or need[2]
        dtype = ctx.bias_dtype if weight is None else weight.dtype
        gx, gw, gb = layer_norm_grad(_as_rows(grad), x, mean, rstd, weight, dtype, need[0], params)
        return gx, gw if need[1] else None, gb if need[2] else None, None


class _LayerNormPacked(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd, kept = _layer_norm(x, weight, bias, eps, None, None, True)
        ctx.save_for_backward(kept.codes, kept.scales, weight, mean, rstd)
        ctx.dtypes = kept.dtype, None if bias is None else bias.dtype
        ctx.mark_non_differentiable(mean, rstd)
        return y, mean, rstd

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, _mean, _rstd):
        codes, scales, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        params = need[1] or need[2]
        dtype = ctx.dtypes[1] if weight is None else weight.dtype
        gx, gw, gb = layer_norm_grad(_as_rows(grad), _packed(codes, scales, ctx.dtypes[0]), mean, rstd, weight, dtype,
                                     need[0], params)
        return gx, gw if need[1] else None, gb if need[2] else None, None


def _tensor_arrays(grads, out):
    """(count, addresses, those of the outputs or None, sizes, types) of tensors
    to clip, checked, as the entry points take them."""
    if not grads:
        raise ValueError("grads is empty")
    if out is not None and len(out) != len(grads):
        raise ValueError(f"out holds {len(out)} tensors, grads {len(grads)}")
    types = []
    for i, g in enumerate(grads):
        types.append(_type(g, f"grads[{i}]"))
        if not g.is_contiguous():
            raise ValueError(f"grads[{i}] must be contiguous")
        _on(grads[0].device, g, f"grads[{i}]")
        if out is not None:
            o = out[i]
            if not isinstance(o, torch.Tensor) or o.dtype != g.dtype or o.shape != g.shape or not o.is_contiguous():
                raise ValueError(f"out[{i}] must be a contiguous tensor of the type and shape of grads[{i}]")
            _on(g.device, o, f"out[{i}]")
    n = len(grads)
    addresses = ctypes.c_void_p * n
    return (n, addresses(*[g.data_ptr() for g in grads]),
            None if out is None else addresses(*[o.data_ptr() for o in out]),
            (ctypes.c_int64 * n)(*[g.numel() for g in grads]), (ctypes.c_int32 * n)(*types))


class GradSet:
    """Owner of an ``ersj_grads*``: gradient tensors that are clipped together.

    ``grads``: contiguous GPU tensors on one device, of any types and sizes.
    ``out``: tensors of the same shapes and types that receive the clipped
    gradients; None clips in place.  Tensors that share memory are refused where
    it is written.  The set keeps the tensors alive and reads their values anew
    on every call; it is made once for tensors that a training loop reuses, and
    has to outlive a captured graph that clips it."""

    def __init__(self, grads, out=None, stream=None):
        self.handle = ctypes.c_void_p()
        self.grads = list(grads)
        self.out = None if out is None else list(out)
        arrays = _tensor_arrays(self.grads, self.out)
        self.device = self.grads[0].device

        def create():
            _check(_library().ersj_grads_create(*arrays, _raw_stream(self.device.index), ctypes.byref(self.handle)))

        if _elsewhere(self.device, stream):
            _run_elsewhere(self.device, stream, (), create)
        else:
            create()

    def free(self):
        if self.handle and self.handle.value:
            _library().ersj_grads_free(self.handle)
            self.handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def clip_grads(grads, max_norm, stream=None):
    """``ersj_grads_clip``: scale the gradients so that their global norm is at
    most ``max_norm``; the norm before, as a float32 tensor of no dimensions.
    ``grads``: a ``GradSet``, or tensors to clip in place (``ersj_clip_tensors``;
    they may be others on every call; none may share memory with another)."""
    kept = grads if isinstance(grads, GradSet) else None
    if kept is None:
        grads = list(grads)
        arrays = _tensor_arrays(grads, None)
        device = grads[0].device
    else:
        device = kept.device
    if _elsewhere(device, stream):
        tensors = grads if kept is None else kept.grads + (kept.out or [])
        return _run_elsewhere(device, stream, tensors, lambda: clip_grads(grads, max_norm))
    L = _library()
    need = GRADS_WORK if kept else L.ersj_clip_tensors_work(arrays[0], *arrays[3:])
    work = torch.empty(need, dtype=torch.uint8, device=device)
    norm = torch.empty((), dtype=torch.float32, device=device)
    end = (max_norm, norm.data_ptr(), work.data_ptr(), need, _raw_stream(device.index))
    if kept:
        _check(L.ersj_grads_clip(kept.handle, *end))
        _written(kept.grads if kept.out is None else kept.out)
    else:
        _check(L.ersj_clip_tensors(*arrays, *end))
        _written(grads)
    return norm
