"""Operators of the encoder whose vectors the join compares: token embedding,
layer norm, their gradients, and clipping by the global gradient norm.

Binding of ``include/ersj_encoder.h``.  The functions carry the C names
without the ``ersj_`` prefix, check and marshal their arguments, and take
output and working memory from torch; all arithmetic runs in the library's
HIP kernels.  ``embed`` and ``layer_norm`` take part in autograd.

Tensors are float32, float16 or bfloat16 on the GPU.  A tensor of rows may
have any leading shape as long as its rows are contiguous and equally spaced.
``stream`` (a torch stream or a raw handle; None: the current one) is where
the work is enqueued; outputs belong to that stream.
"""
import ctypes

import torch

_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}  # ERSJ_F32, ERSJ_F16, ERSJ_BF16
_ID_TYPES = {torch.int32: 0, torch.int64: 1}                      # ERSJ_I32, ERSJ_I64
GRADS_WORK = 16384                                                # ERSJ_GRADS_WORK

ENCODER_SYMBOLS = ("ersj_embed", "ersj_embed_grad", "ersj_embed_grad_work", "ersj_layer_norm",
                   "ersj_layer_norm_grad", "ersj_layer_norm_grad_work", "ersj_grads_create", "ersj_grads_clip",
                   "ersj_grads_free")


def declare(L):
    """Argument types of the entry points on the loaded library."""
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
    L.ersj_grads_free.argtypes = [vp]
    L.ersj_grads_free.restype = None


def _core():
    import exact_range_similarity_amd as ersj
    return ersj


def _check(rc):
    if rc:
        _core()._check(rc)


class _Place:
    """The device and stream of a call.  Inside, torch allocates on that
    stream; tensors of another stream are kept until its work is done."""
    __slots__ = ("raw", "side", "_ctx")

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise TypeError("the tensors must live on the GPU")
        self.side = None
        if stream is None:
            if device.index != torch.cuda.current_device():
                self._ctx = torch.cuda.device(device)
            else:
                self._ctx = None
            self.raw = torch.cuda.current_stream(device).cuda_stream
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            elif stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
            self._ctx = torch.cuda.stream(stream)
            self.raw = stream.cuda_stream
            self.side = stream

    def __enter__(self):
        if self._ctx is not None:
            self._ctx.__enter__()
        return self

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)
        return False

    def keep(self, *tensors):
        if self.side is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.side)


def _type(t, what):
    if not isinstance(t, torch.Tensor) or t.dtype not in _TYPES:
        raise TypeError(f"{what} must be a float32, float16 or bfloat16 tensor")
    return _TYPES[t.dtype]


def _rows(t, what, dim=None):
    """(rows, spacing) of a tensor of rows along its last dimension."""
    if t.dim() < 1:
        raise ValueError(f"{what} must have at least one dimension")
    d = t.shape[-1]
    if dim is not None and d != dim:
        raise ValueError(f"{what} has rows of {d}, {dim} are expected")
    n = t.numel() // d if d else 0
    if n <= 1 or t.is_contiguous():
        if d > 1 and n and t.stride(-1) != 1:
            raise ValueError(f"{what} rows must be contiguous (stride(-1) == 1)")
        return n, d
    if d > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} rows must be contiguous (stride(-1) == 1)")
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


def _same_device(device, **tensors):
    for what, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{what} is on {t.device}, expected {device}")


def _param(t, what, dim, row_type):
    """Type code of a weight or bias vector."""
    code = _type(t, what)
    if t.dim() != 1 or t.shape[0] != dim:
        raise ValueError(f"{what} must have the shape [{dim}]")
    if dim > 1 and t.stride(0) != 1:
        raise ValueError(f"{what} must be contiguous")
    if code and code != row_type:
        raise TypeError(f"{what} must have the rows' type or float32")
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


def _output(out, what, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(out, torch.Tensor) or out.dtype != dtype or tuple(out.shape) != tuple(shape):
        raise ValueError(f"{what} must be a {dtype} tensor of shape {list(shape)}")
    if out.device != device:
        raise ValueError(f"{what} is on {out.device}, expected {device}")
    return out


def embed(weight, ids, scale=1.0, padding_idx=None, dtype=None, out=None, stream=None):
    """``ersj_embed``: ``scale * weight[ids]``, of shape ``ids.shape + [dim]``.

    ``weight``: [rows, dim].  ``dtype``: the result's type, the weight's own by
    default; a float32 weight gives any.  Places that hold ``padding_idx`` get
    zeros; any other id outside the table gets NaN.  Differentiable with
    respect to ``weight`` (the gradient is ``embed_grad``'s)."""
    if torch.is_grad_enabled() and weight.requires_grad:
        if out is not None:
            raise ValueError("out cannot be given where a gradient is wanted")
        return _Embed.apply(weight, ids, scale, padding_idx, dtype, stream)
    return _embed(weight, ids, scale, padding_idx, dtype, out, stream)


def _embed(weight, ids, scale, padding_idx, dtype, out, stream):
    wt = _type(weight, "weight")
    if weight.dim() != 2:
        raise ValueError("weight must have two dimensions")
    rows, dim = weight.shape
    device = weight.device
    dtype = weight.dtype if dtype is None else dtype
    if dtype not in _TYPES:
        raise TypeError("dtype must be float32, float16 or bfloat16")
    with _Place(device, stream) as at:
        ids = _ids(ids, device)
        ldw = _rows(weight, "weight")[1]
        out = _output(out, "out", ids.shape + (dim,), dtype, device)
        ldo = _rows(out, "out")[1]
        _check(_core().lib().ersj_embed(weight.data_ptr(), wt, rows, dim, ldw, ids.data_ptr(), _ID_TYPES[ids.dtype],
                                        ids.numel(), scale, _padding(padding_idx), out.data_ptr(), _TYPES[dtype],
                                        ldo, at.raw))
        at.keep(weight, ids, out)
    return out


def embed_grad(grad, ids, rows, scale=1.0, padding_idx=None, dtype=None, out=None, accumulate=False, stream=None):
    """``ersj_embed_grad``: the gradient [rows, dim] of an embedding's table
    from ``grad``, of shape ``ids.shape + [dim]``.  ``dtype``: grad's type (the
    default) or float32.  With ``accumulate`` it is added to ``out``."""
    gt = _type(grad, "grad")
    device = grad.device
    dtype = dtype or (grad.dtype if out is None else out.dtype)
    if dtype not in _TYPES:
        raise TypeError("dtype must be float32, float16 or bfloat16")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    with _Place(device, stream) as at:
        ids = _ids(ids, device)
        if grad.shape[:-1] != ids.shape:
            raise ValueError(f"grad has the leading shape {list(grad.shape[:-1])}, ids {list(ids.shape)}")
        n, dim = ids.numel(), grad.shape[-1]
        ldg = _rows(grad, "grad")[1]
        out = _output(out, "out", (rows, dim), dtype, device)
        ldo = _rows(out, "out")[1]
        L = _core().lib()
        work = torch.empty(L.ersj_embed_grad_work(n, rows, dim), dtype=torch.uint8, device=device)
        _check(L.ersj_embed_grad(grad.data_ptr(), gt, ldg, ids.data_ptr(), _ID_TYPES[ids.dtype], n, scale,
                                 _padding(padding_idx), out.data_ptr(), _TYPES[dtype], rows, dim, ldo,
                                 1 if accumulate else 0, work.data_ptr(), work.numel(), at.raw))
        at.keep(grad, ids, out)
    return out


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, padding_idx, dtype, stream):
        ctx.save_for_backward(ids)
        ctx.args = (weight.shape[0], weight.dtype, scale, padding_idx)
        return _embed(weight, ids, scale, padding_idx, dtype, None, stream)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        rows, dtype, scale, padding_idx = ctx.args
        return embed_grad(grad.contiguous(), ctx.saved_tensors[0], rows, scale, padding_idx, dtype), None, None, None, None, None


def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """``ersj_layer_norm`` over the last dimension: (y, mean, rstd), mean and
    rstd float32 of shape ``x.shape[:-1]``.  ``weight`` and ``bias``: [dim], of
    x's type or float32 (both of one type), or None.  ``out`` may be ``x``.
    Differentiable with respect to x, weight and bias (``layer_norm_grad``)."""
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad)
                                    or (bias is not None and bias.requires_grad)):
        if out is not None:
            raise ValueError("out cannot be given where a gradient is wanted")
        return _LayerNorm.apply(x, weight, bias, eps, stream)
    return _layer_norm(x, weight, bias, eps, out, stream)


def _layer_norm(x, weight, bias, eps, out, stream):
    xt = _type(x, "x")
    device = x.device
    with _Place(device, stream) as at:
        n, ldx = _rows(x, "x")
        dim = x.shape[-1]
        pt = 0
        if weight is not None:
            pt = _param(weight, "weight", dim, xt)
        if bias is not None:
            bt = _param(bias, "bias", dim, xt)
            if weight is not None and bt != pt:
                raise TypeError("weight and bias must have one type")
            pt = bt
        _same_device(device, weight=weight, bias=bias)
        out = _output(out, "out", x.shape, x.dtype, device)
        ldy = _rows(out, "out")[1]
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=device)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=device)
        _check(_core().lib().ersj_layer_norm(x.data_ptr(), xt, n, dim, ldx,
                                             None if weight is None else weight.data_ptr(),
                                             None if bias is None else bias.data_ptr(), pt, eps, out.data_ptr(), ldy,
                                             mean.data_ptr(), rstd.data_ptr(), at.raw))
        at.keep(x, weight, bias, out)
    return out, mean, rstd


def layer_norm_grad(grad, x, mean, rstd, weight=None, dtype=None, want_x=True, want_params=True, stream=None):
    """``ersj_layer_norm_grad``: (grad of x, of weight, of bias) from ``grad``,
    the gradient of y, and what ``layer_norm`` returned.  The last two have
    ``dtype``: the weight's type (the default; float32 without one), x's, or float32.
    What is not wanted comes back as None."""
    xt = _type(x, "x")
    if _type(grad, "grad") != xt:
        raise TypeError("grad must have the type of x")
    device = x.device
    if grad.shape != x.shape:
        raise ValueError(f"grad has the shape {list(grad.shape)}, x {list(x.shape)}")
    with _Place(device, stream) as at:
        n, ldx = _rows(x, "x")
        ldg = _rows(grad, "grad")[1]
        dim = x.shape[-1]
        for what, t in (("mean", mean), ("rstd", rstd)):
            if t.dtype != torch.float32 or t.shape != x.shape[:-1] or not t.is_contiguous():
                raise ValueError(f"{what} must be a contiguous float32 tensor of shape {list(x.shape[:-1])}")
        _same_device(device, grad=grad, mean=mean, rstd=rstd, weight=weight)
        pt = 0 if weight is None else _param(weight, "weight", dim, xt)
        if dtype is None:
            dtype = torch.float32 if weight is None else weight.dtype
        if weight is None:
            pt = _TYPES[dtype]
        elif _TYPES.get(dtype) != pt:
            raise TypeError("the gradients of weight and bias have the weight's type")
        gx = torch.empty(x.shape, dtype=x.dtype, device=device) if want_x else None
        gw = gb = work = None
        work_bytes = 0
        L = _core().lib()
        if want_params:
            gw = torch.empty(dim, dtype=dtype, device=device)
            gb = torch.empty(dim, dtype=dtype, device=device)
            work_bytes = L.ersj_layer_norm_grad_work(n, dim)
            work = torch.empty(work_bytes, dtype=torch.uint8, device=device)
        _check(L.ersj_layer_norm_grad(grad.data_ptr(), ldg, x.data_ptr(), ldx, xt, n, dim, mean.data_ptr(),
                                      rstd.data_ptr(), None if weight is None else weight.data_ptr(), pt,
                                      gx.data_ptr() if want_x else None, dim, gw.data_ptr() if want_params else None,
                                      gb.data_ptr() if want_params else None, work.data_ptr() if want_params else None,
                                      work_bytes, at.raw))
        at.keep(grad, x, mean, rstd, weight)
    return gx, gw, gb


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, stream):
        y, mean, rstd = _layer_norm(x, weight, bias, eps, None, stream)
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
        gx, gw, gb = layer_norm_grad(grad.contiguous(), x, mean, rstd, weight, dtype, need[0], params)
        return gx, gw if need[1] else None, gb if need[2] else None, None, None


class GradSet:
    """Owner of an ``ersj_grads*``: gradient tensors that are clipped together.

    ``grads``: contiguous GPU tensors on one device, of any types and sizes.
    ``out``: tensors of the same shapes and types that receive the clipped
    gradients; None clips in place.  The set keeps the tensors alive and reads
    their values anew on every call; it is made once for tensors that a
    training loop reuses."""

    def __init__(self, grads, out=None, stream=None):
        self.handle = ctypes.c_void_p()
        self.grads = list(grads)
        self.out = None if out is None else list(out)
        if not self.grads:
            raise ValueError("grads is empty")
        if self.out is not None and len(self.out) != len(self.grads):
            raise ValueError(f"out holds {len(self.out)} tensors, grads {len(self.grads)}")
        for i, g in enumerate(self.grads):
            _type(g, f"grads[{i}]")
            if not g.is_contiguous():
                raise ValueError(f"grads[{i}] must be contiguous")
            _same_device(self.grads[0].device, **{f"grads[{i}]": g})
            if self.out is not None:
                o = self.out[i]
                if not isinstance(o, torch.Tensor) or o.dtype != g.dtype or o.shape != g.shape or not o.is_contiguous():
                    raise ValueError(f"out[{i}] must be a contiguous tensor of the type and shape of grads[{i}]")
                _same_device(g.device, **{f"out[{i}]": o})
        n = len(self.grads)
        self.device = self.grads[0].device
        ptrs = (ctypes.c_void_p * n)(*[g.data_ptr() for g in self.grads])
        outs = None if self.out is None else (ctypes.c_void_p * n)(*[o.data_ptr() for o in self.out])
        sizes = (ctypes.c_int64 * n)(*[g.numel() for g in self.grads])
        types = (ctypes.c_int32 * n)(*[_TYPES[g.dtype] for g in self.grads])
        with _Place(self.device, stream) as at:
            _check(_core().lib().ersj_grads_create(n, ptrs, outs, sizes, types, at.raw, ctypes.byref(self.handle)))

    def free(self):
        if self.handle and self.handle.value:
            _core().lib().ersj_grads_free(self.handle)
            self.handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def clip_grads(grads, max_norm, stream=None):
    """``ersj_grads_clip``: scale the gradients so that their global norm is at
    most ``max_norm``; the norm before, as a float32 tensor of no dimensions.
    ``grads``: a ``GradSet``, or tensors to clip in place."""
    gs = grads if isinstance(grads, GradSet) else GradSet(grads, stream=stream)
    with _Place(gs.device, stream) as at:
        work = torch.empty(GRADS_WORK, dtype=torch.uint8, device=gs.device)
        norm = torch.empty((), dtype=torch.float32, device=gs.device)
        _check(_core().lib().ersj_grads_clip(gs.handle, max_norm, norm.data_ptr(), work.data_ptr(), GRADS_WORK, at.raw))
        at.keep(*gs.grads, *(gs.out or ()))
    return norm
