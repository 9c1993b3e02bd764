"""Plain 64-bit forms of the encoder operators and bounds on the error of a
32-bit evaluation, shared by their tests.

u = 2^-24 is the unit roundoff of 32-bit arithmetic, ``unit(dtype)`` that of
a result's type (2^-24, 2^-11, 2^-8) and ``tiny(dtype)`` half its smallest
subnormal step.  A sum of m terms in any order has an error of at most about
m * u times the sum of their absolute values.
"""
import torch

U = 2.0 ** -24
F64 = torch.float64
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def unit(dtype):
    return {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dtype]


def tiny(dtype):
    return {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}[dtype]


def rounded(ref, err, dtype):
    """Bound for a result with 32-bit error ``err`` that is rounded to dtype.
    The last factor covers the second-order terms of the bounds above."""
    return (err * (1 + unit(dtype)) + ref.abs() * unit(dtype) + tiny(dtype)) * 1.01 + 2.0 ** -140


def close(got, ref, bound, label=""):
    # what rounds to infinity in the result's type is expected as infinity
    over = torch.isinf(ref.to(got.dtype))
    ref = torch.where(over, ref.to(got.dtype).to(F64), ref)
    got = got.to(F64)
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    diff = torch.where(same, torch.zeros_like(ref), (got - ref).abs())
    bad = ~(diff <= bound) & ~same
    if bool(bad.any()):
        k = int(bad.reshape(-1).nonzero()[0])
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} values off, first at {k}: "
                             f"{float(got.reshape(-1)[k])!r}, expected {float(ref.reshape(-1)[k])!r}, "
                             f"bound {float(bound.expand_as(ref).reshape(-1)[k])!r}")


# ---- embedding ----

def embed_ref(weight, ids, scale, pad):
    rows = weight.shape[0]
    ids = ids.long()
    bad = (ids < 0) | (ids >= rows)
    out = weight.to(F64)[ids.clamp(0, rows - 1)] * scale
    out[bad] = float("nan")
    if pad is not None:
        out[ids == pad] = 0.0
    return out


def check_embed(got, weight, ids, scale, pad, label=""):
    ref = embed_ref(weight, ids, scale, pad)
    # one product in 32 bits, one rounding of it
    close(got, ref, rounded(ref, ref.abs() * U, got.dtype), label)


def embed_grad_ref(grad, ids, rows, scale, pad):
    """(sums, sums of absolute values, counts)"""
    dim = grad.shape[-1]
    ids = ids.reshape(-1).long()
    g = grad.reshape(-1, dim)
    keep = (ids >= 0) & (ids < rows)
    if pad is not None:
        keep &= ids != pad
    out = torch.zeros((rows, dim), dtype=F64, device=grad.device)
    mag = torch.zeros_like(out)
    for c in range(0, ids.numel(), 1 << 20):
        k = keep[c:c + (1 << 20)]
        part = g[c:c + (1 << 20)][k].to(F64) * scale
        at = ids[c:c + (1 << 20)][k]
        out.index_add_(0, at, part)
        mag.index_add_(0, at, part.abs())
    return out, mag, torch.bincount(ids[keep], minlength=rows)


def check_embed_grad(got, grad, ids, rows, scale, pad, before=None, label=""):
    ref, mag, count = embed_grad_ref(grad, ids, rows, scale, pad)
    err = (count[:, None] + 2) * U * mag  # count additions, the product with the scale
    if before is not None:
        ref = ref + before.to(F64)
        err = err + U * ref.abs()
    close(got, ref, rounded(ref, err, got.dtype), label)
    if before is None:
        assert bool((got[count == 0] == 0).all()), f"{label}: a row without tokens is not zero"


# ---- layer norm ----

def norm_ref(x, weight, bias, eps):
    x = x.to(F64)
    mean = x.mean(dim=-1, keepdim=True)
    var = (x - mean).square().mean(dim=-1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    xh = (x - mean) * rstd
    y = xh
    if weight is not None:
        y = y * weight.to(F64)
    if bias is not None:
        y = y + bias.to(F64)
    return y, mean, rstd, xh


def check_norm(got, x, weight, bias, eps, label=""):
    y, mean, rstd = got
    dim = x.shape[-1]
    ref, rmean, rrstd, xh = norm_ref(x, weight, bias, eps)
    # a sum of dim terms and a division
    emean = (dim + 1) * U * x.to(F64).abs().mean(dim=-1, keepdim=True)
    close(mean, rmean[..., 0], rounded(rmean, emean, torch.float32)[..., 0], label + " mean")
    # squares of differences (3 roundings each) from a mean off by emean, their
    # sum, the division, eps, the root and the reciprocal (the first two halved)
    erel = (dim + 8) / 2 * U + (emean * rrstd).square() / 2 + 3 * U
    close(rstd, rrstd[..., 0], rounded(rrstd, erel * rrstd, torch.float32)[..., 0], label + " rstd")
    w = torch.ones(dim, dtype=F64, device=x.device) if weight is None else weight.to(F64)
    scaled = xh * w
    err = (w * rrstd * emean).abs() + scaled.abs() * (erel + 3 * U) + U * (ref.abs() + scaled.abs())
    close(y, ref, rounded(ref, err, y.dtype), label + " y")


def norm_grad_ref(grad, x, mean, rstd, weight):
    """The gradient from the given statistics, and the terms of its bounds."""
    dim = x.shape[-1]
    dy, x = grad.to(F64), x.to(F64)
    rstd = rstd.to(F64).unsqueeze(-1)
    xh = (x - mean.to(F64).unsqueeze(-1)) * rstd
    g = dy if weight is None else dy * weight.to(F64)
    s1 = g.mean(dim=-1, keepdim=True)
    s2 = (g * xh).mean(dim=-1, keepdim=True)
    gx = rstd * (g - s1 - xh * s2)
    err = rstd * ((dim + 3) * U * g.abs().mean(dim=-1, keepdim=True)
                  + xh.abs() * (dim + 6) * U * (g * xh).abs().mean(dim=-1, keepdim=True)
                  + 4 * U * (g.abs() + s1.abs() + (xh * s2).abs()) + 4 * U * (xh * s2).abs())
    flat = (dy * xh).reshape(-1, dim)
    fdy = dy.reshape(-1, dim)
    return gx, err, flat.sum(0), flat.abs().sum(0), fdy.sum(0), fdy.abs().sum(0)


def check_norm_grad(got, grad, x, mean, rstd, weight, label=""):
    gx, gw, gb = got
    rx, err, rw, mw, rb, mb = norm_grad_ref(grad, x, mean, rstd, weight)
    n = x.numel() // x.shape[-1]
    if gx is not None:
        close(gx, rx, rounded(rx, err, gx.dtype), label + " grad_x")
    if gw is not None:
        close(gw, rw, rounded(rw, (n + 4) * U * mw, gw.dtype), label + " grad_weight")
        close(gb, rb, rounded(rb, (n + 1) * U * mb, gb.dtype), label + " grad_bias")


# ---- clipping ----

def check_clip(norm, out, grads, max_norm, label=""):
    total = sum(float(g.to(F64).square().sum()) for g in grads)
    ref = torch.tensor(total, dtype=F64).sqrt()
    # squares and sums in binary64, one rounding to 32 bits
    close(norm.cpu(), ref, rounded(ref, ref * 2.0 ** -40, torch.float32), label + " norm")
    factor = min(1.0, max_norm / (float(ref) + 1e-6)) if total == total else float("nan")
    for i, (g, o) in enumerate(zip(grads, out)):
        r = g.to(F64) * factor
        close(o, r, rounded(r, r.abs() * 2 * U, o.dtype), f"{label} tensor {i}")
