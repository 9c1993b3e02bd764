"""Plain 64-bit forms of the gated block and of rows held in 8 bits, with bounds
on the error of the kernels' arithmetic, shared by their tests.

A matrix instruction adds 16 products and its accumulator, each of the 17 terms
through at most 16 additions of error below 2u, so one instruction is off by
less than 32.1u of its terms' magnitudes, and a sum over k of k / 16
instructions by (k / 16) * 36u of the sum of all magnitudes (second-order terms
included).  32-bit values are multiplied as three bf16 parts: bf16 rounding is
off by at most 2^-8, so the second part is at most 2^-8 and the third 2^-16 of
the value, and 3 * 8 bits hold all 24.  Six of the nine products of parts are
summed; the others, two of order 2^-24 and one of 2^-32, are dropped.
"""
import math

import torch

from encoder_util import F64, U, close, rounded, tiny, unit

ACTIVATIONS = ["silu", "gelu", "gelu_tanh"]
KAPPA = math.sqrt(2 / math.pi)


def act_ref(g, act, dtype=torch.float32):
    """act(g), act'(g) and a bound on the 32-bit evaluation of each at an exact g.

    exp by the hardware's exponential of a rounded product: relative error at
    most (|argument| + 4) u; the rest a few roundings.  The product with g and
    the sums in the derivative carry it on."""
    if act == "silu":
        s = torch.sigmoid(g)
        rel = (g.abs() + 10) * U
        return g * s, s + g * s * (1 - s), (g * s).abs() * rel, s * rel * (2 + g.abs())
    if act == "gelu":
        phi = 0.5 * torch.erfc(-g / math.sqrt(2))
        dens = torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
        # the distribution as half of 1 + erf: off by some u at most, however small it is; for 16
        # bits its upper tail by exp and a polynomial, fitted to 1.4e-6 of the tail
        tail = torch.minimum(phi, 1 - phi) * (0.0 if dtype == torch.float32 else 1.4e-6 + (g * g + 10) * U)
        return (g * phi, phi + g * dens, g.abs() * (6 * U + tail),
                6 * U + tail + g.abs() * dens * (g * g + 10) * U)
    z = KAPPA * (g + 0.044715 * g ** 3)
    s = torch.sigmoid(2 * z)
    rel = (2 * z.abs() * 6 + 10) * U  # the argument itself is off by a few u
    inner = 2 * KAPPA * (1 + 3 * 0.044715 * g * g)
    return (g * s, s + g * s * (1 - s) * inner, (g * s).abs() * rel,
            s * rel + (g * s * inner).abs() * rel * (1 - s + U) + (g * s * inner).abs() * U)


def products(dtype, held=False):
    return 1 if dtype != torch.float32 else 3 if held else 6


def sum_error(k, dtype, magnitudes, held=False):
    """Bound on a sum over k of products by matrix instructions."""
    k = -(-k // 16) * 16
    split = 2 * 2.0 ** -24 + 2.0 ** -32 if dtype == torch.float32 else 0.0
    return magnitudes * (k / 16 * 36 * U * products(dtype, held) + split)


def forward(x, w_gate, w_up, act, held=False):
    """g, u, their error bounds, and the activation's terms."""
    a, wg, wu = x.to(F64), w_gate.to(F64), w_up.to(F64)
    k = x.shape[-1]
    g, u = a @ wg.t(), a @ wu.t()
    eg = sum_error(k, x.dtype, a.abs() @ wg.abs().t(), held)
    eu = sum_error(k, x.dtype, a.abs() @ wu.abs().t(), held)
    return g, u, eg, eu, act_ref(g, act, x.dtype)


def check_gated(got, x, w_gate, w_up, act, label=""):
    x = x.reshape(-1, x.shape[-1])
    got = got.reshape(-1, got.shape[-1])
    g, u, eg, eu, (value, _, ev, _) = forward(x, w_gate, w_up, act)
    ref = value * u
    ea = 1.2 * eg + ev * 1.01  # the activations' slopes are below 1.2
    close(got, ref, rounded(ref, ea * u.abs() + value.abs() * eu + ea * eu + 2 * U * ref.abs(), got.dtype), label)


def gated_grad_ref(grad, x, w_gate, w_up, act, held=False):
    """The three gradients and their bounds."""
    dtype = x.dtype
    x, grad = x.reshape(-1, x.shape[-1]), grad.reshape(-1, grad.shape[-1])
    g, u, eg, eu, (value, slope, ev, es) = forward(x, w_gate, w_up, act, held)
    a, dh, wg, wu = x.to(F64), grad.to(F64), w_gate.to(F64), w_up.to(F64)
    dg, du = dh * u * slope, dh * value
    # the slopes' slopes are below 1.2 as well
    edg = dh.abs() * (eu * slope.abs() + (u.abs() + eu) * (1.2 * eg + es)) + 3 * U * dg.abs()
    edu = dh.abs() * (1.2 * eg + ev) + 2 * U * du.abs()
    # rounded to the type multiplied; three bf16 parts hold 32 bits whole
    part = 0.0 if dtype == torch.float32 else unit(dtype)
    edg = edg * (1 + part) + part * dg.abs() + tiny(dtype)
    edu = edu * (1 + part) + part * du.abs() + tiny(dtype)
    n, hidden = grad.shape
    gx = dg @ wg + du @ wu
    ex = (edg @ wg.abs() + edu @ wu.abs()
          + sum_error(2 * (hidden + 15), dtype, (dg.abs() + edg) @ wg.abs() + (du.abs() + edu) @ wu.abs()) + 4 * U * gx.abs())
    out = [(gx, ex)]
    for d, e in ((dg, edg), (du, edu)):
        ref = d.t() @ a
        mag = (d.abs() + e).t() @ a.abs()
        # parts of the sum are added up at the end
        out.append((ref, e.t() @ a.abs() + sum_error(n, dtype, mag, held) + 520 * U * mag))
    return out


def check_gated_grad(got, grad, x, w_gate, w_up, act, held=False, label=""):
    for name, t, (ref, err) in zip(("x", "gate", "up"), got, gated_grad_ref(grad, x, w_gate, w_up, act, held)):
        if t is None:
            continue
        t = t.reshape(ref.shape)
        close(t, ref, rounded(ref, err, t.dtype), f"{label} grad of {name}")
        # as a whole: what is multiplied and the result are rounded, each by at most a unit of the value
        if ref.numel() >= 4096 and t.dtype != torch.float32:
            off = float((t.to(F64) - ref).norm() / ref.norm())
            assert off <= 3 * unit(t.dtype), f"{label} grad of {name}: off by {off:.3g} of its norm"


def held_ref(x):
    """(codes, scale bytes, values) of rows held in 8 bits."""
    dim = x.shape[-1]
    v = x.reshape(-1, dim).to(F64)
    n, blocks = v.shape[0], -(-dim // 32)
    wide = torch.zeros((n, blocks * 32), dtype=F64, device=x.device)
    wide[:, :dim] = v
    wide = wide.view(n, blocks, 32)
    most = wide.abs().amax(dim=2)
    bad = ~torch.isfinite(wide).all(dim=2)
    at, e = torch.frexp(torch.where(bad, torch.ones_like(most), most) / 127)
    # (zero has no exponent of its own: the least)
    e = torch.where(at == 0, torch.full_like(e, -126), torch.where(at == 0.5, e - 1, e)).clamp(min=-126).to(torch.int64)
    top = 10 if x.dtype == torch.float16 else 122
    lim = torch.where(e == top, 63.0, 127.0).to(F64).unsqueeze(-1)
    step = ((e + 1023) << 52).view(F64).unsqueeze(-1)
    code = torch.round(wide / step)
    code = torch.maximum(torch.minimum(code, lim), -lim)
    code = torch.where(bad.unsqueeze(-1), torch.zeros_like(code), code)
    value = code * step + 0.0
    value = torch.where(bad.unsqueeze(-1), torch.full_like(value, float("nan")), value)
    cut = lambda t: t.reshape(n, blocks * 32)[:, :dim].reshape(x.shape)  # noqa: E731
    scales = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return cut(code).to(torch.int8), scales.view(x.shape[:-1] + (blocks,)), cut(value)
