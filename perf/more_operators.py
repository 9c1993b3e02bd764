"""What is timed of the feed-forward operators: the gated feed-forward block and
its gradient, rows held in 8 bits for a backward pass, and the gradients of
the block and of layer norm from such rows.

The encoder that makes the vectors of the join looks tokens up, normalises
them and, where it is more than a table, passes them through feed-forward
blocks.  The widths are those of the join's workloads (64 and 384 dimensions,
a million rows) and generic ones next to them.

``run`` computes a case in plain torch (``own`` false) or through the
package's entry points (``own`` true); ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS_LN = 1e-5
BLOCK = 32  # neighbours along a row that share a scale
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one query of nine tokens through a small encoder's block
        dict(name="gated_query", op="gated", rows=9, dim=384, hidden=1024, act="gelu", type="bf16", pad=0),
        # a single token through a wide block, where the weights' reading counts
        dict(name="gated_token", op="gated", rows=1, dim=4096, hidden=11008, act="silu", type="bf16", pad=0),
        # a batch of 128 texts of 512 tokens through the small encoder's block
        dict(name="gated_batch", op="gated", rows=65536, dim=384, hidden=1024, act="gelu", type="bf16", pad=0),
        # odd widths and spaced rows in 32 bits
        dict(name="gated_odd", op="gated", rows=1999, dim=385, hidden=1001, act="silu", type="f32", pad=11),
        # a prompt batch through a wide block
        dict(name="gated_wide", op="gated", rows=8192, dim=4096, hidden=11008, act="silu", type="bf16", pad=0),
        # the gradients of a handful of short texts, narrow and in 32 bits
        dict(name="gated_grad_small", op="gated_grad", rows=496, dim=64, hidden=171, act="gelu_tanh", type="f32", pad=0),
        # the gradients of a training batch of 64 texts of about 312 tokens
        dict(name="gated_grad_batch", op="gated_grad", rows=20000, dim=384, hidden=1024, act="gelu", type="f16", pad=0),
        # the gradients of a wide block
        dict(name="gated_grad_wide", op="gated_grad", rows=8192, dim=4096, hidden=11008, act="silu", type="bf16", pad=0),
        # a training step of the small encoder's block that keeps its input in 8 bits
        dict(name="gated_step", op="gated_step", rows=65536, dim=384, hidden=1024, act="gelu", type="bf16", pad=0),
        # a million vectors to 8 bits and back
        dict(name="pack_rows", op="pack", rows=1000000, dim=384, type="bf16", pad=0),
        # a training step of layer norm over a million rows that keeps its input in 8 bits
        dict(name="norm_step", op="norm_step", rows=1000000, dim=384, type="bf16", pad=0),
        # the same for a small batch of an odd width whose rows are part of a larger buffer
        dict(name="norm_step_odd", op="norm_step", rows=1500, dim=1001, type="f32", pad=99),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_grad", "gated_grad", "gated_step", "pack", "norm_step"])
    kind = rng.choice(["f32", "f16", "bf16", "bf16"])
    pad = 0 if rng.random() < 0.6 else rng.randrange(1, 65)
    if op in ("pack", "norm_step"):
        rows, dim = _log_int(rng, 1, 1000000), _log_int(rng, 8, 8192)
        most = 380000000 if kind != "f32" else 190000000
        return dict(op=op, rows=max(1, min(rows, most // (dim + pad))), dim=dim, type=kind, pad=pad)
    dim, hidden = _log_int(rng, 16, 4096), _log_int(rng, 16, 11008)
    if rng.random() < 0.6:  # widths of models are mostly round
        dim, hidden = -(-dim // 16) * 16, -(-hidden // 16) * 16
    rows = _log_int(rng, 1, 65536)
    most = {"gated": 3.6e11, "gated_grad": 3.6e11, "gated_step": 2.4e11}[op]
    if kind == "f32":
        most /= 8
    rows = max(1, min(rows, int(most / (dim * hidden))))
    return dict(op=op, rows=rows, dim=dim, hidden=hidden, act=rng.choice(["silu", "gelu", "gelu_tanh"]), type=kind,
                pad=pad)


def _randn(shape, gen, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV).mul_(scale).to(dtype)


def _rows(case, gen, offset=0.0):
    """Rows of ``dim`` values that lie ``pad`` values apart, with a few channels
    larger than the rest, as activations have."""
    ld = case["dim"] + case["pad"]
    buf = torch.randn((case["rows"], ld), generator=gen, device=DEV)
    channel = torch.ones(ld, device=DEV)
    channel[:: max(8, ld // 6)] = 4.0
    return buf.mul_(channel).add_(offset).to(DTYPES[case["type"]])[:, :case["dim"]]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, kind = case["op"], DTYPES[case["type"]]
    st = {"case": case}
    if own:
        import exact_range_similarity_amd as ersj
        st["ersj"] = ersj
    st["x"] = _rows(case, gen, 0.25 if op == "norm_step" else 0.0)
    if op in ("gated", "gated_grad", "gated_step"):
        shape = (case["hidden"], case["dim"])
        st["gate"] = _randn(shape, gen, kind, 0.7 / math.sqrt(case["dim"]))
        st["up"] = _randn(shape, gen, kind, 0.7 / math.sqrt(case["dim"]))
        if op != "gated":
            st["grad"] = _randn((case["rows"], case["hidden"]), gen, kind, 0.05)
    elif op == "norm_step":
        st["weight"] = 1 + 0.1 * torch.randn(case["dim"], generator=gen, device=DEV)
        st["bias"] = 0.1 * torch.randn(case["dim"], generator=gen, device=DEV)
        st["grad"] = _randn((case["rows"], case["dim"]), gen, kind, 0.05)
    return st


def _run_own(st):
    ersj, case = st["ersj"], st["case"]
    op = case["op"]
    if op == "gated":
        return ersj.gated(st["x"], st["gate"], st["up"], case["act"])
    if op == "gated_grad":
        return ersj.gated_grad(st["grad"], st["x"], st["gate"], st["up"], case["act"])
    if op == "gated_step":
        h = ersj.gated(st["x"], st["gate"], st["up"], case["act"])
        kept = ersj.pack_rows(st["x"])
        return (h,) + ersj.gated_grad(st["grad"], kept, st["gate"], st["up"], case["act"])
    if op == "pack":
        return ersj.unpack_rows(ersj.pack_rows(st["x"]))
    y, mean, rstd, kept = ersj.layer_norm_pack(st["x"], st["weight"], st["bias"], EPS_LN)
    return (y, mean, rstd) + ersj.layer_norm_grad(st["grad"], kept, mean, rstd, st["weight"])


def _held(x):
    """The values that rows held in 8 bits stand for: -127 to 127 times a power of
    two, the least that reaches the largest value of a run of 32."""
    rows, dim = x.shape
    v = torch.zeros((rows, -(-dim // BLOCK) * BLOCK), device=DEV)
    v[:, :dim] = x
    v = v.view(rows, -1, BLOCK)
    part, exponent = torch.frexp(v.abs().amax(dim=2, keepdim=True))
    e = torch.where(part > 127 / 128, exponent - 6, exponent - 7).clamp(min=-126)
    step, inverse = ((e + 127) << 23).view(torch.float32), ((127 - e) << 23).view(torch.float32)
    # 63 where 64 of them would be beyond the largest value of the type
    most = torch.where(e == (10 if x.dtype == torch.float16 else 122), 63.0, 127.0)
    code = torch.minimum(torch.maximum(torch.round(v * inverse), -most), most)
    return (code * step).view(rows, -1)[:, :dim].to(x.dtype)


def _activation(g, act):
    """An activation and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        c = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2 * math.pi))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g)


def _gated_grad(grad, x, gate, up, act):
    x32, wg, wu, dh = x.float(), gate.float(), up.float(), grad.float()
    u = x32 @ wu.t()
    a, da = _activation(x32 @ wg.t(), act)
    dg = dh * u * da
    du = dh * a
    return (dg @ wg + du @ wu).to(x.dtype), (dg.t() @ x32).to(gate.dtype), (du.t() @ x32).to(up.dtype)


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    op, x = case["op"], st["x"]
    if op == "pack":
        return _held(x)
    if op == "norm_step":
        x32 = x.float()
        mean = x32.mean(dim=1, keepdim=True)
        c = x32 - mean
        rstd = ((c * c).mean(dim=1, keepdim=True) + EPS_LN).rsqrt()
        y = (c * rstd * st["weight"] + st["bias"]).to(x.dtype)
        xhat = (_held(x).float() - mean) * rstd
        dy = st["grad"].float()
        g = dy * st["weight"]
        dx = rstd * (g - g.mean(dim=1, keepdim=True) - xhat * (g * xhat).mean(dim=1, keepdim=True))
        return y, mean.squeeze(1), rstd.squeeze(1), dx.to(x.dtype), (dy * xhat).sum(dim=0), dy.sum(dim=0)
    if op == "gated_grad":
        return _gated_grad(st["grad"], x, st["gate"], st["up"], case["act"])
    x32 = x.float()
    h = (_activation(x32 @ st["gate"].float().t(), case["act"])[0] * (x32 @ st["up"].float().t())).to(x.dtype)
    if op == "gated":
        return h
    return (h,) + _gated_grad(st["grad"], _held(x), st["gate"], st["up"], case["act"])


def work(case):
    op, size = case["op"], 4 if case["type"] == "f32" else 2
    n = case["rows"] * case["dim"]
    if op == "pack":
        # each value read and its 8-bit form written, read, and the value written
        return {"bytes": int(2 * n * (size + 1 + 1 / BLOCK)), "flops": 5 * n}
    if op == "norm_step":
        # x in, y out, the 8-bit form out and in, the gradient in and out
        return {"bytes": int(n * (4 * size + 2 * (1 + 1 / BLOCK))) + 16 * case["rows"], "flops": 25 * n}
    hidden = case["hidden"]
    weights, out, product = 2 * hidden * case["dim"], case["rows"] * hidden, 2 * n * hidden
    if op == "gated":
        return {"bytes": size * (n + weights + out), "flops": 2 * product + 6 * out}
    # both projections again, the gradient of x through both, and of both weights
    grad = {"bytes": size * (2 * n + 2 * weights + out), "flops": 6 * product + 20 * out}
    if op == "gated_grad":
        return grad
    return {"bytes": grad["bytes"] + int(2 * n * (1 + 1 / BLOCK)) + size * (weights + out),
            "flops": grad["flops"] + 2 * product + 6 * out + 5 * n}


# ---- the operators' definitions in 64 bits ----

def _held_exact(x):
    out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    for c in range(0, x.shape[1], BLOCK):
        v = x[:, c:c + BLOCK].to(torch.float64)
        # 2^e with the least e for which 127 of them are no less than the largest
        at, e = torch.frexp(torch.linalg.vector_norm(v, ord=float("inf"), dim=1, keepdim=True) / 127)
        e = torch.where(at == 0.5, e - 1, e).clamp(min=-126)
        top = torch.finfo(x.dtype).max
        code = torch.round(torch.ldexp(v, -e))
        code = torch.where(torch.ldexp(code.abs(), e) > top, 63 * code.sign(), code)
        out[:, c:c + BLOCK] = torch.ldexp(code, e)
    return out


def _phi(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return torch.nn.functional.gelu(g, approximate="tanh" if act == "gelu_tanh" else "none")


def _slope(g, act):
    """The derivative of _phi, by torch's differentiation."""
    with torch.enable_grad():
        v = g.detach().requires_grad_()
        return torch.autograd.grad(_phi(v, act).sum(), v)[0]


def exact(case, seed):
    st = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "pack":
        return _held_exact(st["x"])
    if op == "norm_step":
        w, b = st["weight"].to(f64), st["bias"].to(f64)
        step = max(1, 20000000 // case["dim"])
        parts, dw, db = [], torch.zeros_like(w), torch.zeros_like(b)
        for r in range(0, case["rows"], step):
            x = st["x"][r:r + step]
            var, mean = torch.var_mean(x.to(f64), dim=1, correction=0, keepdim=True)
            std = (var + EPS_LN).sqrt()
            y = torch.addcmul(b, (x.to(f64) - mean) / std, w)
            n = (_held_exact(x) - mean) / std
            dy = st["grad"][r:r + step].to(f64)
            dw += (dy * n).sum(dim=0)
            db += dy.sum(dim=0)
            h = dy * w
            h -= h.sum(dim=1, keepdim=True) / case["dim"]
            # n is not quite centred, so its product is taken with the uncentred part as well
            s = (dy * w * n).sum(dim=1, keepdim=True) / case["dim"]
            parts.append((y, mean[:, 0], 1 / std[:, 0], (h - n * s) / std))
        cols = [torch.cat([p[i] for p in parts]) for i in range(4)]
        return (*cols, dw, db)
    gate, up = st["gate"].to(f64), st["up"].to(f64)
    step = max(1, 60000000 // max(case["dim"], case["hidden"]))
    hs, dxs, dgate, dup = [], [], torch.zeros_like(gate), torch.zeros_like(up)
    for r in range(0, case["rows"], step):
        x = st["x"][r:r + step]
        if op != "gated_grad":
            v = x.to(f64)
            hs.append(_phi(torch.matmul(v, gate.T), case["act"]) * torch.matmul(v, up.T))
        if op == "gated":
            continue
        v = _held_exact(x) if op == "gated_step" else x.to(f64)
        g, u, dh = torch.matmul(v, gate.T), torch.matmul(v, up.T), st["grad"][r:r + step].to(f64)
        to_gate = _slope(g, case["act"]) * u * dh
        to_up = _phi(g, case["act"]) * dh
        dxs.append(torch.addmm(torch.matmul(to_up, up), to_gate, gate))
        dgate.addmm_(to_gate.T, v)
        dup.addmm_(to_up.T, v)
    grads = (torch.cat(dxs), dgate, dup) if dxs else ()
    if op == "gated":
        return torch.cat(hs)
    return grads if op == "gated_grad" else (torch.cat(hs),) + grads
