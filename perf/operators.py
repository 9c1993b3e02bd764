"""What is timed of the encoder operators: token embedding and its gradient,
layer norm and its gradient, and clipping by the global gradient norm.

These are the operators that make and train the vectors which the join
compares: rows of a token table, normalised, pooled and joined.  The widths
are those of the join's workloads (16, 32, 64 and 384 dimensions, 20,000 and
1,000,000 rows) and generic ones next to them.

``run`` computes a case in plain torch (``own`` false) or through the
package's entry points (``own`` true); ``exact`` computes it in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS_LN = 1e-5
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one short text looked up on its own, as a query is before it is searched
        dict(name="embed_query", op="embed", batch=1, length=9, vocab=32768, dim=384, table="bf16", act="bf16",
             ids="i64", pad=0.0),
        # a training batch of 128 texts padded to 512 tokens, 32-bit table, 16-bit activations
        dict(name="embed_batch", op="embed", batch=128, length=512, vocab=32768, dim=384, table="f32", act="bf16",
             ids="i64", pad=0.2),
        # the gradient of a handful of short texts with a narrow 32-bit table (the 64-dimension workload)
        dict(name="embed_grad_small", op="embed_grad", batch=16, length=31, vocab=5000, dim=64, table="f32",
             act="f32", ids="i64", pad=0.1),
        # the gradient of the training batch above, 16-bit throughout
        dict(name="embed_grad_batch", op="embed_grad", batch=128, length=512, vocab=32768, dim=384, table="bf16",
             act="bf16", ids="i64", pad=0.2),
        # a million tokens, a large vocabulary and an odd width, gradients kept in 32 bits
        dict(name="embed_grad_large", op="embed_grad", batch=1001, length=999, vocab=250001, dim=385, table="f32",
             act="bf16", ids="i32", pad=0.1),
        # the pooled vectors of a few queries
        dict(name="norm_query", op="norm", rows=33, dim=384, ld=384, act="bf16", param="f32"),
        # one million vectors of 384 dimensions, the embedding workload's size
        dict(name="norm_rows", op="norm", rows=1000000, dim=384, ld=384, act="bf16", param="f32"),
        # a batch of a wide odd model whose rows are part of a larger buffer
        dict(name="norm_odd", op="norm", rows=20000, dim=1001, ld=1100, act="f32", param="f32"),
        # the gradient over a training batch of 64 texts of about 312 tokens
        dict(name="norm_grad_batch", op="norm_grad", rows=20000, dim=384, ld=384, act="f16", param="f32"),
        # the gradient over wide rows
        dict(name="norm_grad_wide", op="norm_grad", rows=32768, dim=4096, ld=4096, act="bf16", param="bf16"),
        # the gradients of a small encoder: a table, a few matrices, many short vectors
        dict(name="clip_model", op="clip", tensors=61, total=21000000, act="bf16", mixed=True, flat=False),
        # a large model's gradients as odd-sized views of one flat buffer
        dict(name="clip_large", op="clip", tensors=301, total=268000000, act="f32", mixed=False, flat=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "norm", "norm_grad", "norm_grad", "clip"])
    act = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op in ("embed", "embed_grad"):
        tokens, dim = _log_int(rng, 1, 1000000), _log_int(rng, 8, 1024)
        tokens = min(tokens, 380000000 // dim)
        length = min(tokens, _log_int(rng, 1, 2048))
        return dict(op=op, batch=max(1, tokens // length), length=length, vocab=_log_int(rng, 64, 250000), dim=dim,
                    table=rng.choice([act, "f32"]), act=act, ids=rng.choice(["i32", "i64"]),
                    pad=rng.choice([0.0, 0.1, 0.3]))
    if op in ("norm", "norm_grad"):
        rows, dim = _log_int(rng, 1, 1000000), _log_int(rng, 8, 8192)
        # a gradient moves three tensors where the forward pass moves two
        rows = min(rows, (250000000 if op == "norm" else 130000000) // dim)
        ld = dim if rng.random() < 0.7 else dim + rng.randrange(1, 129)
        return dict(op=op, rows=max(1, rows), dim=dim, ld=ld, act=act, param=rng.choice([act, "f32"]))
    total = _log_int(rng, 2000, 260000000)
    flat = rng.random() < 0.5
    return dict(op="clip", tensors=min(_log_int(rng, 1, 400 if flat else 60), total // 16), total=total, act=act,
                mixed=not flat and rng.random() < 0.6, flat=flat)


def _token_law(vocab):
    """Probability of each id: a Zipf law as in running text, its ranks spread
    over the ids so that frequent tokens do not sit next to each other."""
    p = 1.0 / (np.arange(vocab, dtype=np.float64) + 3.0)
    p /= p.sum()
    step = max(1, int(vocab * 0.6180339887))
    while math.gcd(step, vocab) != 1:
        step += 1
    out = np.empty(vocab)
    out[(np.arange(vocab) * step) % vocab] = p
    return out


def _tokens(case, gen):
    """[batch, length] ids; the last id of the vocabulary fills each text's
    tail, about the case's ``pad`` share of all places."""
    vocab = case["vocab"]
    cdf = torch.from_numpy(np.cumsum(_token_law(vocab))).to(DEV)
    u = torch.rand((case["batch"], case["length"]), generator=gen, device=DEV, dtype=torch.float64)
    ids = torch.searchsorted(cdf, u).clamp_(max=vocab - 1)
    if case["pad"]:
        ids[ids == vocab - 1] = 0
        # texts of lengths spread evenly from (1 - 2 pad) of the longest to the whole
        short = torch.rand((case["batch"], 1), generator=gen, device=DEV) * (2 * case["pad"] * case["length"])
        place = torch.arange(case["length"], device=DEV)[None, :]
        ids[place >= case["length"] - short.long()] = vocab - 1
    return ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)


def _sizes(case):
    """Element counts of the tensors of a set of gradients: one table with about
    a third, matrices in falling sizes, and every third tensor a short vector."""
    n, total = case["tensors"], case["total"]
    if n == 1:
        return [total]
    weight = [0.0] * n
    for i in range(1, n):
        weight[i] = 0.001 if i % 3 == 0 else 1.0 / (1 + i % 7)
    weight[0] = 0.5 * sum(weight)
    unit = total / sum(weight)
    return [max(1, int(w * unit)) for w in weight]


def _randn(shape, gen, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV).mul_(scale).to(dtype)


def _rows(case, gen, scale, offset):
    """Rows of ``dim`` values, ``ld`` apart, with a few channels far larger than
    the rest, as activations have."""
    buf = torch.randn((case["rows"], case["ld"]), generator=gen, device=DEV)
    channel = torch.ones(case["ld"], device=DEV)
    channel[:: max(8, case["ld"] // 6)] = 12.0
    return buf.mul_(channel).mul_(scale).add_(offset).to(DTYPES[case["act"]])[:, :case["dim"]]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, act = case["op"], DTYPES[case["act"]]
    st = {"case": case}
    if own:
        import exact_range_similarity_amd as ersj
        st["ersj"] = ersj
    if op in ("embed", "embed_grad"):
        st["ids"] = _tokens(case, gen)
        st["pad"] = case["vocab"] - 1 if case["pad"] else None
        st["scale"] = math.sqrt(case["dim"])
        if op == "embed":
            st["table"] = _randn((case["vocab"], case["dim"]), gen, DTYPES[case["table"]], 1 / math.sqrt(case["dim"]))
        else:
            st["grad"] = _randn((case["batch"], case["length"], case["dim"]), gen, act, 0.01)
    elif op in ("norm", "norm_grad"):
        st["x"] = _rows(case, gen, 1.5, 0.25)
        par = DTYPES[case["param"]]
        st["weight"] = (1 + 0.1 * torch.randn(case["dim"], generator=gen, device=DEV)).to(par)
        st["bias"] = _randn(case["dim"], gen, par, 0.1)
        if op == "norm_grad":
            st["grad"] = _randn((case["rows"], case["dim"]), gen, act, 0.05)
            # the forward pass's statistics, which training keeps
            x = st["x"].float()
            st["mean"] = x.mean(dim=1)
            st["rstd"] = (x.var(dim=1, unbiased=False) + EPS_LN).rsqrt()
    else:
        sizes = _sizes(case)
        # in a mixed set the long tensors have 16 bits and the short vectors 32
        types = [torch.float32 if case["mixed"] and i % 3 == 0 and i else act for i in range(len(sizes))]
        grads, out = [], []
        if case["flat"]:
            flat = _randn(sum(sizes), gen, act, 0.01)
            whole = torch.empty_like(flat)
            at = 0
            for s in sizes:
                grads.append(flat[at:at + s])
                out.append(whole[at:at + s])
                at += s
            st["result"] = [whole]
        else:
            grads = [_randn(s, gen, t, 0.01) for s, t in zip(sizes, types)]
            out = [torch.empty_like(g) for g in grads]
            st["result"] = out
        # a threshold that the norm passes two times in three
        st["max_norm"] = 0.01 * math.sqrt(sum(sizes)) * (0.5, 0.9, 1.5)[seed % 3]
        st["grads"] = grads
        if own:
            st["set"] = st["ersj"].GradSet(grads, out)
    return st


def _run_own(st):
    ersj, case = st["ersj"], st["case"]
    op = case["op"]
    if op == "embed":
        return ersj.embed(st["table"], st["ids"], scale=st["scale"], padding_idx=st["pad"],
                          dtype=DTYPES[case["act"]])
    if op == "embed_grad":
        return ersj.embed_grad(st["grad"], st["ids"], case["vocab"], scale=st["scale"], padding_idx=st["pad"],
                               dtype=DTYPES[case["table"]])
    if op == "norm":
        return ersj.layer_norm(st["x"], st["weight"], st["bias"], EPS_LN)
    if op == "norm_grad":
        return ersj.layer_norm_grad(st["grad"], st["x"], st["mean"], st["rstd"], st["weight"])
    return [ersj.clip_grads(st["set"], st["max_norm"])] + st["result"]


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    op, act = case["op"], DTYPES[case["act"]]
    if op == "embed":
        out = st["table"][st["ids"]].float() * st["scale"]
        if st["pad"] is not None:
            out = out * (st["ids"] != st["pad"]).unsqueeze(-1)
        return out.to(act)
    if op == "embed_grad":
        ids = st["ids"].reshape(-1)
        grad = st["grad"].reshape(-1, case["dim"]).float()
        if st["pad"] is not None:
            grad = grad * (ids != st["pad"]).unsqueeze(-1)
        out = torch.zeros((case["vocab"], case["dim"]), device=DEV)
        out.index_add_(0, ids, grad)
        return (out * st["scale"]).to(DTYPES[case["table"]])
    if op == "norm":
        x = st["x"].float()
        mean = x.mean(dim=1, keepdim=True)
        c = x - mean
        rstd = ((c * c).mean(dim=1, keepdim=True) + EPS_LN).rsqrt()
        y = c * rstd * st["weight"].float() + st["bias"].float()
        return y.to(act), mean.squeeze(1), rstd.squeeze(1)
    if op == "norm_grad":
        par = DTYPES[case["param"]]
        rstd = st["rstd"][:, None]
        xhat = (st["x"].float() - st["mean"][:, None]) * rstd
        dy = st["grad"].float()
        g = dy * st["weight"].float()
        dx = rstd * (g - g.mean(dim=1, keepdim=True) - xhat * (g * xhat).mean(dim=1, keepdim=True))
        return dx.to(act), (dy * xhat).sum(dim=0).to(par), dy.sum(dim=0).to(par)
    total = torch.stack([g.float().square().sum() for g in st["grads"]]).sum()
    norm = total.sqrt()
    coef = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    out = [(g.float() * coef).to(g.dtype) for g in st["grads"]]
    return [norm] + ([torch.cat(out)] if case["flat"] else out)


def _expected_distinct(case):
    n = max(1, int(case["batch"] * case["length"] * (1 - case["pad"])))
    return float(np.sum(-np.expm1(n * np.log1p(-np.minimum(_token_law(case["vocab"]), 1 - 1e-12)))))


def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}
    op = case["op"]
    if op in ("embed", "embed_grad"):
        tokens, dim = case["batch"] * case["length"], case["dim"]
        ids = tokens * (4 if case["ids"] == "i32" else 8)
        kept = tokens * (1 - case["pad"])  # padded places have no row to read
        if op == "embed":
            moved = _expected_distinct(case) * dim * size[case["table"]] + tokens * dim * size[case["act"]]
        else:
            moved = kept * dim * size[case["act"]] + case["vocab"] * dim * size[case["table"]]
        return {"bytes": int(ids + moved), "flops": int(kept * dim)}
    if op in ("norm", "norm_grad"):
        n, act, par = case["rows"] * case["dim"], size[case["act"]], size[case["param"]]
        if op == "norm":
            return {"bytes": 2 * n * act + 8 * case["rows"] + 2 * case["dim"] * par, "flops": 8 * n}
        return {"bytes": 3 * n * act + 8 * case["rows"] + 3 * case["dim"] * par, "flops": 14 * n}
    sizes = _sizes(case)
    moved = sum(s * (4 if case["mixed"] and i % 3 == 0 and i else size[case["act"]]) for i, s in enumerate(sizes))
    return {"bytes": 2 * moved + 4, "flops": 3 * sum(sizes)}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "embed":
        ids = st["ids"].reshape(-1).long()
        out = torch.index_select(st["table"].to(f64), 0, ids)
        out *= st["scale"]
        if st["pad"] is not None:
            out[ids == st["pad"]] = 0
        return out.reshape(case["batch"], case["length"], case["dim"])
    if op == "embed_grad":
        # the tokens in the order of their ids, each id's run of rows added up
        ids = st["ids"].reshape(-1).long().cpu().numpy()
        grad = st["grad"].reshape(-1, case["dim"])
        order = np.argsort(ids, kind="stable")
        if st["pad"] is not None:
            order = order[ids[order] != st["pad"]]
        out = np.zeros((case["vocab"], case["dim"]))
        if len(order):
            runs = ids[order]
            first = np.flatnonzero(np.r_[True, runs[1:] != runs[:-1]])
            at = torch.from_numpy(order).to(DEV)
            for c in range(0, case["dim"], 64):
                part = grad[:, c:c + 64].index_select(0, at).to(f64).cpu().numpy()
                out[runs[first], c:c + 64] = np.add.reduceat(part, first, axis=0)
        return torch.from_numpy(out * st["scale"])
    if op in ("norm", "norm_grad"):
        step = max(1, 50000000 // case["dim"])
        w, b = st["weight"].to(f64), st["bias"].to(f64)
        parts, dw, db = [], torch.zeros_like(w), torch.zeros_like(w)
        for r in range(0, case["rows"], step):
            x = st["x"][r:r + step].to(f64)
            mean = x.sum(dim=1, keepdim=True) / case["dim"]
            var = (x - mean).pow(2).sum(dim=1, keepdim=True) / case["dim"]
            std = (var + EPS_LN).sqrt()
            n = (x - mean) / std
            if op == "norm":
                parts.append((torch.addcmul(b, n, w), mean[:, 0], 1 / std[:, 0]))
                continue
            dy = st["grad"][r:r + step].to(f64)
            dw += (dy * n).sum(dim=0)
            db += dy.sum(dim=0)
            h = dy * w
            # the part of h orthogonal to the constant row and to n
            h = h - h.sum(dim=1, keepdim=True) / case["dim"]
            parts.append((h - n * ((h * n).sum(dim=1, keepdim=True) / case["dim"])) / std)
        if op == "norm":
            return tuple(torch.cat([p[i] for p in parts]) for i in range(3))
        return torch.cat(parts), dw, db
    square = 0.0
    for g in st["grads"]:
        for c in range(0, g.numel(), 1 << 26):
            square += float(torch.linalg.vector_norm(g[c:c + (1 << 26)].to(f64))) ** 2
    norm = math.sqrt(square)
    coef = min(1.0, st["max_norm"] / (norm + 1e-6))
    out = [g.to(f64) * coef for g in st["grads"]]
    return [torch.tensor(norm, dtype=f64)] + ([torch.cat(out)] if case["flat"] else out)
