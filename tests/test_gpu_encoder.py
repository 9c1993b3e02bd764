"""The encoder operators against their plain 64-bit forms (encoder_util.py,
which also derives the bounds): token embedding and its gradient, layer norm
and its gradient, clipping by the global gradient norm."""
import gc

import pytest
import torch

import exact_range_similarity_amd as ersj
from encoder_util import (F64, TYPES, U, check_clip, check_embed, check_embed_grad, check_norm, check_norm_grad,
                          close, embed_grad_ref, norm_grad_ref, norm_ref, rounded)
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAIRS = [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ersj.lib()


@pytest.fixture(autouse=True)
def _case(request):
    say(f"[encoder] {request.node.name}")


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(shape, g, dtype="f32", scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale + shift).to(TYPES[dtype])


def spread(t, ld, lead=0):
    """The same rows ``ld`` elements apart, starting ``lead`` elements into a
    buffer whose other elements are NaN."""
    n, d = t.shape
    buf = torch.full((n * ld + lead + ld,), float("nan"), dtype=t.dtype, device=t.device)
    view = buf[lead:lead + n * ld].view(n, ld)[:, :d] if n else buf[:0].view(0, ld)[:, :d]
    view.copy_(t)
    return view


def zipf(n, rows, g):
    u = torch.rand(n, generator=g, device=DEV)
    return (torch.exp(u * torch.log(torch.tensor(float(rows), device=DEV))).long() - 1).clamp(0, rows - 1)


# ---- embedding ----

@pytest.mark.parametrize("table,out", PAIRS)
@pytest.mark.parametrize("n,rows,dim", [(1, 1, 1), (3, 7, 5), (64, 5, 8), (257, 100, 16), (33, 11, 384),
                                        (70, 9, 385), (5, 3, 1000), (2, 4, 8193), (1500, 4000, 18), (0, 4, 8)])
def test_embed(table, out, n, rows, dim):
    g = gen(n * 7 + dim)
    w = randn((rows, dim), g, table)
    for id_type in (torch.int64, torch.int32):
        ids = torch.randint(0, rows, (n,), generator=g, device=DEV).to(id_type)
        got = ersj.embed(w, ids, scale=dim ** 0.5, dtype=TYPES[out])
        check_embed(got, w, ids, dim ** 0.5, None, f"n={n} dim={dim}")


@pytest.mark.parametrize("table,out", PAIRS)
def test_embed_padding_and_bad_ids(table, out):
    g = gen(3)
    w = randn((10, 21), g, table)
    ids = torch.tensor([[0, 9, 4, 4], [-1, 10, 4, 3], [2 ** 40, -2 ** 40, 4, 2 ** 31]], device=DEV)
    check_embed(ersj.embed(w, ids, 2.0, 4, TYPES[out]), w, ids, 2.0, 4)
    # the padding id may lie outside the table
    ids = torch.tensor([3, 10, 2, 11, -1], device=DEV, dtype=torch.int32)
    check_embed(ersj.embed(w, ids, 2.0, 10, TYPES[out]), w, ids, 2.0, 10)
    check_embed(ersj.embed(w, ids, 1.0, None, TYPES[out]), w, ids, 1.0, None)


@pytest.mark.parametrize("table,out", PAIRS)
@pytest.mark.parametrize("dim,ldw,leadw,ldo,leado", [(16, 16, 1, 17, 3), (385, 400, 5, 386, 1), (64, 65, 0, 64, 1),
                                                     (7, 9, 2, 8, 0)])
def test_embed_spacing(table, out, dim, ldw, leadw, ldo, leado):
    g = gen(dim)
    w = spread(randn((50, dim), g, table), ldw, leadw)
    ids = torch.randint(0, 50, (130,), generator=g, device=DEV)
    buf = torch.full((130 * ldo + leado + ldo,), 7.0, dtype=TYPES[out], device=DEV)
    view = buf[leado:leado + 130 * ldo].view(130, ldo)[:, :dim]
    check_embed(ersj.embed(w, ids, 3.0, 2, TYPES[out], out=view), w, ids, 3.0, 2)
    view.fill_(7.0)
    assert bool((buf == 7.0).all()), "wrote outside the rows"
    # ids with a spacing of their own
    ids = torch.randint(0, 50, (20, 6), generator=g, device=DEV)[:, ::2]
    check_embed(ersj.embed(w, ids, 3.0, 2, TYPES[out]), w, ids, 3.0, 2)


def test_embed_special_values():
    w = torch.tensor([[float("inf"), 1.0, float("nan")], [-0.0, 1e-42, 3e38]], device=DEV)
    ids = torch.tensor([1, 0, 1], device=DEV)
    check_embed(ersj.embed(w, ids, 2.0), w, ids, 2.0, None)
    half = torch.tensor([[60000.0, 1e-7]], device=DEV).half()
    got = ersj.embed(half, ids * 0, 2.0)
    assert bool(torch.isinf(got[:, 0]).all())  # beyond the type's range


# ---- the table's gradient ----

@pytest.mark.parametrize("act,table", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"),
                                       ("bf16", "f32")])
@pytest.mark.parametrize("n,rows,dim", [(1, 1, 1), (1, 300, 33), (5, 3, 8), (63, 1000, 16), (257, 2, 18),
                                        (4096, 50, 32), (4097, 5000, 64), (12289, 300, 385), (2000, 70000, 24),
                                        (30000, 1, 20), (9000, 600, 1), (700, 513, 2048), (100, 12, 8193)])
def test_embed_grad(act, table, n, rows, dim):
    g = gen(n + rows)
    grad = randn((n, dim), g, act)
    ids = zipf(n, rows, g).to(torch.int32 if n % 2 else torch.int64)
    got = ersj.embed_grad(grad, ids, rows, 1.5, None, TYPES[table])
    check_embed_grad(got, grad, ids, rows, 1.5, None, label=f"n={n} rows={rows} dim={dim}")
    again = ersj.embed_grad(grad, ids, rows, 1.5, None, TYPES[table])
    assert torch.equal(got, again), "another order of the sums on a second call"


@pytest.mark.parametrize("kind", ["none", "all_padding", "all_bad", "one_id", "last_row", "first_row", "mixed",
                                  "descending", "ascending"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_embed_grad_id_patterns(kind, act):
    g = gen(17)
    n, rows, dim, pad = 9001, 4100, 48, 77
    if kind == "none":
        n = 0
    grad = randn((n, dim), g, act)
    ids = torch.randint(0, rows, (n,), generator=g, device=DEV)
    if kind == "all_padding":
        ids[:] = pad
        grad[:] = float("nan")  # padded places may hold anything
    elif kind == "all_bad":
        ids = torch.where(ids % 2 == 0, ids + rows, -1 - ids)
        grad[:] = float("inf")
    elif kind == "one_id":
        ids[:] = 4000
    elif kind == "last_row":
        ids[:] = rows - 1
    elif kind == "first_row":
        ids[:] = 0
    elif kind == "mixed":
        ids[::3] = pad
        ids[1::7] = 12
        ids[5::11] = -4
        grad[ids == pad] = float("nan")
        grad[ids == -4] = float("nan")
    elif kind == "descending":
        ids = torch.arange(n, 0, -1, device=DEV) % rows
    elif kind == "ascending":
        ids = torch.arange(n, device=DEV) * rows // n
    got = ersj.embed_grad(grad, ids, rows, 0.5, pad)
    check_embed_grad(got, grad, ids, rows, 0.5, pad, label=kind)


@pytest.mark.parametrize("act,table", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
def test_embed_grad_accumulate(act, table):
    g = gen(5)
    n, rows, dim = 5000, 900, 100
    grad = randn((n, dim), g, act)
    ids = zipf(n, rows // 2, g)
    out = randn((rows, dim), g, table)
    before = out.clone()
    got = ersj.embed_grad(grad, ids, rows, 2.0, 3, out=out, accumulate=True)
    assert got.data_ptr() == out.data_ptr()
    check_embed_grad(out, grad, ids, rows, 2.0, 3, before=before)
    untouched = embed_grad_ref(grad, ids, rows, 2.0, 3)[2] == 0
    assert torch.equal(out[untouched], before[untouched])


@pytest.mark.parametrize("act,table", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("dim,ldg,leadg,ldo,leado", [(16, 17, 1, 16, 3), (385, 386, 3, 400, 1), (64, 72, 8, 65, 0)])
def test_embed_grad_spacing(act, table, dim, ldg, leadg, ldo, leado):
    g = gen(dim)
    n, rows = 700, 90
    grad = spread(randn((n, dim), g, act), ldg, leadg)
    ids = zipf(n, rows, g)
    buf = torch.full((rows * ldo + leado + ldo,), 7.0, dtype=TYPES[table], device=DEV)
    view = buf[leado:leado + rows * ldo].view(rows, ldo)[:, :dim]
    ersj.embed_grad(grad, ids, rows, 1.0, None, out=view)
    check_embed_grad(view, grad, ids, rows, 1.0, None)
    view.fill_(7.0)
    assert bool((buf == 7.0).all()), "wrote outside the rows"


def test_embed_grad_special_values():
    # an infinity or NaN stays in its own row
    grad = torch.ones((300, 40), device=DEV)
    ids = torch.arange(300, device=DEV) % 30
    grad[31, 5], grad[61, 5] = float("inf"), float("-inf")
    grad[62, 7] = float("nan")
    grad[33, 8] = float("inf")
    check_embed_grad(ersj.embed_grad(grad, ids, 30), grad, ids, 30, 1.0, None)


# ---- layer norm ----

NORM_SIZES = [(1, 1), (3, 2), (5, 7), (130, 8), (64, 16), (1000, 18), (77, 32), (65, 64), (40, 100), (33, 384), (9, 385),
              (17, 1001), (6, 2048), (5, 2049), (3, 4096), (2, 8200), (1, 33000), (2, 65536), (0, 16), (5000, 24)]


def norm_inputs(n, dim, act, param, affine, seed):
    g = gen(seed)
    x = randn((n, dim), g, act, 2.0, 0.5)
    w = randn(dim, g, param, 0.3, 1.0) if affine else None
    b = randn(dim, g, param, 0.3) if affine else None
    return x, w, b, randn((n, dim), g, act)


@pytest.mark.parametrize("act,param", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"),
                                       ("bf16", "f32")])
@pytest.mark.parametrize("n,dim", NORM_SIZES)
def test_layer_norm(act, param, n, dim):
    for affine in (True, False):
        x, w, b, _ = norm_inputs(n, dim, act, param, affine, n + dim)
        check_norm(ersj.layer_norm(x, w, b, 1e-5), x, w, b, 1e-5, f"n={n} dim={dim} affine={affine}")


@pytest.mark.parametrize("act,param", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"),
                                       ("bf16", "f32")])
@pytest.mark.parametrize("n,dim", NORM_SIZES)
def test_layer_norm_grad(act, param, n, dim):
    for affine in (True, False):
        x, w, b, dy = norm_inputs(n, dim, act, param, affine, n + dim)
        mean, rstd = ersj.layer_norm(x, w, b)[1:]
        dtype = None if affine else TYPES[param]
        got = ersj.layer_norm_grad(dy, x, mean, rstd, w, dtype)
        check_norm_grad(got, dy, x, mean, rstd, w, f"n={n} dim={dim} affine={affine}")
        again = ersj.layer_norm_grad(dy, x, mean, rstd, w, dtype)
        for a, b2 in zip(got, again):
            assert torch.equal(a, b2), "another order of the sums on a second call"
        only_x = ersj.layer_norm_grad(dy, x, mean, rstd, w, dtype, want_params=False)
        assert only_x[1] is None and only_x[2] is None and torch.equal(only_x[0], got[0])
        only_p = ersj.layer_norm_grad(dy, x, mean, rstd, w, dtype, want_x=False)
        assert only_p[0] is None and torch.equal(only_p[1], got[1]) and torch.equal(only_p[2], got[2])


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("n,dim", [(40000, 16), (20011, 384), (3000, 2051), (1025, 5000), (70001, 33)])
def test_layer_norm_many_rows(act, n, dim):
    x, w, b, dy = norm_inputs(n, dim, act, "f32", True, dim)
    got = ersj.layer_norm(x, w, b)
    check_norm(got, x, w, b, 1e-5)
    check_norm_grad(ersj.layer_norm_grad(dy, x, got[1], got[2], w), dy, x, got[1], got[2], w)


@pytest.mark.parametrize("act,param", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("n,dim,ld,lead", [(100, 16, 17, 1), (33, 385, 400, 3), (20, 1001, 1100, 0), (7, 4099, 4101, 5),
                                           (50, 64, 64, 1)])
def test_layer_norm_spacing(act, param, n, dim, ld, lead):
    x, w, b, dy = norm_inputs(n, dim, act, param, True, ld)
    x, dy = spread(x, ld, lead), spread(dy, ld + 2, lead + 1)
    buf = torch.full((n * ld + lead + ld,), 7.0, dtype=x.dtype, device=DEV)
    view = buf[lead:lead + n * ld].view(n, ld)[:, :dim]
    got = ersj.layer_norm(x, w, b, out=view)
    check_norm(got, x, w, b, 1e-5)
    check_norm_grad(ersj.layer_norm_grad(dy, x, got[1], got[2], w), dy, x, got[1], got[2], w)
    view.fill_(7.0)
    assert bool((buf == 7.0).all()), "wrote outside the rows"


def test_layer_norm_in_place_and_shapes():
    x, w, b, _ = norm_inputs(60, 48, "bf16", "f32", True, 1)
    copy = x.clone()
    got = ersj.layer_norm(copy, w, b, out=copy)
    assert got[0].data_ptr() == copy.data_ptr()
    check_norm(got, x, w, b, 1e-5)
    y, mean, rstd = ersj.layer_norm(x.view(3, 4, 5, 48), w, b)
    assert y.shape == (3, 4, 5, 48) and mean.shape == rstd.shape == (3, 4, 5)
    assert torch.equal(y.view(60, 48), got[0])
    y, mean, rstd = ersj.layer_norm(x[0], w, b)
    assert y.shape == (48,) and mean.shape == () and torch.equal(y, got[0][0])


@pytest.mark.parametrize("dim", [40, 3000])
def test_layer_norm_grad_in_place(dim):
    # through the C ABI, the gradient of x may replace either input
    x, w, _, dy = norm_inputs(90, dim, "f32", "f32", True, 4)
    _, mean, rstd = ersj.layer_norm(x, w)
    want = ersj.layer_norm_grad(dy, x, mean, rstd, w)
    L = ersj.lib()
    for which in (0, 1):
        a = [dy.clone(), x.clone()]
        gw, gb = torch.empty_like(w), torch.empty_like(w)
        need = L.ersj_layer_norm_grad_work(90, dim)
        work = torch.empty(need, dtype=torch.uint8, device=DEV)
        rc = L.ersj_layer_norm_grad(a[0].data_ptr(), dim, a[1].data_ptr(), dim, 0, 90, dim, mean.data_ptr(),
                                    rstd.data_ptr(), w.data_ptr(), 0, a[which].data_ptr(), dim, gw.data_ptr(),
                                    gb.data_ptr(), work.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert rc == ersj.OK
        assert torch.equal(a[which], want[0]) and torch.equal(gw, want[1]) and torch.equal(gb, want[2])


@pytest.mark.parametrize("dim", [5, 384, 3001])
def test_layer_norm_special_rows(dim):
    g = gen(dim)
    x = randn((12, dim), g)
    x[0] = 3.0                   # no variance: y is the bias
    x[1] = 0.0
    x[2, 0] = float("nan")
    x[3, dim - 1] = float("inf")
    x[4] = 1e-30                 # the variance vanishes beside eps
    x[5] += 5000.0               # a mean far above the deviation
    w, b = randn(dim, g), randn(dim, g)
    got = ersj.layer_norm(x, w, b)
    keep = [0, 1, 4, 5, 6, 7, 8, 9, 10, 11]
    check_norm([t[keep] for t in got], x[keep], w, b, 1e-5)
    assert bool(torch.isnan(got[0][2]).all()) and bool(torch.isnan(got[0][3]).all())
    assert torch.equal(got[0][1], b)
    dy = randn((12, dim), g)
    gx = ersj.layer_norm_grad(dy, x, got[1], got[2], w, want_params=False)[0]
    check_norm_grad((gx[keep], None, None), dy[keep], x[keep], got[1][keep], got[2][keep], w)


# ---- gradients against differences ----

def test_layer_norm_grad_against_differences():
    g = gen(11)
    n, dim, eps, h = 4, 37, 1e-5, 1e-5
    x, w, b, dy = randn((n, dim), g), randn(dim, g), randn(dim, g), randn((n, dim), g)
    _, mean, rstd = ersj.layer_norm(x, w, b, eps)
    gx, gw, gb = ersj.layer_norm_grad(dy, x, mean, rstd, w)

    def loss(x, w, b):
        return (norm_ref(x, w, b, eps)[0] * dy.to(F64)).sum()

    args = [x.to(F64), w.to(F64), b.to(F64)]
    for which, got in ((0, gx), (1, gw), (2, gb)):
        diff = torch.empty_like(args[which])
        for k in range(diff.numel()):
            step = torch.zeros_like(diff)
            step.view(-1)[k] = h
            up, down = list(args), list(args)
            up[which], down[which] = args[which] + step, args[which] - step
            diff.view(-1)[k] = (loss(*up) - loss(*down)) / (2 * h)
        # differences: h^2 of third derivatives and rounding over h, both near
        # 1e-9 here; the kernel: about dim roundings of terms near 3
        assert float((got.to(F64) - diff).abs().max()) < 40 * dim * U, which


def test_embed_grad_against_differences():
    # the loss is linear in the table, so a difference of any step is exact
    g = gen(12)
    rows, dim = 6, 5
    w, ids = randn((rows, dim), g), torch.tensor([[1, 4, 1], [5, 2, 1]], device=DEV)
    dy = randn((2, 3, dim), g)
    got = ersj.embed_grad(dy, ids, rows, 3.0, 2)
    for k in range(rows * dim):
        step = torch.zeros((rows, dim), device=DEV)
        step.view(-1)[k] = 1.0
        up = ersj.embed(w + step, ids, 3.0, 2).to(F64) * dy.to(F64)
        down = ersj.embed(w - step, ids, 3.0, 2).to(F64) * dy.to(F64)
        # values below 16, a few roundings each
        assert abs(float((up - down).sum() / 2) - float(got.view(-1)[k])) < 16 * 30 * U


def test_autograd():
    g = gen(13)
    rows, dim = 50, 24
    w0, gamma0, beta0 = randn((rows, dim), g), randn(dim, g), randn(dim, g)
    ids = torch.randint(0, rows, (7, 9), generator=g, device=DEV)
    target = randn((7, 9, dim), g)

    w, gamma, beta = (t.clone().requires_grad_() for t in (w0, gamma0, beta0))
    e = ersj.embed(w, ids, 4.0, 3)
    y, mean, rstd = ersj.layer_norm(e, gamma, beta)
    assert not mean.requires_grad and not rstd.requires_grad
    (y * target).sum().backward()

    # the same in 64 bits on the CPU
    v, gam, bet = (t.cpu().to(F64).requires_grad_() for t in (w0, gamma0, beta0))
    keep = (ids != 3).cpu().unsqueeze(-1)
    (norm_ref((v[ids.cpu()] * 4.0 * keep), gam, bet, 1e-5)[0] * target.cpu().to(F64)).sum().backward()
    # sums of at most 63 terms, each with about 2 dim roundings; a padded row's
    # gradient of x is amplified by rstd = 1 / sqrt(eps) and belongs to no token
    for got, ref in ((w.grad, v.grad), (gamma.grad, gam.grad), (beta.grad, bet.grad)):
        scale = float(ref.abs().max())
        assert float((got.cpu().to(F64) - ref).abs().max()) < scale * 63 * 2 * dim * U

    # a broadcast gradient, and a part of the graph alone
    gamma2 = gamma0.clone().requires_grad_()
    ersj.layer_norm(e.detach(), gamma2, None)[0].sum().backward()
    assert gamma2.grad.shape == (dim,)
    w2 = w0.clone().requires_grad_()
    ersj.embed(w2, ids, 4.0, 3).sum().backward()
    count = torch.bincount(ids.view(-1), minlength=rows).to(F64)
    count[3] = 0
    assert torch.equal(w2.grad.to(F64), (4.0 * count)[:, None].expand(rows, dim))
    with pytest.raises(ValueError):
        ersj.embed(w2, ids, out=torch.empty((7, 9, dim), device=DEV))


# ---- clipping ----

def grads_of(sizes, g, types=("f32",), scale=0.1):
    return [randn(s, g, types[i % len(types)], scale) for i, s in enumerate(sizes)]


@pytest.mark.parametrize("types", [("f32",), ("bf16",), ("f16",), ("bf16", "f32", "f16")])
@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [3, 1, 7, 2], [(33, 77), 5, (3, 3, 3), 0], [8191, 8192, 8193],
                                   [16383, 16384, 16385, 1], [1000003], [17] * 301, [300000, 1, 4, 70001]])
@pytest.mark.parametrize("share", [0.3, 2.0])
def test_clip(types, sizes, share):
    g = gen(len(sizes))
    grads = grads_of(sizes, g, types)
    total = sum(t.numel() for t in grads)
    max_norm = share * 0.1 * total ** 0.5
    before = [t.clone() for t in grads]
    out = [torch.full_like(t, 7.0) for t in grads]
    gs = ersj.GradSet(grads, out)
    norm = ersj.clip_grads(gs, max_norm)
    assert norm.shape == () and norm.dtype == torch.float32
    check_clip(norm, out, before, max_norm)
    for a, b in zip(grads, before):
        assert torch.equal(a, b), "an input changed"
    # new values in the same tensors, and a second call's bits
    for t in grads:
        t.mul_(-0.5)
    n2 = ersj.clip_grads(gs, max_norm)
    check_clip(n2, out, [t.clone() for t in grads], max_norm)
    first = [o.clone() for o in out]
    n3 = ersj.clip_grads(gs, max_norm)
    assert torch.equal(n2, n3) and all(torch.equal(a, b) for a, b in zip(first, out))
    # in place
    norm = ersj.clip_grads(grads, max_norm)
    check_clip(norm, grads, [t * -0.5 for t in before], max_norm)


def test_clip_views_of_a_flat_buffer():
    g = gen(2)
    for dtype in ("f32", "bf16"):
        sizes = [1, 3, 1000, 7, 20001, 2, 5]
        flat = randn(sum(sizes) + 2, g, dtype)
        whole = flat.clone()
        views, at = [], 1
        for s in sizes:
            views.append(flat[at:at + s])
            at += s
        norm = ersj.clip_grads(views, 3.0)
        check_clip(norm, [flat[1:-1]], [whole[1:-1]], 3.0)
        assert torch.equal(flat[0], whole[0]) and torch.equal(flat[-1], whole[-1])


def test_clip_special_values():
    def one(values, max_norm):
        t = torch.tensor(values, device=DEV)
        o = torch.empty_like(t)
        n = ersj.clip_grads(ersj.GradSet([t], [o]), max_norm)
        return float(n), o.tolist()

    assert one([0.0, 0.0], 1.0) == (0.0, [0.0, 0.0])
    assert one([3.0, 4.0], float("inf")) == (5.0, [3.0, 4.0])
    assert one([3.0, 4.0], 0.0) == (5.0, [0.0, 0.0])
    # squares beyond and below the range of 32 bits
    n, o = one([3e30, 4e30], 5.0)
    assert abs(n / 5e30 - 1) < 1e-6 and abs(o[0] - 3) < 1e-5 and abs(o[1] - 4) < 1e-5
    n, o = one([3e-30, 4e-30], 1.0)
    assert abs(n / 5e-30 - 1) < 1e-6
    n, o = one([1.0, float("inf")], 1.0)
    assert n == float("inf") and o[0] == 0.0 and o[1] != o[1]
    n, o = one([1.0, float("nan")], 1.0)
    assert n != n and o[0] != o[0]


def test_clip_refuses():
    t = torch.zeros(8, 8, device=DEV)
    with pytest.raises(ValueError):
        ersj.GradSet([t.t()[:3]])
    with pytest.raises(ValueError):
        ersj.GradSet([t], [t[:4]])
    with pytest.raises(ValueError):
        ersj.GradSet([t], [])
    with pytest.raises(TypeError):
        ersj.GradSet([t.double()])
    with pytest.raises(ersj.ErsjError):
        ersj.clip_grads([t], -1.0)


def test_refusals():
    w = torch.zeros((6, 8), device=DEV)
    ids = torch.zeros(3, dtype=torch.int64, device=DEV)
    for call in (lambda: ersj.embed(w, ids.float()), lambda: ersj.embed(w, ids, dtype=torch.float64),
                 lambda: ersj.embed(w.to(torch.int32), ids), lambda: ersj.layer_norm(w.half(), w[0].bfloat16()),
                 lambda: ersj.layer_norm(w, w[0], w[0].half())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: ersj.embed(w[0], ids), lambda: ersj.embed(w.t(), ids), lambda: ersj.embed(w, ids.cpu()),
                 lambda: ersj.embed(w, ids, padding_idx=-1), lambda: ersj.embed(w, ids, out=w),
                 lambda: ersj.embed_grad(w, ids, 6), lambda: ersj.embed_grad(w[:3], ids, 6, accumulate=True),
                 lambda: ersj.embed_grad(w[:3], ids, 6, out=w[:5]), lambda: ersj.layer_norm(w.t()),
                 lambda: ersj.layer_norm(w, w[0, :4]), lambda: ersj.layer_norm(w, w[:, :1].expand(6, 8)[0]),
                 lambda: ersj.layer_norm(w[:1].expand(6, 8)), lambda: ersj.layer_norm(w, out=w[:3]),
                 lambda: ersj.layer_norm_grad(w[:3], w, w[:, 0], w[:, 0]),
                 lambda: ersj.layer_norm_grad(w, w, w[:, 0], w[:, 0])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ersj.embed(w.half(), ids, dtype=torch.float32), lambda: ersj.layer_norm(w, eps=-1.0),
                 lambda: ersj.embed_grad(w[:3], ids, 6, dtype=torch.float16),
                 lambda: ersj.embed_grad(w[:3], ids, 0)):
        with pytest.raises(ersj.ErsjError):
            call()


# ---- streams, graphs, long tensors ----

def test_side_stream():
    g = gen(21)
    side = torch.cuda.Stream()
    for k in range(3):
        w, ids = randn((2000, 64), g), torch.randint(0, 2000, (4000,), generator=g, device=DEV)
        dy = randn((4000, 64), g)
        side.wait_stream(torch.cuda.current_stream())
        stream = side if k < 2 else side.cuda_stream
        e = ersj.embed(w, ids, 2.0, stream=stream)
        y, mean, rstd = ersj.layer_norm(e, stream=stream)
        gx, gw, gb = ersj.layer_norm_grad(dy, e, mean, rstd, stream=stream)
        table = ersj.embed_grad(gx, ids, 2000, 2.0, stream=stream)
        clipped = torch.empty_like(table)
        gs = ersj.GradSet([table], [clipped], stream=stream)
        norm = ersj.clip_grads(gs, 1.0, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        check_embed(e, w, ids, 2.0, None)
        check_norm((y, mean, rstd), e, None, None, 1e-5)
        check_norm_grad((gx, gw, gb), dy, e, mean, rstd, None)
        check_embed_grad(table, gx, ids, 2000, 2.0, None)
        check_clip(norm, [clipped], [table], 1.0)
        torch.cuda.synchronize()


def test_graph_replay():
    g = gen(22)
    n, rows, dim = 6000, 3000, 96
    w, gamma, beta = randn((rows, dim), g), randn(dim, g), randn(dim, g)
    ids = torch.randint(0, rows, (n,), generator=g, device=DEV)
    dy = randn((n, dim), g)
    table = torch.empty_like(w)
    out = [torch.empty_like(table), torch.empty_like(gamma)]
    gw = torch.empty_like(gamma)
    gs = ersj.GradSet([table, gw], out)

    def step():
        e = ersj.embed(w, ids, 3.0, 5)
        y, mean, rstd = ersj.layer_norm(e, gamma, beta)
        gx, gg, gb = ersj.layer_norm_grad(dy, e, mean, rstd, gamma)
        gw.copy_(gg)
        ersj.embed_grad(gx, ids, rows, 3.0, 5, out=table)
        return [y, gx, gb, ersj.clip_grads(gs, 2.0), *out]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        ids.copy_(zipf(n, rows, g))
        dy.copy_(randn((n, dim), g))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        junk = randn((500, 500), g)
        (junk @ junk).sum().item()
        want = [t.clone() for t in step()]
        for a, b in zip(got, want):
            assert torch.equal(a, b), f"replay {k} differs from the eager step"


def test_offsets_beyond_32_bits():
    g = gen(31)
    dim = 384
    n = 2 ** 31 // dim + 1003  # rows whose elements pass 2^31
    x = torch.empty((n, dim), dtype=torch.bfloat16, device=DEV)
    for r in range(0, n, 1 << 20):
        x[r:r + (1 << 20)] = randn((min(1 << 20, n - r), dim), g, "bf16")
    w = randn(dim, g)
    y, mean, rstd = ersj.layer_norm(x, w)
    for part in (slice(0, 500), slice(n - 1500, n)):
        check_norm((y[part], mean[part], rstd[part]), x[part], w, None, 1e-5)
    gx, gw, gb = ersj.layer_norm_grad(y, x, mean, rstd, w)
    rw = torch.zeros(dim, dtype=F64, device=DEV)
    mw = torch.zeros(dim, dtype=F64, device=DEV)
    for r in range(0, n, 1 << 19):
        part = slice(r, min(n, r + (1 << 19)))
        ref, _, a, m, _, _ = norm_grad_ref(y[part], x[part], mean[part], rstd[part], w)
        rw += a
        mw += m
        if r == 0 or part.stop == n:
            check_norm_grad((gx[part], None, None), y[part], x[part], mean[part], rstd[part], w)
        del ref
    # n roundings bound the error; sums in groups stay within thousands
    assert bool(((gw.to(F64) - rw).abs() <= 20000 * U * mw).all())
    del y, gx, mean, rstd
    gc.collect()
    # a table that long, and its gradient
    ids = torch.randint(0, n, (4000,), generator=g, device=DEV)
    ids[:3] = torch.tensor([n - 1, 0, n - 2], device=DEV)
    check_embed(ersj.embed(x, ids, 2.0), x, ids, 2.0, None)
    grad = x[:4000]
    big = ersj.embed_grad(grad, ids, n, 1.0)
    hit = torch.unique(ids)
    where = torch.searchsorted(hit, ids)
    check_embed_grad(big[hit], grad, where, len(hit), 1.0, None)
    assert int((big != 0).any(dim=1).sum()) == len(hit)
    del big
    # as many tokens
    ids = torch.randint(0, 1000, (n,), generator=g, device=DEV)
    check_embed_grad(ersj.embed_grad(x, ids, 1000, 1.0, 3, torch.float32), x, ids, 1000, 1.0, 3)
    e = ersj.embed(x[:1000], ids)
    for part in (slice(0, 500), slice(n - 500, n)):
        check_embed(e[part], x[:1000], ids[part], 1.0, None)
    del e
    last = x[-1000:].clone()
    total = sum(float(x[r:r + (1 << 20)].to(F64).square().sum()) for r in range(0, n, 1 << 20)) ** 0.5
    norm = ersj.clip_grads([x], 10.0)
    assert abs(float(norm) / total - 1) <= 2 * U
    ref = last.to(F64) * (10.0 / (total + 1e-6))
    close(x[-1000:], ref, rounded(ref, ref.abs() * 2 * U, x.dtype))


# ---- sizes at which the kernels change their plan ----

@pytest.mark.parametrize("n,rows,dim", [(1024, 40, 16), (1025, 40, 16), (1024, 70000, 9), (1025, 70001, 9), (4096, 511, 8),
                                        (4097, 511, 8), (4097, 512, 8), (5000, 262143, 4), (5000, 262144, 4),
                                        (65536, 1000, 8), (65537, 1000, 8), (131072, 300, 5), (131073, 300, 5),
                                        (270000, 5000, 3), (5000, 1023, 8), (5000, 1024, 8), (300000, 1023, 3),
                                        (5000, 1048575, 3), (5000, 1048576, 3), (70000, 1048576, 2), (6000, 2, 33), (300, 100000, 520), (2000, 20, 1030), (1500, 20, 65535), (40, 7, 65536)])
@pytest.mark.parametrize("act,table", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_embed_grad_plans(act, table, n, rows, dim):
    g = gen(n + dim)
    grad = randn((n, dim), g, act)
    ids = zipf(n, rows, g)
    ids[::17] = rows - 1
    check_embed_grad(ersj.embed_grad(grad, ids, rows, 1.0, 1, TYPES[table]), grad, ids, rows, 1.0, 1)
    out = randn((rows, dim), g, table)
    before = out.clone()
    ersj.embed_grad(grad, ids, rows, 1.0, 1, out=out, accumulate=True)
    check_embed_grad(out, grad, ids, rows, 1.0, 1, before=before)


@pytest.mark.parametrize("n", [200, 1000, 3000, 20000, 200000])
def test_embed_grad_long_rows(n):
    # few ids, each of them long: rows cut over many shares, and neighbours of long rows
    g = gen(n)
    rows, dim = 400, 40
    grad = randn((n, dim), g, "bf16")
    for ids in (torch.randint(0, 3, (n,), generator=g, device=DEV) * 199,
                torch.where(torch.rand(n, generator=g, device=DEV) < 0.9, 7,
                            torch.randint(0, rows, (n,), generator=g, device=DEV)),
                torch.arange(n, device=DEV) * 40 // n + 5):
        got = ersj.embed_grad(grad, ids, rows, 1.0, None, torch.float32)
        check_embed_grad(got, grad, ids, rows, 1.0, None)
        assert torch.equal(got, ersj.embed_grad(grad, ids, rows, 1.0, None, torch.float32))


@pytest.mark.parametrize("act", ["f32", "f16"])
@pytest.mark.parametrize("dim", [3, 4, 15, 16, 17, 31, 33, 63, 65, 127, 129, 255, 256, 257, 511, 513, 1023, 1024, 1025, 2047,
                                 4095, 4097, 8191, 8193, 16384, 16385, 32769])
def test_layer_norm_plans(act, dim):
    x, w, b, dy = norm_inputs(19, dim, act, "f32", True, dim)
    got = ersj.layer_norm(x, w, b)
    check_norm(got, x, w, b, 1e-5)
    check_norm_grad(ersj.layer_norm_grad(dy, x, got[1], got[2], w), dy, x, got[1], got[2], w)


@pytest.mark.parametrize("n,dim", [(5000, 6), (3000, 1028), (40000, 40), (50, 65535)])
def test_embed_many_rows(n, dim):
    g = gen(n)
    w = randn((n // 3, dim), g)
    ids = torch.randint(0, n // 3, (n,), generator=g, device=DEV)
    check_embed(ersj.embed(w, ids, 1.5, 7, torch.bfloat16), w, ids, 1.5, 7)


@pytest.mark.parametrize("dim", [3, 7, 100, 384, 1001, 6000])
def test_layer_norm_constant_rows(dim):
    # integers whose sums are exact: the mean is exact, so y is the bias itself
    x = torch.tensor([[3.0], [-7.0], [1000.0], [0.0]], device=DEV).expand(4, dim).contiguous()
    b = randn(dim, gen(dim))
    y, mean, rstd = ersj.layer_norm(x, None, b, 1e-5)
    assert mean.tolist() == [3.0, -7.0, 1000.0, 0.0]
    assert torch.equal(y, b.expand(4, dim))
