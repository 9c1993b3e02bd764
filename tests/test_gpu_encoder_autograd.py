"""The encoder operators inside autograd: streams, saved tensors, tensors that
the operators write."""
import pytest
import torch

import exact_range_similarity_amd as ersj
from exact_range_similarity_amd import encoder
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"


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


def step_inputs(n, rows, dim, seed):
    g = gen(seed)
    table = torch.randn((rows, dim), generator=g, device=DEV)
    gamma = 1 + 0.1 * torch.randn(dim, generator=g, device=DEV)
    beta = torch.randn(dim, generator=g, device=DEV)
    ids = torch.randint(0, rows, (n,), generator=g, device=DEV)
    dy = torch.randn((n, dim), generator=g, device=DEV)
    return table, gamma, beta, ids, dy


def direct(table, gamma, beta, ids, dy):
    """The same gradients by the direct calls, whose bits are always the same."""
    e = ersj.embed(table, ids, 2.0)
    _, mean, rstd = ersj.layer_norm(e, gamma, beta)
    gx, gw, gb = ersj.layer_norm_grad(dy, e, mean, rstd, gamma)
    return ersj.embed_grad(gx, ids, len(table), 2.0), gw, gb


@pytest.mark.parametrize("raw", [False, True])
def test_backward_runs_on_the_given_stream(raw, monkeypatch):
    side, streams = torch.cuda.Stream(), []

    def noting(call):
        def noted(*args, **kw):
            streams.append(torch.cuda.current_stream().cuda_stream)
            return call(*args, **kw)
        return noted

    monkeypatch.setattr(encoder, "layer_norm_grad", noting(encoder.layer_norm_grad))
    monkeypatch.setattr(encoder, "embed_grad", noting(encoder.embed_grad))
    table, gamma, beta, ids, dy = step_inputs(3000, 500, 64, 1)
    want = direct(table, gamma, beta, ids, dy)
    params = [t.clone().requires_grad_() for t in (table, gamma, beta)]
    side.wait_stream(torch.cuda.current_stream())
    given = side.cuda_stream if raw else side
    # the statistics are dropped here, so that only the node holds them
    y = ersj.layer_norm(ersj.embed(params[0], ids, 2.0, stream=given), *params[1:], stream=given)[0]
    torch.cuda.current_stream().wait_stream(side)
    streams.clear()
    torch.cuda._sleep(500000)  # the gradient of y comes late
    y.backward(dy * 1.0)
    # whatever the backward pass released is handed out on the stream again
    with torch.cuda.stream(side):
        junk = [torch.full((size,), float("nan"), device=DEV) for size in (3000, 3000 * 64, 3000, 64) for _ in range(20)]
    torch.cuda.synchronize()
    assert streams == [side.cuda_stream] * 2
    for p, ref in zip(params, want):
        assert torch.equal(p.grad, ref)
    del junk


def test_backward_of_steps_in_a_row_on_a_stream():
    side = torch.cuda.Stream()
    table, gamma, beta, _, _ = step_inputs(10, 500, 64, 2)
    params = [t.clone().requires_grad_() for t in (table, gamma, beta)]
    total = [torch.zeros_like(t) for t in params]
    steps = [step_inputs(2000 + 100 * k, 500, 64, 3 + k)[3:] for k in range(6)]
    for ids, dy in steps:
        for t, part in zip(total, direct(table, gamma, beta, ids, dy)):
            t += part
    side.wait_stream(torch.cuda.current_stream())
    for ids, dy in steps:
        y = ersj.layer_norm(ersj.embed(params[0], ids, 2.0, stream=side), *params[1:], stream=side)[0]
        torch.cuda.current_stream().wait_stream(side)
        (y * dy).sum().backward()
    torch.cuda.synchronize()
    for p, ref in zip(params, total):
        assert torch.equal(p.grad, ref)


# ---- tensors that the operators write ----

def saved_then(write, t):
    """The backward pass of a product that saved ``t``, which ``write`` overwrites."""
    w = torch.ones(t.shape, device=DEV, dtype=t.dtype, requires_grad=True)
    z = (w * t).sum()
    write()
    z.backward()


def writes(g):
    """Each call that writes a tensor of the caller's, as (name, tensor, call)."""
    x = torch.randn((40, 24), generator=g, device=DEV)
    ids = torch.randint(0, 40, (40,), generator=g, device=DEV)
    a, b, c, d, e, f = (torch.randn((40, 24), generator=g, device=DEV) for _ in range(6))
    kept, target = ersj.GradSet([x, e]), ersj.GradSet([x], [f])
    return [("embed", a, lambda: ersj.embed(x, ids, out=a)),
            ("embed_grad", b, lambda: ersj.embed_grad(x, ids, 40, out=b)),
            ("embed_grad accumulate", b, lambda: ersj.embed_grad(x, ids, 40, out=b, accumulate=True)),
            ("layer_norm", c, lambda: ersj.layer_norm(c, out=c)),
            ("layer_norm other", d, lambda: ersj.layer_norm(x, out=d)),
            ("clip_grads kept", e, lambda: ersj.clip_grads(kept, 1.0)),
            ("clip_grads into others", f, lambda: ersj.clip_grads(target, 1.0)),
            ("clip_grads", d, lambda: ersj.clip_grads([a, d], 1.0)),
            ("clip_grads flat", d, lambda: ersj.clip_grads([d.view(-1)[5:17]], 1.0))]


def test_autograd_sees_what_is_written():
    side = torch.cuda.Stream()
    for name, t, call in writes(gen(5)):
        before = t._version
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved_then(call, t)
        assert t._version > before, name
        torch.cuda.synchronize()
    x, out = torch.randn((2, 40, 24), generator=gen(6), device=DEV)
    before = out._version
    ersj.layer_norm(x, out=out, stream=side)
    torch.cuda.synchronize()
    assert out._version > before
    # inputs keep their versions
    before = x._version
    ersj.layer_norm_grad(x, x, *ersj.layer_norm(x)[1:])
    assert x._version == before


def test_an_output_that_requires_a_gradient_is_refused():
    x = torch.randn((40, 24), generator=gen(7), device=DEV)
    ids = torch.zeros(40, dtype=torch.int64, device=DEV)
    out = torch.zeros((40, 24), device=DEV, requires_grad=True)
    for target in (out, out * 1.0):
        for call in (lambda: ersj.embed(x, ids, out=target), lambda: ersj.layer_norm(x, out=target),
                     lambda: ersj.embed_grad(x, ids, 40, out=target),
                     lambda: ersj.embed_grad(x, ids, 40, out=target, accumulate=True)):
            with pytest.raises(ValueError, match="gradient"):
                call()
            with torch.no_grad():  # as torch's own calls with out do
                call()
    with torch.inference_mode():
        y = torch.zeros((40, 24), device=DEV)
        ersj.layer_norm(x, out=y)
    assert torch.equal(y, ersj.layer_norm(x)[0])


# ---- forward mode ----

def test_forward_tangents_are_refused():
    # there is no forward-mode rule: a tangent must not be dropped in silence
    fwd = torch.autograd.forward_ad
    g = gen(8)
    x, t = torch.randn((2, 40, 24), generator=g, device=DEV)
    v, tv = torch.randn((2, 24), generator=g, device=DEV)
    ids = torch.randint(0, 40, (40,), generator=g, device=DEV)
    mean, rstd = ersj.layer_norm(x)[1:]
    with fwd.dual_level():
        dx, dv = fwd.make_dual(x, t), fwd.make_dual(v, tv)
        for call in (lambda: ersj.embed(dx, ids), lambda: ersj.layer_norm(dx), lambda: ersj.layer_norm(x, dv),
                     lambda: ersj.layer_norm(x, None, dv), lambda: ersj.embed_grad(dx, ids, 40),
                     lambda: ersj.layer_norm_grad(dx, x, mean, rstd), lambda: ersj.layer_norm_grad(x, dx, mean, rstd),
                     lambda: ersj.clip_grads([x * 1, dx], 1.0)):
            with pytest.raises(NotImplementedError):
                call()
            with torch.no_grad(), pytest.raises(NotImplementedError):
                call()
        w = x.clone().requires_grad_()
        with pytest.raises(NotImplementedError):
            ersj.embed(fwd.make_dual(w, t), ids)
        # tensors without a tangent are as ever
        assert torch.equal(ersj.embed(x, ids), x[ids])
        ersj.embed(w, ids).backward(x)
        assert torch.equal(w.grad, ersj.embed_grad(x, ids, 40))


def test_backward_of_a_part_of_a_wider_tensor():
    # the gradients arrive as spaced rows, of y and of the embedding
    table, gamma, beta, ids, dy = step_inputs(3000, 500, 64, 9)
    more = torch.randn((3000, 37), generator=gen(10), device=DEV)
    params = [t.clone().requires_grad_() for t in (table, gamma, beta)]
    e = ersj.embed(params[0], ids, 2.0)
    y = ersj.layer_norm(e, *params[1:])[0]
    torch.cat([more, y], dim=1).backward(torch.cat([more, dy], dim=1))
    for p, ref in zip(params, direct(table, gamma, beta, ids, dy)):
        assert torch.equal(p.grad, ref)
    t = table.clone().requires_grad_()
    torch.cat([more, ersj.embed(t, ids, 2.0)], dim=1).backward(torch.cat([more, dy], dim=1))
    assert torch.equal(t.grad, ersj.embed_grad(dy, ids, 500, 2.0))
