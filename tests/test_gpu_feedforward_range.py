"""The gated block's gradient of f16 tensors over the range of the type: gradients
whose terms are subnormal or beyond the largest f16 number, though the sums over
rows or columns are neither.

dg and du are held as f16 multiplied by a power of two F with F B >= 2^14, B the
largest of max|grad_h| |x| over the rows times the largest |w| of the weights: off
by at most 2^-11 of the value, and 2^-25 / F <= 2^-39 B below f16's normal range.
"""
import pytest
import torch

import exact_range_similarity_amd as ersj
from encoder_util import F64, U, close, rounded, tiny, unit
from feedforward_util import forward, sum_error
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16 = torch.float16
INF, NAN = float("inf"), float("nan")
# dg and du in two parts of f16, in one, and in one with tiles of 256
SIZES = [(4096, 64, 160), (9000, 200, 331), (4200, 4104, 2100)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ersj.lib()


@pytest.fixture(autouse=True)
def _case(request):
    say(f"[feedforward] {request.node.name}")


def randn(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).mul_(scale)


def block(n, dim, hidden, seed, x=1.0, w=1.0, grad=0.1):
    return (randn((n, dim), seed, x).to(F16), randn((hidden, dim), seed + 1, w * dim ** -0.5).to(F16),
            randn((hidden, dim), seed + 2, w * dim ** -0.5).to(F16), randn((n, hidden), seed + 3, grad).to(F16))


def check(got, grad, x, w_gate, w_up, act, rows=slice(None), held=False, label=""):
    """``rows``: those that are compared of the gradient of x."""
    a, dh, wg, wu = (t.to(F64) for t in (x, grad, w_gate, w_up))
    g, u, eg, eu, (value, slope, ev, es) = forward(x, w_gate, w_up, act, held)
    dg, du = dh * u * slope, dh * value
    edg = dh.abs() * (eu * slope.abs() + (u.abs() + eu) * (1.2 * eg + es)) + 3 * U * dg.abs()
    edu = dh.abs() * (1.2 * eg + ev) + 2 * U * du.abs()
    finite = lambda t: torch.where(torch.isfinite(t), t, torch.zeros_like(t))  # noqa: E731
    most = finite(finite(dh).abs().amax(dim=1) * a.norm(dim=1)).max() * finite(torch.cat([wg, wu]).norm(dim=1)).max()
    part, low = unit(F16), float(most) * 2.0 ** -39 * 1.01
    edg, edu = (e * (1 + part) + part * d.abs() + low for e, d in ((edg, dg), (edu, du)))
    n, hidden = grad.shape
    mag = (dg.abs() + edg) @ wg.abs() + (du.abs() + edu) @ wu.abs()
    want = [(dg @ wg + du @ wu, edg @ wg.abs() + edu @ wu.abs() + sum_error(2 * (hidden + 15), F16, mag))]
    for d, e in ((dg, edg), (du, edu)):
        mag = (d.abs() + e).t() @ a.abs()
        want.append((d.t() @ a, e.t() @ a.abs() + sum_error(n, F16, mag, held) + 520 * U * mag))
    for k, (name, t, (ref, err)) in enumerate(zip(("x", "gate", "up"), got, want)):
        if t is None:
            continue
        if k == 0:
            t, ref, err = t[rows], ref[rows], err[rows]
        err = err + 4 * U * ref.abs()
        close(t, ref, rounded(ref, err, F16), f"{label} grad of {name}")
        # what is multiplied and the result are rounded, each by at most a unit of the value, or by half
        # the least step of the result's type
        over = ref.abs() > torch.finfo(F16).max
        t, ref = t.to(F64).masked_fill(over, 0), ref.masked_fill(over, 0)
        off, size = float((t - ref).norm()), float(ref.norm())
        assert off <= 3 * unit(F16) * size + tiny(F16) * ref.numel() ** 0.5, f"{label} grad of {name}: off by {off / size:.3g} of its norm"


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("n,dim,hidden", SIZES)
@pytest.mark.parametrize("grad", [2.0 ** -17, 2.0 ** -20, 2.0 ** -23])
def test_small_gradients(grad, n, dim, hidden, act):
    # the weights' gradients are normal numbers, their terms are not
    x, wg, wu, dh = block(n, dim, hidden, 1, x=64.0, w=2.0 ** -6, grad=grad)
    check(ersj.gated_grad(dh, x, wg, wu, act), dh, x, wg, wu, act)


@pytest.mark.parametrize("n,dim,hidden", [(1, 64, 96), (50, 64, 96), (9000, 200, 331)])
def test_terms_beyond_the_type_give_finite_rows(n, dim, hidden):
    # u about 30, dg to 3e5 and more; small weights bring dx back
    x, wg, wu, dh = block(n, dim, hidden, 2, x=400.0, w=0.08, grad=3000.0)
    got = ersj.gated_grad(dh, x, wg, wu, "silu", True, False, False)
    assert bool(torch.isfinite(got[0]).all())
    assert float((dh.to(F64) * (x.to(F64) @ wu.to(F64).t())).abs().max()) > 1e5
    check(got, dh, x, wg, wu, "silu")


@pytest.mark.parametrize("n,dim,hidden", [(1, 64, 96), (50, 64, 96), (9000, 200, 331)])
def test_terms_beyond_the_type_give_finite_weights(n, dim, hidden):
    # the same with small rows and large weights: dW is within the type, or, over 9000 rows
    # (3000 * 30 * 0.7 * 0.004 * sqrt(9000) = 2.4e4 and up to 4.5 times that), nearly everywhere
    x, wg, wu, dh = block(n, dim, hidden, 3, x=0.004, w=8000.0, grad=3000.0)
    got = ersj.gated_grad(dh, x, wg, wu, "gelu", False, True, True)
    assert float((dh.to(F64) * (x.to(F64) @ wu.to(F64).t())).abs().max()) > 1e5
    assert all(float(torch.isfinite(t).float().mean()) > 0.9 for t in got[1:])
    check(got, dh, x, wg, wu, "gelu")


@pytest.mark.parametrize("n,dim,hidden", SIZES[:2])
def test_rows_of_unlike_size(n, dim, hidden):
    x, wg, wu, dh = block(n, dim, hidden, 4)
    dh = (dh.float() * torch.exp2(torch.randint(-14, 12, (n, 1), device=DEV, generator=torch.Generator(DEV).manual_seed(5)))).to(F16)
    check(ersj.gated_grad(dh, x, wg, wu, "silu"), dh, x, wg, wu, "silu")
    kept = ersj.pack_rows(x)
    values = ersj.unpack_rows(kept)
    check(ersj.gated_grad(dh, kept, wg, wu, "silu"), dh, values, wg, wu, "silu", held=True)


@pytest.mark.parametrize("hidden", [1, 7, 511, 513, 1100])
def test_layouts_of_small_gradients(hidden):
    # spaced rows off 16 bytes, with NaN beside them
    x, wg, wu, dh = block(3000, 40, hidden, 6, x=64.0, w=2.0 ** -6, grad=2.0 ** -20)
    wide = torch.full((3002, hidden + 9), NAN, device=DEV, dtype=F16)
    wide[1:-1, 5:5 + hidden] = dh
    check(ersj.gated_grad(wide[1:-1, 5:5 + hidden], x, wg, wu, "silu"), dh, x, wg, wu, "silu")


def test_values_that_are_not_finite_do_not_set_the_factor():
    x, wg, wu, dh = block(3000, 40, 96, 7, x=64.0, w=2.0 ** -6, grad=2.0 ** -20)
    x[5, 3], x[2999, 39], dh[17, 0], dh[18, 95] = INF, NAN, INF, NAN
    rest = torch.ones(3000, dtype=torch.bool, device=DEV)
    rest[[5, 17, 18, 2999]] = False
    got = ersj.gated_grad(dh, x, wg, wu, "silu", True, False, False)
    assert not bool(torch.isfinite(got[0][~rest]).any())
    keep = lambda t: t[rest].contiguous()  # noqa: E731
    check((keep(got[0]), None, None), keep(dh), keep(x), wg, wu, "silu")
    # a weight that is not finite leaves the other one's gradient right
    bad = wu.clone()
    bad[95, 0] = INF
    got = ersj.gated_grad(keep(dh), keep(x), wg, bad, "silu", False, False, True)
    check((None, None, got[2]), keep(dh), keep(x), wg, wu, "silu")


def test_no_gradient_at_all():
    x, wg, wu, dh = block(300, 40, 96, 8)
    for zero in ((dh * 0, x, wg, wu), (dh, x * 0, wg, wu), (dh, x, wg * 0, wu * 0)):
        for t, ref in zip(ersj.gated_grad(*zero, "silu"), ersj.gated_grad(*(z.float() for z in zero), "silu")):
            assert torch.equal(t, ref.to(F16))


def test_a_captured_call_follows_its_gradients():
    x, wg, wu, dh = block(3000, 64, 160, 9, x=64.0, w=2.0 ** -6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ersj.gated_grad(dh, x, wg, wu)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ersj.gated_grad(dh, x, wg, wu)
    for turn, scale in enumerate((2.0 ** -20, 1.0, 2.0 ** -23, 2.0 ** -4)):
        dh.copy_(randn((3000, 160), 20 + turn, scale))
        want = ersj.gated_grad(dh, x, wg, wu)
        torch.cuda.synchronize()
        for t in out:
            t.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
        check((None, *out[1:]), dh, x, wg, wu, "silu")
