"""32-bit products by three bf16 parts, in every form of tile: as a whole, and by
inputs that show each of the six products exactly.  Rows held in 8 bits at the
same sizes.  (What the bounds notice is checked in test_feedforward_parts.py.)"""
import pytest
import torch

import exact_range_similarity_amd as ersj
from encoder_util import F64, TYPES
from feedforward_parts import EXACT_PAIRS, THREE, one_of_each_row, pattern, whole_bound
from feedforward_util import act_ref, check_gated_grad
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
# the projections in tiles of 64, of 128 with four slabs and with two, and of 256 (128 in the
# gradient); both sums of the gradient in 64, 128 and 256, in one part and in several
SIZES = [(200, 64, 100), (1500, 1100, 700), (9000, 384, 300), (4200, 4104, 2100), (9000, 1300, 3300)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ersj.lib()


@pytest.fixture(autouse=True)
def _case(request):
    say(f"[feedforward] {request.node.name}")


def randn(shape, seed, scale=1.0):
    return torch.randn(shape, generator=torch.Generator(DEV).manual_seed(seed), device=DEV).mul_(scale)


def near(got, ref, bound, label):
    off = float((got.to(F64) - ref).norm() / ref.norm())
    assert off <= bound, f"{label}: off by {off:.3g} of its norm, {bound:.3g} is the bound"


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("n,dim,hidden", SIZES)
def test_whole(n, dim, hidden, held):
    x, wg, wu, dh = randn((n, dim), 1), randn((hidden, dim), 2, dim ** -0.5), randn((hidden, dim), 3, dim ** -0.5), randn((n, hidden), 4)
    rows = x
    if held:
        rows = ersj.pack_rows(x)
        x = ersj.unpack_rows(rows)
    a, g64, u64, d64 = (t.to(F64) for t in (x, wg, wu, dh))
    g, u = a @ g64.t(), a @ u64.t()
    value, slope = act_ref(g, "gelu_tanh")[:2]
    if not held:
        near(ersj.gated(x, wg, wu, "gelu_tanh"), value * u, whole_bound(dim), "h")
    dg, du = d64 * u * slope, d64 * value
    gx, gg, gu = ersj.gated_grad(dh, rows, wg, wu, "gelu_tanh")
    near(gx, dg @ g64 + du @ u64, whole_bound(dim, 2 * hidden), "grad of x")
    near(gg, dg.t() @ a, whole_bound(dim, n), "grad of gate")
    near(gu, du.t() @ a, whole_bound(dim, n), "grad of up")


def same(got, want):
    assert torch.equal(want.float().to(F64), want)  # 32-bit numbers all
    assert torch.equal(got.to(F64), want)


@pytest.mark.parametrize("pair", EXACT_PAIRS)
@pytest.mark.parametrize("n,dim,hidden", SIZES)
def test_forward_exactly(n, dim, hidden, pair):
    # column 0 makes one factor, one value of each row's others the other one; silu(g) = g for g >= 64
    a, b = pair
    x, at = one_of_each_row(n, dim, 1, a, 1, DEV)
    x[:, 0] = 1
    w = pattern((hidden, dim), b, 2, DEV)
    w[:, 0] = 0
    once = torch.zeros_like(w)
    r = torch.arange(n, device=DEV)
    want = x[r, at].to(F64)[:, None] * w[:, at].to(F64).t()
    once[:, 0] = 128
    same(ersj.gated(x, once, w), 128 * want)
    once[:, 0] = 1
    same(ersj.gated(x, 64 * w, once), 64 * want)


@pytest.mark.parametrize("pair", EXACT_PAIRS)
@pytest.mark.parametrize("n,dim,hidden", SIZES)
def test_gradient_of_x_exactly(n, dim, hidden, pair):
    # g = 128 everywhere, so du = 128 grad_h; one value of grad_h in each row
    a, b = pair
    x = torch.zeros((n, dim), device=DEV)
    x[:, 0] = 1
    wg = torch.zeros((hidden, dim), device=DEV)
    wg[:, 0] = 128
    wu = pattern((hidden, dim), b, 3, DEV)
    dh, at = one_of_each_row(n, hidden, 0, a, 4, DEV)
    gx = ersj.gated_grad(dh, x, wg, wu, "silu", True, False, False)[0]
    want = 128 * dh[torch.arange(n, device=DEV), at].to(F64)[:, None] * wu[at].to(F64)
    same(gx[:, 1:], want[:, 1:])
    # through the gate: u = 1 from column 0, dg = grad_h
    wu.zero_()[:, 0] = 1
    wg = pattern((hidden, dim), b, 5, DEV)
    wg[:, 0] = 128
    gx = ersj.gated_grad(dh, x, wg, wu, "silu", True, False, False)[0]
    want = dh[torch.arange(n, device=DEV), at].to(F64)[:, None] * wg[at].to(F64)
    same(gx[:, 1:], want[:, 1:])


# held rows are of one part
@pytest.mark.parametrize("pair,held", [(p, False) for p in EXACT_PAIRS] + [((THREE, 1.0), True)])
@pytest.mark.parametrize("n,dim,hidden", SIZES)
def test_gradient_of_the_weights_exactly(n, dim, hidden, pair, held):
    # g = 128, u = 2; one value of grad_h in each column
    a, b = pair
    x = pattern((n, dim), b, 6, DEV)
    x[:, 0] = 1
    w = torch.zeros((2, hidden, dim), device=DEV)
    w[0, :, 0], w[1, :, 0] = 128, 2
    dh, at = one_of_each_row(hidden, n, 0, a, 7, DEV)
    _, gg, gu = ersj.gated_grad(dh.t().contiguous(), ersj.pack_rows(x) if held else x, w[0], w[1], "silu", False)
    want = dh[torch.arange(hidden, device=DEV), at].to(F64)[:, None] * x[at].to(F64)
    same(gu[:, 1:], 128 * want[:, 1:])
    same(gg[:, 1:], 2 * want[:, 1:])


@pytest.mark.parametrize("pair,held", [(p, False) for p in EXACT_PAIRS] + [((1.0, THREE), True)])
@pytest.mark.parametrize("n,dim,hidden", SIZES)
def test_the_gradients_projections_exactly(n, dim, hidden, pair, held):
    # u = a b from column 1, shown by dWg = grad_h u x with powers of two for the rest
    a, b = pair
    x = pattern((n, dim), 1.0, 8, DEV)
    x[:, 0] = 1
    x[:, 1] = pattern((n,), a, 9, DEV)
    w = torch.zeros((2, hidden, dim), device=DEV)
    w[0, :, 0] = 128
    w[1, :, 1] = pattern((hidden,), b, 10, DEV)
    dh, at = one_of_each_row(hidden, n, 0, 1.0, 11, DEV)
    _, gg, _ = ersj.gated_grad(dh.t().contiguous(), ersj.pack_rows(x) if held else x, w[0], w[1], "silu", False, True, False)
    h = torch.arange(hidden, device=DEV)
    want = (dh[h, at].to(F64) * x[at, 1].to(F64) * w[1, :, 1].to(F64))[:, None] * x[at].to(F64)
    same(gg[:, 2:], want[:, 2:])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("n,dim,hidden", SIZES[1:] + [(9001, 199, 331)])
def test_gradient_from_held_rows(n, dim, hidden, kind):
    # dg and du of 16 bits in two parts and in one, in tiles of 128 and 256
    dtype = TYPES[kind]
    x, wg, wu, dh = (t.to(dtype) for t in (randn((n, dim), 20), randn((hidden, dim), 21, dim ** -0.5),
                                           randn((hidden, dim), 22, dim ** -0.5), randn((n, hidden), 23, 0.1)))
    kept = ersj.pack_rows(x)
    check_gated_grad(ersj.gated_grad(dh, kept, wg, wu, "gelu"), dh, ersj.unpack_rows(kept), wg, wu, "gelu", held=True)
