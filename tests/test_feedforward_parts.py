"""That the checks of 32-bit products by three bf16 parts notice every product that
is left out (mistakes planted in an emulation, on the CPU)."""
import pytest
import torch

from encoder_util import F64
from feedforward_parts import EXACT_PAIRS, PRODUCTS, one_of_each_row, parts, pattern, product, whole_bound


def rel(got, ref):
    return float((got - ref).norm() / ref.norm())


def randn(shape, seed, scale=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).mul_(scale)


def test_parts_hold_all_bits():
    x = torch.cat([randn((4000,), 1), randn((1000,), 2, 1e20), randn((1000,), 3, 1e-20)])
    assert torch.equal(sum(parts(x)), x.to(F64))


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("k", [64, 385, 1100, 4104, 9000])
def test_the_whole_bound_notices_each_product(k, held):
    x, y = randn((96, k), 1), randn((64, k), 2, k ** -0.5)
    if held:  # bf16 numbers
        x = x.to(torch.bfloat16).float()
    ref = x.to(F64) @ y.to(F64).t()
    # all of them: nothing is missed that the bound sees, with room for the additions
    assert rel(product(x, y, held=held), ref) < 0.1 * whole_bound(k)
    for but in PRODUCTS:
        if held and but[0]:
            continue
        assert rel(product(x, y, but, held), ref) > 1.2 * whole_bound(k), but


@pytest.mark.parametrize("dim,k", [(64, 171), (384, 1000), (1100, 1400), (4104, 4200), (384, 9000)])
def test_the_whole_bound_of_two_sums_notices_each_product(dim, k):
    # a sum over k of what comes from sums over dim, as dx of dg: left out in the second sum
    x, y = randn((64, k), 1), randn((64, k), 2, k ** -0.5)
    ref = x.to(F64) @ y.to(F64).t()
    for but in PRODUCTS:
        assert rel(product(x, y, but), ref) > 1.1 * whole_bound(dim, k), but


def test_the_exact_inputs_notice_each_product():
    noticed = set()
    for a, b in EXACT_PAIRS:
        x, at = one_of_each_row(50, 90, 1, a, 1, "cpu")
        y = pattern((70, 90), b, 2, "cpu")
        want = x.to(F64) @ y.to(F64).t()
        assert torch.equal(want.float().to(F64), want)  # 32-bit numbers
        assert torch.equal(product(x, y), want)
        noticed |= {but for but in PRODUCTS if not torch.equal(product(x, y, but), want)}
    assert noticed == set(PRODUCTS)
