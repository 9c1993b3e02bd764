"""The activations of the gated block and their derivatives where their parts
overflow, underflow or cancel."""
import math

import pytest
import torch

import exact_range_similarity_amd as ersj
from encoder_util import F64, TYPES, U, close
from feedforward_util import ACTIVATIONS
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
    say(f"[feedforward] {request.node.name}")


def through(g, act, dtype):
    """act(g) and act'(g) by the block: one weight of 1 for g itself, u and grad_h 1."""
    x = torch.stack([g, torch.ones_like(g)], dim=1).to(dtype).contiguous()
    wg = torch.tensor([[1.0, 0.0]], device=DEV).to(dtype)
    wu = torch.tensor([[0.0, 1.0]], device=DEV).to(dtype)
    h = ersj.gated(x, wg, wu, act)
    gx, _, _ = ersj.gated_grad(torch.ones_like(h), x, wg, wu, act, True, False, False)
    return x[:, 0], h[:, 0], gx[:, 0]


@pytest.mark.parametrize("act", ACTIVATIONS)
@pytest.mark.parametrize("kind", list(TYPES))
def test_far_out(kind, act):
    # g^2 and g^3 overflow; the activation is g or 0 and its derivative 1 or 0
    g = torch.tensor([120.0, 6e4] if kind == "f16" else [120.0, 6e4, 1e7, 1e13, 1e19, 1e25, 3e38], device=DEV)
    for sign in (1.0, -1.0):
        x, h, slope = through(sign * g, act, TYPES[kind])
        assert torch.equal(h.abs(), x if sign > 0 else torch.zeros_like(x))
        assert torch.equal(slope.abs(), torch.ones_like(x) if sign > 0 else torch.zeros_like(x))


def test_gelu_keeps_the_bits_of_its_tail_in_32_bits():
    # Phi(g) relative to itself: erfcf of a rounded argument z is off by 16 steps of its
    # result, 32 u, and 2 z^2 = g^2 times the argument's 2 u; a few roundings follow.  The
    # derivative Phi + g phi adds 12 u of g phi (expf, and the density's products).
    g = torch.cat([torch.linspace(-12.5, 6, 60001, device=DEV), -torch.logspace(-6, 1, 2000, device=DEV)])
    x, h, slope = through(g, "gelu", torch.float32)
    x = x.to(F64)
    phi = 0.5 * torch.erfc(-x / math.sqrt(2))
    density = torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    rel = (36 + 2 * x * x) * U
    close(h, x * phi, x.abs() * phi * (rel + 2 * U) + 2.0 ** -148, "gelu")
    ref = phi + x * density
    close(slope, ref, phi * rel + x.abs() * density * 12 * U + ref.abs() * 2 * U + 2.0 ** -148, "slope")
