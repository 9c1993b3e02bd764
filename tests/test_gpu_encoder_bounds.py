"""Layer norm and its gradient under bounds that follow the kernels' sums.

A sum in which no term passes through more than c additions has an error of at
most c * u times the sum of the absolute values.  A lane adds its own columns one
after the other, at most four vectors of 16 bytes, or every 1024th column of a
row that is too long for that; then come six exchanges between the lanes of a
wave and at most 16 waves.  encoder_util.py's bounds count as many additions as a
row has columns instead, which leaves a row whose mean is far above its deviation
almost unchecked."""
import pytest
import torch

import exact_range_similarity_amd as ersj
from encoder_util import F64, TYPES, U, close, norm_grad_ref, norm_ref, rounded
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
SHIFTS = [0.0, 5000.0, -300.0, 1e6]  # of rows whose deviation is 1


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ersj.lib()


@pytest.fixture(autouse=True)
def _case(request):
    say(f"[encoder] {request.node.name}")


def additions(dtype, dim):
    lane = max(4 * 16 // dtype.itemsize, -(-dim // 1024))
    return min(lane, dim) + 6 + 16


def inputs(dim, act, param, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn((len(SHIFTS) * 5, dim), generator=g, device=DEV)
    x += torch.tensor(SHIFTS * 5, device=DEV)[:, None] if act == "f32" else 0.25
    w = 1 + 0.2 * torch.randn(dim, generator=g, device=DEV)
    b = torch.randn(dim, generator=g, device=DEV)
    dy = torch.randn(x.shape, generator=g, device=DEV)
    return x.to(TYPES[act]), w.to(TYPES[param]), b.to(TYPES[param]), dy.to(TYPES[act])


@pytest.mark.parametrize("act,param", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("dim", [7, 64, 385, 1001, 3001, 8200, 33001, 65536])
def test_layer_norm_within_its_sums_bounds(act, param, dim):
    x, w, b, dy = inputs(dim, act, param, dim)
    c = additions(x.dtype, dim)
    y, mean, rstd = ersj.layer_norm(x, w, b)
    ref, rmean, rrstd, xh = norm_ref(x, w, b, 1e-5)
    # c additions and a division
    emean = (c + 1) * U * x.to(F64).abs().mean(dim=-1, keepdim=True)
    close(mean, rmean[:, 0], rounded(rmean, emean, torch.float32)[:, 0], "mean")
    # squares of differences (3 roundings each), c additions, the division, eps, half
    # of each for the root; the square of the mean's error; root and reciprocal
    erel = (c + 8) / 2 * U + (emean * rrstd).square() / 2 + 3 * U
    close(rstd, rrstd[:, 0], rounded(rrstd, erel * rrstd, torch.float32)[:, 0], "rstd")
    scaled = xh * w.to(F64)
    err = (w.to(F64) * rrstd * emean).abs() + scaled.abs() * (erel + 3 * U) + U * (ref.abs() + scaled.abs())
    close(y, ref, rounded(ref, err, y.dtype), "y")

    # the gradient of x, from the statistics as they are
    gx = ersj.layer_norm_grad(dy, x, mean, rstd, w)[0]
    rx = norm_grad_ref(dy, x, mean, rstd, w)[0]
    r = rstd.to(F64)[:, None]
    xh = (x.to(F64) - mean.to(F64)[:, None]) * r
    g = dy.to(F64) * w.to(F64)
    s1, s2 = g.mean(dim=1, keepdim=True), (g * xh).mean(dim=1, keepdim=True)
    # terms of g (one rounding) and g * xh (four), c additions, the product with 1 / dim
    # (two); then the roundings of the sum that they enter
    err = r * ((c + 3) * U * g.abs().mean(dim=1, keepdim=True)
               + xh.abs() * (c + 6) * U * (g * xh).abs().mean(dim=1, keepdim=True)
               + 4 * U * (g.abs() + s1.abs() + (xh * s2).abs()) + 4 * U * (xh * s2).abs())
    close(gx, rx, rounded(rx, err, gx.dtype), "grad_x")
