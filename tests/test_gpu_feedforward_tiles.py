"""The gated block and its gradient where the form of the projections' tiles
changes: sums of one to a few slabs with one tile of 128 to a compute unit, and the
sizes on both sides of 512 tiles of 64."""
import pytest
import torch

import exact_range_similarity_amd as ersj
from encoder_util import TYPES
from feedforward_util import check_gated, check_gated_grad
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


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("n,dim,hidden", [
    (1100, 1, 1000), (1100, 40, 1000), (1090, 65, 1001), (250, 130, 8000), (1100, 200, 997), (1100, 300, 1000),  # 1 to 5 slabs
    (1024, 72, 1024), (1025, 72, 1024), (64, 520, 16384), (65, 520, 16384), (1, 264, 9000), (128, 264, 9000),
    (2048, 40, 1024), (2049, 40, 1024),  # one tile of 128 to a unit, and more
])
def test_tiles(n, dim, hidden, kind):
    def rows(shape, seed, scale, pad):
        g = torch.Generator(DEV).manual_seed(seed)
        return torch.randn(shape[:1] + (shape[1] + pad,), generator=g, device=DEV).mul_(scale).to(TYPES[kind])[:, :shape[1]]

    for pad in (0, 3):
        x, dh = rows((n, dim), 1, 1.0, pad), rows((n, hidden), 2, 0.1, pad)
        wg, wu = rows((hidden, dim), 3, dim ** -0.5, pad), rows((hidden, dim), 4, dim ** -0.5, pad)
        check_gated(ersj.gated(x, wg, wu, "silu"), x, wg, wu, "silu", f"pad {pad}")
        check_gated_grad(ersj.gated_grad(dh, x, wg, wu, "silu"), dh, x, wg, wu, "silu", label=f"pad {pad}")
