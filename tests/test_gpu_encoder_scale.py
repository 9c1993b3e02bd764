"""The table's gradient where the scale is not finite."""
import pytest
import torch

import exact_range_similarity_amd as ersj
from encoder_util import TYPES
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


@pytest.mark.parametrize("scale", [float("inf"), float("nan"), -float("inf")])
@pytest.mark.parametrize("n", [0, 40, 3000])
@pytest.mark.parametrize("act,table,dim", [("f32", "f32", 5), ("bf16", "bf16", 384), ("bf16", "f32", 1030)])
def test_rows_without_tokens_are_zeros_whatever_the_scale(n, act, table, dim, scale):
    g = gen(n + dim)
    rows = 200
    ids = torch.randint(0, rows // 2, (n,), generator=g, device=DEV) * 2  # odd rows have none
    ids[:n // 3] = 8  # one row in several parts
    grad = torch.randint(1, 4, (n, dim), generator=g, device=DEV).to(TYPES[act])
    got = ersj.embed_grad(grad, ids, rows, scale, 4, TYPES[table])
    used = torch.bincount(ids, minlength=rows) > 0
    used[4] = False
    assert bool((got[~used] == 0).all())
    want = torch.tensor(scale, device=DEV).expand(int(used.sum()), dim)  # a positive sum times the scale
    assert torch.equal(got[used].float().nan_to_num(7.0), want.nan_to_num(7.0))
