"""The table's gradient for few tokens of very tall tables: more rows than one
launch has workgroups for."""
import gc

import pytest
import torch

import exact_range_similarity_amd as ersj
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
TURN = 2 ** 28  # rows of one launch


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ersj.lib()


@pytest.fixture(autouse=True)
def _case(request):
    say(f"[encoder] {request.node.name}")
    yield
    gc.collect()
    torch.cuda.empty_cache()


def nonzero_rows(t):
    step = 1 << 27
    return torch.cat([(t[r:r + step] != 0).any(dim=1).nonzero()[:, 0] + r for r in range(0, len(t), step)])


@pytest.mark.parametrize("rows,dim,dtype", [(TURN + 1, 1, torch.bfloat16), (600000003, 2, torch.bfloat16),
                                            (2 ** 31 - 2, 1, torch.float16)])
def test_tall_table_gradient(rows, dim, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows)
    # small whole numbers, so that every sum is exact; some rows of every launch have
    # more tokens than one wave adds alone
    some = torch.tensor([0, 1, 63, 64, TURN - 1, TURN, rows - 1, rows - 2, min(rows - 1, 2 * TURN + 5)], device=DEV)
    ids = some[torch.randint(0, len(some), (1000,), generator=g, device=DEV)]
    ids[::50] = torch.randint(0, rows, (20,), generator=g, device=DEV)
    grad = torch.randint(-2, 3, (1000, dim), generator=g, device=DEV).to(dtype)
    hit, where = torch.unique(ids, return_inverse=True)
    want = torch.zeros((len(hit), dim), device=DEV).index_add_(0, where, grad.float())
    out = torch.full((rows, dim), 3.0, dtype=dtype, device=DEV)
    ersj.embed_grad(grad, ids, rows, out=out)
    assert torch.equal(out[hit].float(), want)
    touched = nonzero_rows(out)
    assert torch.equal(touched, hit[(want != 0).any(dim=1)])
    ersj.embed_grad(grad, ids, rows, out=out, accumulate=True)
    assert torch.equal(out[hit].float(), 2 * want)
    assert torch.equal(nonzero_rows(out), touched)
    # no token at all: zeros everywhere
    out[-1] = 1
    ersj.embed_grad(grad[:0], ids[:0], rows, out=out)
    assert nonzero_rows(out).numel() == 0
