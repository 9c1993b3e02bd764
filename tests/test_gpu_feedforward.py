"""The gated block, its gradient and rows held in 8 bits against their 64-bit
forms (MI355X)."""
import pytest
import torch

import exact_range_similarity_amd as ersj
from encoder_util import F64, TYPES, check_norm, check_norm_grad
from feedforward_util import ACTIVATIONS, check_gated, check_gated_grad, held_ref
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


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rows(shape, dtype, seed, pad=0, scale=1.0):
    """Rows of normal values that lie ``pad`` values apart, off the start of their buffer."""
    wide = torch.randn(shape[:-1] + (shape[-1] + pad,), generator=gen(seed), device=DEV).mul_(scale).to(dtype)
    return wide[..., :shape[-1]]


def block(n, dim, hidden, dtype, seed=0, pad=0):
    x = rows((n, dim), dtype, seed, pad)
    w = [rows((hidden, dim), dtype, seed + k, pad, dim ** -0.5) for k in (1, 2)]
    return x, w[0], w[1], rows((n, hidden), dtype, seed + 3, pad, 0.1)


SIZES = [(1, 1, 1), (1, 8, 16), (2, 16, 64), (3, 7, 5), (16, 64, 128), (17, 33, 65), (31, 64, 171), (64, 16, 16),
         (128, 128, 64), (129, 80, 72), (130, 385, 200), (257, 48, 129), (300, 72, 1000), (9, 384, 1024), (1, 1000, 333)]


@pytest.mark.parametrize("act", ACTIVATIONS)
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("n,dim,hidden", SIZES)
def test_gated(n, dim, hidden, kind, act):
    for pad in (0, 5, 8):
        x, wg, wu, _ = block(n, dim, hidden, TYPES[kind], 10, pad)
        check_gated(ersj.gated(x, wg, wu, act), x, wg, wu, act, f"pad {pad}")


@pytest.mark.parametrize("act", ACTIVATIONS)
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("n,dim,hidden", SIZES)
def test_gated_grad(n, dim, hidden, kind, act):
    for pad in (0, 3, 8):
        x, wg, wu, dh = block(n, dim, hidden, TYPES[kind], 20, pad)
        check_gated_grad(ersj.gated_grad(dh, x, wg, wu, act), dh, x, wg, wu, act, label=f"pad {pad}")


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("n,dim,hidden", [(5000, 384, 256), (1030, 520, 4000), (70000, 24, 40), (2500, 1040, 2080)])
def test_gated_of_many_rows(n, dim, hidden, kind):
    x, wg, wu, dh = block(n, dim, hidden, TYPES[kind], 30)
    check_gated(ersj.gated(x, wg, wu, "silu"), x, wg, wu, "silu")
    check_gated_grad(ersj.gated_grad(dh, x, wg, wu, "silu"), dh, x, wg, wu, "silu")


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("n,dim,hidden", [(4200, 4104, 2100), (4300, 4099, 2111), (1500, 1100, 700), (1500, 1097, 704)])
def test_gated_in_large_tiles(n, dim, hidden, kind):
    # enough of them for tiles of 256 in every product, with edges in both directions;
    # and just enough for one tile of 128 to a compute unit
    x, wg, wu, dh = block(n, dim, hidden, TYPES[kind], 50)
    check_gated(ersj.gated(x, wg, wu, "gelu"), x, wg, wu, "gelu")
    check_gated_grad(ersj.gated_grad(dh, x, wg, wu, "gelu"), dh, x, wg, wu, "gelu")


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("n,dim,hidden", [(9000, 1300, 3300), (9001, 1299, 3297), (9000, 770, 1030)])
def test_gated_grad_in_more_parts_than_run_at_once(n, dim, hidden, kind):
    x, wg, wu, dh = block(n, dim, hidden, TYPES[kind], 70)
    check_gated_grad(ersj.gated_grad(dh, x, wg, wu, "silu"), dh, x, wg, wu, "silu")


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("dim", [1, 3, 7, 8, 15, 16, 31, 32, 33, 63, 64, 65, 100, 384, 385, 1001])
def test_pack(dim, kind):
    for n, pad in ((1, 0), (7, 5), (300, 0), (333, 9)):
        x = rows((n, dim), TYPES[kind], dim, pad) * torch.exp2(torch.randint(-8, 8, (n, 1), generator=gen(dim), device=DEV))
        x = x.to(TYPES[kind])
        got = ersj.pack_rows(x)
        codes, scales, values = held_ref(x)
        assert torch.equal(got.codes, codes) and torch.equal(got.scales, scales)
        assert torch.equal(ersj.unpack_rows(got).to(F64), values)


@pytest.mark.parametrize("wkind", ["f32", "own"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("dim", [1, 2, 3, 5, 7, 8, 9, 16, 24, 31, 32, 33, 40, 63, 64, 65, 100, 127, 129, 384, 385, 500,
                                 1001, 2048, 4097, 8192, 12000, 20000])
def test_layer_norm_pack(dim, kind, wkind):
    dtype = TYPES[kind]
    for n, pad in ((1, 0), (65, 3), (400 if dim < 5000 else 40, 0)):
        x = (rows((n, dim), dtype, dim, pad) + 0.25).to(dtype)
        w = 1 + 0.1 * rows((dim,), torch.float32, 1)
        b = rows((dim,), torch.float32, 2)
        if wkind == "own":
            w, b = w.to(dtype), b.to(dtype)
        y, mean, rstd, kept = ersj.layer_norm_pack(x, w, b)
        check_norm((y, mean, rstd), x, w, b, 1e-5, f"n {n}")
        codes, scales, values = held_ref(x)
        assert torch.equal(kept.codes, codes) and torch.equal(kept.scales, scales)
        dy = rows((n, dim), dtype, 3, pad)
        check_norm_grad(ersj.layer_norm_grad(dy, kept, mean, rstd, w), dy, values, mean, rstd, w, f"n {n}")


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("n,dim,hidden", [(1, 8, 16), (31, 33, 65), (130, 384, 200), (700, 64, 171)])
def test_gated_grad_of_held_rows(n, dim, hidden, kind):
    x, wg, wu, dh = block(n, dim, hidden, TYPES[kind], 40)
    kept = ersj.pack_rows(x)
    values = ersj.unpack_rows(kept)
    check_gated_grad(ersj.gated_grad(dh, kept, wg, wu, "gelu"), dh, values, wg, wu, "gelu", held=True)
