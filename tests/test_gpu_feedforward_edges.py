"""The feed-forward operators where they can go wrong: empty and single rows,
extreme values, memory that is not theirs, layouts, streams, graphs, autograd."""
import pytest
import torch

import exact_range_similarity_amd as ersj
from encoder_util import F64, TYPES, check_norm_grad
from feedforward_util import ACTIVATIONS, act_ref, check_gated, check_gated_grad, held_ref
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")


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


def randn(shape, dtype, seed, scale=1.0):
    return torch.randn(shape, generator=gen(seed), device=DEV).mul_(scale).to(dtype)


def block(n, dim, hidden, dtype, seed=0):
    return (randn((n, dim), dtype, seed), randn((hidden, dim), dtype, seed + 1, dim ** -0.5),
            randn((hidden, dim), dtype, seed + 2, dim ** -0.5), randn((n, hidden), dtype, seed + 3, 0.1))


# ---- no rows, one row ----

@pytest.mark.parametrize("kind", list(TYPES))
def test_no_rows(kind):
    dtype = TYPES[kind]
    x, wg, wu, dh = block(0, 24, 40, dtype)
    assert ersj.gated(x, wg, wu).shape == (0, 40)
    gx, gg, gu = ersj.gated_grad(dh, x, wg, wu)
    assert gx.shape == (0, 24) and bool((gg == 0).all()) and bool((gu == 0).all())
    assert gg.shape == gu.shape == (40, 24)
    kept = ersj.pack_rows(x)
    assert kept.shape == (0, 24) and ersj.unpack_rows(kept).shape == (0, 24)
    gx, gg, gu = ersj.gated_grad(dh, kept, wg, wu)
    assert gx.shape == (0, 24) and bool((gg == 0).all()) and bool((gu == 0).all())
    y, mean, rstd, kept = ersj.layer_norm_pack(x)
    gx, gw, gb = ersj.layer_norm_grad(y, kept, mean, rstd)
    assert gx.shape == (0, 24) and bool((gw == 0).all()) and bool((gb == 0).all())
    assert ersj.gated(x.view(3, 0, 24), wg, wu).shape == (3, 0, 40)


@pytest.mark.parametrize("kind", list(TYPES))
def test_only_what_is_wanted(kind):
    x, wg, wu, dh = block(70, 40, 72, TYPES[kind], 3)
    whole = ersj.gated_grad(dh, x, wg, wu, "gelu")
    for want in range(8):
        wants = [bool(want >> k & 1) for k in range(3)]
        got = ersj.gated_grad(dh, x, wg, wu, "gelu", *wants)
        for g, w, ref in zip(got, wants, whole):
            assert (g is None) == (not w)
        # how a sum is cut depends on what is asked for
        check_gated_grad(got, dh, x, wg, wu, "gelu", label=f"want {wants}")


# ---- values ----

def test_pack_extremes():
    for dtype in TYPES.values():
        top, low = torch.finfo(dtype).max, torch.finfo(dtype).tiny
        x = randn((12, 70), dtype, 5)
        x[0] = 0
        x[1, 3] = top
        x[2, 40] = -top
        x[3] = top
        x[4] = low
        x[5] = low / 8  # subnormal
        x[6, :32] = 127.0
        x[7, :32] = 127.5 if dtype != torch.bfloat16 else 127.0
        x[8, 5] = NAN
        x[9, 69] = INF
        x[10, 32] = -INF
        x[11] *= low
        codes, scales, values = held_ref(x)
        got = ersj.pack_rows(x)
        assert torch.equal(got.codes, codes) and torch.equal(got.scales, scales)
        back = ersj.unpack_rows(got)
        assert torch.equal(torch.isnan(back), torch.isnan(values)) and not bool(torch.isinf(back).any())
        assert torch.equal(back.to(F64).nan_to_num(3.0), values.nan_to_num(3.0))
        # a block is lost as a whole, its neighbours are not
        assert bool(torch.isnan(back[8, :32]).all()) and bool(torch.isfinite(back[8, 32:]).all())
        # the norm's own holding agrees
        held = ersj.layer_norm_pack(x)[3]
        assert torch.equal(held.codes, codes) and torch.equal(held.scales, scales)


def test_held_values_are_near():
    # at most half a step 2^e off; e is the least for which 127 * 2^e reaches the
    # largest, so 127 * 2^(e - 1) is below it, and half a step below 1/127 of it
    for dtype in TYPES.values():
        x = randn((500, 96), dtype, 6)
        back = ersj.unpack_rows(ersj.pack_rows(x)).to(F64)
        most = x.to(F64).view(500, 3, 32).abs().amax(dim=2).repeat_interleave(32, dim=1)
        assert bool(((back - x.to(F64)).abs() <= most / 127).all())
        # held once, held for good
        again = ersj.pack_rows(back.to(dtype))
        assert torch.equal(ersj.unpack_rows(again).to(F64), back)


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("act", ACTIVATIONS)
def test_activations_over_their_range(act, kind):
    # g is x itself (one weight of 1), u is 1
    dtype = TYPES[kind]
    g = torch.cat([torch.linspace(-30, 30, 4001, device=DEV), torch.tensor([0.0, -0.0, 1e-6, -1e-6, 60.0, -60.0, 200.0,
                                                                            -200.0], device=DEV)]).to(dtype)
    x = torch.stack([g, torch.ones_like(g)], dim=1).contiguous()
    wg = torch.tensor([[1.0, 0.0]], device=DEV).to(dtype)
    wu = torch.tensor([[0.0, 1.0]], device=DEV).to(dtype)
    check_gated(ersj.gated(x, wg, wu, act), x, wg, wu, act)
    dh = torch.ones((len(g), 1), device=DEV, dtype=dtype)
    check_gated_grad(ersj.gated_grad(dh, x, wg, wu, act, True, False, False), dh, x, wg, wu, act)


@pytest.mark.parametrize("kind", list(TYPES))
def test_a_row_that_is_not_finite_stays_alone(kind):
    dtype = TYPES[kind]
    x, wg, wu, dh = block(150, 48, 80, dtype, 7)
    clean = ersj.gated(x, wg, wu)
    gclean = ersj.gated_grad(dh, x, wg, wu, "silu", True, False, False)[0]
    bad = x.clone()
    bad[3, 5] = NAN
    bad[149, 47] = INF  # the last of the last row
    h = ersj.gated(bad, wg, wu)
    gx = ersj.gated_grad(dh, bad, wg, wu, "silu", True, False, False)[0]
    rest = torch.ones(150, dtype=torch.bool, device=DEV)
    rest[3] = rest[149] = False
    assert torch.equal(h[rest], clean[rest]) and torch.equal(gx[rest], gclean[rest])
    assert bool(torch.isnan(h[3]).all()) and not bool(torch.isfinite(h[149]).any())


def test_zeros_behind_the_rows_are_not_read():
    # what lies beside the rows (a wider buffer full of NaN) must not count
    for kind, dtype in TYPES.items():
        for n, dim, hidden in ((5, 40, 24), (130, 72, 136), (33, 7, 9)):
            x, wg, wu, dh = block(n, dim, hidden, dtype, 8)

            def inside(t):
                wide = torch.full((t.shape[0] + 4, t.shape[1] + 24), NAN, device=DEV, dtype=dtype)
                wide[2:-2, 8:-16] = t
                return wide[2:-2, 8:-16]

            a, b, c, d = (inside(t) for t in (x, wg, wu, dh))
            check_gated(ersj.gated(a, b, c, "gelu"), x, wg, wu, "gelu", f"{kind} {n}")
            check_gated_grad(ersj.gated_grad(d, a, b, c, "gelu"), dh, x, wg, wu, "gelu", label=f"{kind} {n}")


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("n,dim,hidden", [(1, 8, 16), (5, 33, 9), (130, 72, 136), (300, 384, 129)])
def test_nothing_is_written_beside_the_results(n, dim, hidden, kind):
    dtype = TYPES[kind]
    x, wg, wu, _ = block(n, dim, hidden, dtype, 9)
    for left, right in ((8, 16), (3, 4)):
        wide = torch.full((n + 4, hidden + left + right), 7.0, device=DEV, dtype=dtype)
        out = wide[2:-2, left:left + hidden]
        assert ersj.gated(x, wg, wu, out=out) is out
        check_gated(out, x, wg, wu, "silu")
        out.fill_(7.0)
        assert bool((wide == 7.0).all())
    wide = torch.full((n + 4, dim + 11), 7.0, device=DEV, dtype=dtype)
    out = wide[2:-2, 3:3 + dim]
    assert ersj.unpack_rows(ersj.pack_rows(x), out=out) is out
    assert torch.equal(out.to(F64), held_ref(x)[2])
    out.fill_(7.0)
    assert bool((wide == 7.0).all())


# ---- layouts ----

def test_weights_as_halves_of_one_matrix_and_of_unlike_spacing():
    for kind, dtype in TYPES.items():
        x, wg, wu, dh = block(140, 64, 96, dtype, 11)
        both = torch.cat([wg, wu])
        check_gated(ersj.gated(x, both[:96], both[96:]), x, wg, wu, "silu", kind)
        spaced = torch.zeros((96, 80), device=DEV, dtype=dtype)
        spaced[:, :64] = wu
        check_gated(ersj.gated(x, wg, spaced[:, :64]), x, wg, wu, "silu", kind)
        check_gated_grad(ersj.gated_grad(dh, x, wg, spaced[:, :64]), dh, x, wg, wu, "silu", label=kind)
        # one of them off the 16 bytes that the loads take
        off = torch.zeros(96 * 64 + 1, device=DEV, dtype=dtype)[1:].view(96, 64)
        off.copy_(wg)
        check_gated_grad(ersj.gated_grad(dh, x, off, wu), dh, x, wg, wu, "silu", label=kind)
        # the same matrix twice
        check_gated_grad(ersj.gated_grad(dh, x, wg, wg), dh, x, wg, wg, "silu", label=kind)


def test_leading_shapes_and_refusals():
    x, wg, wu, dh = block(30, 16, 24, torch.bfloat16, 12)
    h = ersj.gated(x.view(2, 3, 5, 16), wg, wu)
    assert h.shape == (2, 3, 5, 24) and torch.equal(h.view(30, 24), ersj.gated(x, wg, wu))
    one = ersj.gated(x[0], wg, wu)  # a single row without a leading dimension
    assert one.shape == (24,)
    check_gated(one[None], x[:1], wg, wu, "silu")
    for call in (lambda: ersj.gated(x, wg, wu[:-1]), lambda: ersj.gated(x[:, :8], wg, wu), lambda: ersj.gated(x, wg.t(), wu),
                 lambda: ersj.gated(x[:, ::2], wg[:, :8], wu[:, :8]), lambda: ersj.gated(x, wg, wu, "relu"),
                 lambda: ersj.gated(x, wg[:0], wu[:0]), lambda: ersj.gated(x, wg, wu, out=h),
                 lambda: ersj.gated(x, wg, wu.cpu()), lambda: ersj.gated_grad(dh[:-1], x, wg, wu),
                 lambda: ersj.gated_grad(dh, x, wg, wu, "silu ")):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ersj.gated(x, wg.half(), wu), lambda: ersj.gated_grad(dh.float(), x, wg, wu),
                 lambda: ersj.gated_grad(dh.float(), ersj.pack_rows(x), wg, wu),
                 lambda: ersj.unpack_rows(x), lambda: ersj.layer_norm_grad(x.float(), ersj.pack_rows(x), None, None)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="overlap"):
        ersj.gated(x[:1].expand(4, 16), wg, wu)


def test_offsets_past_31_bits():
    # results of more than 2^31 values, rows whose offsets pass 2^32 bytes
    n, dim, hidden = 280000, 32, 8192
    x, wg, wu, _ = block(n, dim, hidden, torch.bfloat16, 13)
    h = ersj.gated(x, wg, wu)
    for r in (0, 131072, 262144, n - 200):
        check_gated(h[r:r + 200], x[r:r + 200], wg, wu, "silu", f"rows from {r}")
    del h
    wide = torch.empty((2200000, 1024), device=DEV, dtype=torch.bfloat16)
    x = wide[:, :64]
    x.copy_(randn((2200000, 64), torch.bfloat16, 14))
    wg, wu = randn((2, 24, 64), torch.bfloat16, 15, 0.125)
    h = ersj.gated(x, wg, wu)
    check_gated(h[-300:], x[-300:], wg, wu, "silu")
    dh = randn((2200000, 24), torch.bfloat16, 16)
    gx, gg, _ = ersj.gated_grad(dh, x, wg, wu, "silu", True, True, False)
    want = ersj.gated_grad(dh[-300:], x[-300:], wg, wu, "silu", True, False, False)[0]
    assert float((gx[-300:].to(F64) - want.to(F64)).norm() / want.to(F64).norm()) < 2.0 ** -8
    # the sum over all rows, with the rows side by side
    ref = ersj.gated_grad(dh, x.contiguous(), wg, wu, "silu", False, True, False)[1]
    assert torch.equal(gg, ref)
    kept = ersj.pack_rows(wide)  # 2.25e9 codes
    assert torch.equal(ersj.unpack_rows(ersj.PackedRows(kept.codes[-50:], kept.scales[-50:], kept.dtype))[:, :64].to(F64),
                       held_ref(x[-50:].contiguous())[2])


@pytest.mark.parametrize("dim,kind", [(33000, "bf16"), (17000, "f32"), (20000, "f16"), (65536, "bf16")])
def test_layer_norm_of_long_held_rows(dim, kind):
    x = randn((9, dim), TYPES[kind], dim)
    w, b = 1 + 0.1 * randn((dim,), torch.float32, 1), randn((dim,), torch.float32, 2)
    y, mean, rstd, kept = ersj.layer_norm_pack(x.clone(), w, b)
    codes, scales, values = held_ref(x)
    assert torch.equal(kept.codes, codes) and torch.equal(kept.scales, scales)
    z = x.clone()  # in place
    got = ersj.layer_norm_pack(z, w, b, out=z)
    assert got[0] is z and torch.equal(z, y) and torch.equal(got[3].codes, codes)
    dy = randn((9, dim), TYPES[kind], 3)
    check_norm_grad(ersj.layer_norm_grad(dy, kept, mean, rstd, w), dy, values, mean, rstd, w)


# ---- the same bits, streams, graphs ----

def test_the_same_bits_on_every_call():
    for n, dim, hidden, kind in ((700, 384, 1000, "bf16"), (3000, 100, 60, "f32"), (40, 64, 171, "f16")):
        x, wg, wu, dh = block(n, dim, hidden, TYPES[kind], 17)
        first = [ersj.gated(x, wg, wu), *ersj.gated_grad(dh, x, wg, wu)]
        for _ in range(5):
            for a, b in zip(first, [ersj.gated(x, wg, wu), *ersj.gated_grad(dh, x, wg, wu)]):
                assert torch.equal(a, b)


def test_calls_on_two_streams_at_once():
    jobs = [block(3000, 256, 512, torch.bfloat16, 20), block(2500, 260, 500, torch.float32, 30)]
    want = [[ersj.gated(x, g, u), *ersj.gated_grad(d, x, g, u), ersj.unpack_rows(ersj.pack_rows(x))] for x, g, u, d in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = [[], []]
        for k, ((x, g, u, d), s) in enumerate(zip(jobs, streams)):
            got[k] = [ersj.gated(x, g, u, stream=s), *ersj.gated_grad(d, x, g, u, stream=s),
                      ersj.unpack_rows(ersj.pack_rows(x, stream=s.cuda_stream), stream=s)]
        torch.cuda.synchronize()
        for a, b in zip(want[0] + want[1], got[0] + got[1]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", list(TYPES))
def test_graph_replay(kind):
    dtype = TYPES[kind]
    x, wg, wu, dh = block(600, 136, 200, dtype, 40)
    gamma, beta = randn((136,), torch.float32, 41), randn((136,), torch.float32, 42)

    def step():
        y, mean, rstd, kept = ersj.layer_norm_pack(x, gamma, beta)
        h = ersj.gated(y, wg, wu, "gelu")
        held = ersj.pack_rows(y)
        gy, gg, gu = ersj.gated_grad(dh, held, wg, wu, "gelu")
        return [h, gg, gu, *ersj.layer_norm_grad(gy, kept, mean, rstd, gamma), ersj.unpack_rows(held)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for turn in range(4):
        x.copy_(randn((600, 136), dtype, 50 + turn))
        dh.copy_(randn((600, 200), dtype, 60 + turn, 0.1))
        want = step()
        torch.cuda.synchronize()
        for t in out:
            t.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


# ---- autograd ----

@pytest.mark.parametrize("pack", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
def test_autograd_agrees_with_the_direct_calls(kind, pack):
    dtype = TYPES[kind]
    x, wg, wu, dh = block(90, 72, 40, dtype, 70)
    gamma, beta = 1 + 0.1 * randn((72,), torch.float32, 71), randn((72,), torch.float32, 72)
    leaves = [t.clone().requires_grad_() for t in (x, gamma, beta, wg, wu)]
    y = ersj.layer_norm(leaves[0], leaves[1], leaves[2], pack=pack)[0]
    h = ersj.gated(y, leaves[3], leaves[4], "gelu_tanh", pack=pack)
    h.backward(dh)
    z, mean, rstd, kept = ersj.layer_norm_pack(x, gamma, beta)
    assert torch.equal(y, ersj.layer_norm(x, gamma, beta)[0]) and torch.equal(h, ersj.gated(y.detach(), wg, wu, "gelu_tanh"))
    y = y.detach()
    gy, gg, gu = ersj.gated_grad(dh, ersj.pack_rows(y) if pack else y, wg, wu, "gelu_tanh")
    want = (*ersj.layer_norm_grad(gy, kept if pack else x, mean, rstd, gamma), gg, gu)
    for leaf, ref in zip(leaves, want):
        assert torch.equal(leaf.grad, ref)


def test_what_a_packed_graph_keeps():
    x, wg, wu, _ = block(4096, 256, 64, torch.bfloat16, 80)
    x.requires_grad_()
    torch.cuda.synchronize()

    def kept(pack):
        before = torch.cuda.memory_allocated()
        y = ersj.layer_norm(x * 1.0, pack=pack)[0]
        now = torch.cuda.memory_allocated() - before - y.numel() * y.element_size()
        del y
        return now

    rows = 4096 * 256
    assert kept(False) >= 2 * rows and kept(True) < 1.2 * rows


def test_gradients_of_one_weight_for_both_and_of_a_broadcast_result():
    x, w, _, _ = block(50, 24, 40, torch.float32, 81)
    leaf = w.clone().requires_grad_()
    ersj.gated(x, leaf, leaf).sum().backward()  # the gradient arrives expanded
    ones = torch.ones((50, 40), device=DEV)
    _, gg, gu = ersj.gated_grad(ones, x, w, w)
    assert torch.allclose(leaf.grad, gg + gu, rtol=0, atol=0)
    # a part of a wider result: spaced rows arrive
    more = randn((50, 13), torch.float32, 82)
    leaf = w.clone().requires_grad_()
    d = randn((50, 53), torch.float32, 83)
    torch.cat([more, ersj.gated(x, leaf, w)], dim=1).backward(d)
    assert torch.equal(leaf.grad, ersj.gated_grad(d[:, 13:], x, w, w, "silu", False, True, False)[1])


def test_saved_tensors_that_change_are_refused():
    x, wg, wu, dh = block(20, 16, 24, torch.float32, 84)
    wg.requires_grad_()
    h = ersj.gated(x, wg, wu)
    x.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        h.backward(dh)
    # held in 8 bits, x is not needed any more
    h = ersj.gated(x, wg, wu, pack=True)
    kept = ersj.pack_rows(x)
    x.zero_()
    h.backward(dh)
    assert torch.equal(wg.grad, ersj.gated_grad(dh, kept, wg.detach(), wu, "silu", False, True, False)[1])
    # outputs that are given count as written
    out = torch.zeros((20, 24), device=DEV)
    for call in (lambda: ersj.gated(x, wg.detach(), wu, out=out), lambda: ersj.unpack_rows(ersj.pack_rows(dh), out=out)):
        before = out._version
        call()
        assert out._version > before


def test_backward_runs_on_the_given_stream():
    side = torch.cuda.Stream()
    x, wg, wu, dh = block(2000, 64, 96, torch.bfloat16, 85)
    want = ersj.gated_grad(dh, ersj.pack_rows(x), wg, wu)
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu)]
    side.wait_stream(torch.cuda.current_stream())
    h = ersj.gated(*leaves, pack=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(500000)
    h.backward(dh * 1.0)
    with torch.cuda.stream(side):
        junk = [torch.full((2000 * 64,), NAN, device=DEV) for _ in range(20)]
    torch.cuda.synchronize()
    for leaf, ref in zip(leaves, want):
        assert torch.equal(leaf.grad, ref)
    del junk


@pytest.mark.parametrize("act", ACTIVATIONS)
def test_gradients_against_differences(act):
    # <gradient, direction> against central differences of the 64-bit form
    x, wg, wu, dh = block(12, 16, 24, torch.float32, 90)
    got = ersj.gated_grad(dh, x, wg, wu, act)

    def loss(x, wg, wu):
        return float((act_ref(x @ wg.t(), act)[0] * (x @ wu.t()) * dh.to(F64)).sum())

    at = [t.to(F64) for t in (x, wg, wu)]
    for k in range(3):
        v = torch.randn(at[k].shape, generator=gen(91 + k), device=DEV, dtype=F64)
        step = 1e-5
        plus = loss(*[t + step * v if i == k else t for i, t in enumerate(at)])
        minus = loss(*[t - step * v if i == k else t for i, t in enumerate(at)])
        slope = (plus - minus) / (2 * step)
        # 32-bit sums: 2^-24 times the number of terms, well below 1e-5 of their magnitude
        scale = float((got[k].to(F64).abs() * v.abs()).sum())
        assert abs(float((got[k].to(F64) * v).sum()) - slope) <= 1e-5 * scale


def test_forward_tangents_are_refused():
    fwd = torch.autograd.forward_ad
    x, wg, wu, dh = block(20, 16, 24, torch.float32, 95)
    mean, rstd = ersj.layer_norm(x)[1:]
    with fwd.dual_level():
        d = fwd.make_dual(x, x)
        for call in (lambda: ersj.gated(d, wg, wu), lambda: ersj.gated(x, fwd.make_dual(wg, wg), wu),
                     lambda: ersj.gated_grad(fwd.make_dual(dh, dh), x, wg, wu), lambda: ersj.gated_grad(dh, d, wg, wu),
                     lambda: ersj.pack_rows(d), lambda: ersj.layer_norm_pack(d),
                     lambda: ersj.layer_norm_grad(d, ersj.pack_rows(x), mean, rstd)):
            with pytest.raises(NotImplementedError):
                call()


def test_bf16_products_are_matrix_products():
    # whole numbers small enough to be exact: every product and sum is exact, whatever the tile
    for n, dim, hidden in ((3, 8, 8), (70, 40, 33), (400, 128, 300), (2100, 520, 2100)):
        for dtype in (torch.bfloat16, torch.float16, torch.float32):
            x = torch.randint(-1, 2, (n, dim), generator=gen(n), device=DEV).to(dtype)
            wg = torch.zeros((hidden, dim), device=DEV, dtype=dtype)
            wg[:, 0] = 64.0
            x[:, 0] = 1.0  # g = 64: silu(64) is 64 in 32 bits
            wu = torch.randint(-1, 2, (hidden, dim), generator=gen(n + 1), device=DEV).to(dtype)
            ref = 64.0 * (x.to(F64) @ wu.to(F64).t())
            assert torch.equal(ersj.gated(x, wg, wu).to(F64), ref.to(dtype).to(F64))
