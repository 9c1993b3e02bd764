"""Clipping of tensors that are given directly, whose addresses may be new on
every call: no waiting, graphs, many tensors."""
import pytest
import torch

import exact_range_similarity_amd as ersj
from encoder_util import TYPES, check_clip
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


def occupy(ms):
    """Keep the current stream busy for about that time."""
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    torch.cuda._sleep(100000)
    b.record()
    b.synchronize()
    torch.cuda._sleep(int(100000 * ms / max(a.elapsed_time(b), 1e-3)))


def test_clipping_tensors_waits_for_nothing():
    g = gen(1)
    sizes = [5, 1000, 70000]
    ersj.clip_grads([torch.randn(s, generator=g, device=DEV) for s in sizes], 1.0)  # first use
    sets = [[torch.randn(s, generator=g, device=DEV) for s in sizes] for _ in range(4)]
    before = [[t.clone() for t in s] for s in sets]
    side, done, here = torch.cuda.Stream(), torch.cuda.Event(), torch.cuda.Event()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        occupy(100)
        done.record()
    occupy(60)
    here.record()
    norms = [ersj.clip_grads(s, 1.0) for s in sets]
    assert not here.query(), "the call waited for its own stream"
    assert not done.query(), "the call waited for another stream"
    torch.cuda.synchronize()
    for norm, s, b in zip(norms, sets, before):
        check_clip(norm, s, b, 1.0)


def test_clipping_tensors_in_a_graph():
    g = gen(2)
    sizes, types = [3, 50000, 17, 40001], ["f32", "bf16", "f16", "f32"]
    held = [torch.empty(s, dtype=TYPES[t], device=DEV) for s, t in zip(sizes, types)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = ersj.clip_grads(held, 2.0)
    for k in range(4):
        values = [torch.randn(s, generator=g, device=DEV).to(h.dtype) for s, h in zip(sizes, held)]
        for h, v in zip(held, values):
            h.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got, got_norm = [h.clone() for h in held], norm.clone()
        junk = torch.randn((500, 500), generator=g, device=DEV)
        (junk @ junk).sum().item()
        check_clip(got_norm, got, values, 2.0)
        eager = [v.clone() for v in values]
        assert torch.equal(ersj.clip_grads(eager, 2.0), got_norm)
        assert all(torch.equal(a, b) for a, b in zip(eager, got)), f"replay {k} differs from the eager call"


# around the number of tensors that one launch takes, lengths around those of the chunks
@pytest.mark.parametrize("count", [1, 2, 95, 96, 97, 192, 193, 500])
@pytest.mark.parametrize("types", [["f32"], ["bf16"], ["f32", "f16", "bf16"]])
def test_clipping_tensors_as_a_kept_set(count, types):
    g = gen(count)
    lengths = [0, 1, 7, 8192, 8193, 16384 - 63, 16384 + 63, 16385, 24600, 50001, 3, 0]
    grads = []
    for i in range(count):
        t, n = TYPES[types[i % len(types)]], lengths[i * 5 % len(lengths)]
        lead = i * 3 % 70  # any alignment
        grads.append(torch.randn(n + lead, generator=g, device=DEV).to(t)[lead:])
    before = [t.clone() for t in grads]
    # a set of the same addresses, so that the same chunks are summed
    out = [torch.empty_like(t) for t in grads]
    kept = ersj.GradSet(grads, out)
    for share in (0.5, 2.0, float("inf")):
        for t, b in zip(grads, before):
            t.copy_(b)
        norm = sum(float(b.double().square().sum()) for b in before) ** 0.5
        max_norm = norm * share if norm else 1.0
        want = ersj.clip_grads(kept, max_norm)
        got = ersj.clip_grads(iter(grads), max_norm)
        check_clip(got, grads, before, max_norm, f"{count} tensors")
        assert torch.equal(got, want)
        assert all(torch.equal(a, b) for a, b in zip(grads, out))


def test_clipping_tensors_on_a_stream():
    g = gen(3)
    side = torch.cuda.Stream()
    for k in range(4):
        grads = [torch.randn(s, generator=g, device=DEV) for s in (100, 30000)]
        before = [t.clone() for t in grads]
        side.wait_stream(torch.cuda.current_stream())
        norm = ersj.clip_grads(grads, 1.0, stream=side if k % 2 else side.cuda_stream)
        torch.cuda.current_stream().wait_stream(side)
        check_clip(norm, grads, before, 1.0)


def test_tensors_that_share_memory_are_refused():
    flat = torch.ones(1000, device=DEV)
    a, b, c = flat[:400], flat[400:], flat[399:500]
    other = torch.zeros(1000, device=DEV)
    ersj.GradSet([a, b])
    ersj.GradSet([a, c], [other[:400], other[400:501]])  # read twice, written once
    for grads, out in (([a, a], None), ([a, c], None), ([c, a], None), ([flat, b], None),
                       ([a, c], [other[:400], other[399:500]]), ([a, b], [a, flat[:600]]), ([a], [flat[1:401]])):
        with pytest.raises(ersj.ErsjError, match="share"):
            ersj.GradSet(grads, out)
        if out is None:
            with pytest.raises(ersj.ErsjError, match="share"):
                ersj.clip_grads(grads, 1.0)
    ersj.clip_grads([a, b[:0], a[:0], b], 1.0)
    torch.cuda.synchronize()
    assert bool((flat == flat[0]).all()) and abs(float(flat.norm()) - 1.0) < 1e-3


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_the_norm_at_other_places_in_memory(kind):
    # sums follow the tensors' places modulo 128 bytes: the same bits at places
    # that are equal in that, and anywhere the same norm within its rounding
    g = gen(4)
    sizes = [70001, 5, 16384, 40000, 129]
    values = [torch.randn(s, generator=g, device=DEV).mul_(torch.randn(s, generator=g, device=DEV).mul_(3).exp_())
              .to(TYPES[kind]) for s in sizes]
    line = 128 // values[0].element_size()

    def placed(lead):
        tensors = []
        for i, v in enumerate(values):
            buf = torch.empty(lead + i + v.numel(), dtype=v.dtype, device=DEV)
            assert buf.data_ptr() % 128 == 0
            buf[lead + i:] = v
            tensors.append(buf[lead + i:])
        return tensors

    for lead in (0, 1, 3, line // 2, line - 1):
        results = []
        for far in (0, line, 3 * line):
            tensors = placed(lead + far)
            results.append((ersj.clip_grads(tensors, 5.0), tensors))
            check_clip(*results[-1], values, 5.0, f"{lead} elements in")
        for norm, tensors in results[1:]:
            assert torch.equal(norm, results[0][0])
            assert all(torch.equal(a, b) for a, b in zip(tensors, results[0][1]))
