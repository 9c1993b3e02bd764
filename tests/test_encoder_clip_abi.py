"""C ABI checks of the clipping of tensors given directly that need no GPU."""
import ctypes

import pytest
import torch

import exact_range_similarity_amd as ersj
from exact_range_similarity_amd import encoder

FAKE = 0x10000  # never dereferenced: validation fails first
NAN = float("nan")


def arrays(ptrs, outs, sizes, types):
    n = len(sizes if sizes is not None else types)
    return (None if ptrs is None else (ctypes.c_void_p * n)(*ptrs), None if outs is None else (ctypes.c_void_p * n)(*outs),
            None if sizes is None else (ctypes.c_int64 * n)(*sizes),
            None if types is None else (ctypes.c_int32 * n)(*types))


def clip(count=2, ptrs=(FAKE, 2 * FAKE), outs=None, sizes=(4, 5), types=(0, 2), max_norm=1.0, norm=FAKE, work=FAKE,
         work_bytes=1 << 20):
    return ersj.lib().ersj_clip_tensors(count, *arrays(ptrs, outs, sizes, types), max_norm, norm, work, work_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(count=0), dict(count=-3), dict(count=65537), dict(ptrs=None), dict(sizes=None), dict(types=None),
    dict(ptrs=(FAKE, None)), dict(ptrs=(FAKE, FAKE + 1)), dict(outs=(None, FAKE)), dict(outs=(FAKE + 2, FAKE)),
    dict(sizes=(4, -1)), dict(sizes=(4, 2 ** 41)), dict(types=(0, 3)), dict(sizes=(2 ** 40, 2 ** 40)),
    dict(max_norm=-1.0), dict(max_norm=NAN), dict(norm=FAKE + 2), dict(work=None), dict(work=FAKE + 4),
    dict(work_bytes=16384), dict(work_bytes=0),
])
def test_clip_tensors_rejects_bad_arguments(kw):
    assert clip(**kw) == ersj.ERR_INVALID_ARG
    assert ersj.lib().ersj_last_error()


def work(sizes, types, count=None):
    return ersj.lib().ersj_clip_tensors_work(len(sizes) if count is None else count, *arrays(None, None, sizes, types)[2:])


def test_clip_tensors_work():
    assert work((4,), (0,), 0) == work((4,), (0,), 65537) == 0
    assert work((4, -1), (0, 0)) == work((4, 2 ** 41), (0, 0)) == work((4, 4), (0, 3)) == 0
    assert ersj.lib().ersj_clip_tensors_work(1, None, None) == 0
    assert work((0, 0), (0, 1)) == encoder.GRADS_WORK
    # the largest do not overflow
    assert work((2 ** 40,) * 65536, (0,) * 65536) > 2 ** 40
    need = work((4, 5), (0, 2))
    assert need > encoder.GRADS_WORK
    assert clip(work_bytes=need - 1) == ersj.ERR_INVALID_ARG
    if not torch.cuda.is_available():
        assert clip(work_bytes=need) == ersj.ERR_HIP  # what is refused then is the launch


def test_binding_rejects_tensors():
    w = torch.zeros(4, 8)
    for bad in ([w.double()], [w, None], [w.to(torch.int32)]):
        with pytest.raises(TypeError):
            ersj.clip_grads(bad, 1.0)
    for bad in ([w.t()], [w, w[:, :3]], []):
        with pytest.raises(ValueError):
            ersj.clip_grads(bad, 1.0)


def overlap_cases():
    a, b, c = FAKE, 2 * FAKE, 3 * FAKE
    f32, sizes = (0, 0), (100, 50)
    return [
        ("one tensor twice", dict(ptrs=(a, a), sizes=(100, 100), types=f32), False),
        ("a part of another", dict(ptrs=(a, a + 396), sizes=sizes, types=f32), False),
        ("a part of another, first", dict(ptrs=(a + 196, a), sizes=sizes, types=f32), False),
        ("a part of another, within", dict(ptrs=(a, a + 40), sizes=sizes, types=f32), False),
        ("end to end", dict(ptrs=(a, a + 400), sizes=sizes, types=f32), True),
        ("end to end, 16 bits", dict(ptrs=(a + 100, a), sizes=(100, 50), types=(0, 2)), True),
        ("empty and anywhere", dict(ptrs=(a, a + 4), sizes=(100, 0), types=f32), True),
        ("one output for two", dict(ptrs=(a, b), outs=(c, c), sizes=sizes, types=f32), False),
        ("an output in another's input", dict(ptrs=(a, b), outs=(c, a + 4), sizes=sizes, types=f32), False),
        ("an output next to its own input", dict(ptrs=(a, b), outs=(a + 4, c), sizes=sizes, types=f32), False),
        ("inputs exchanged", dict(ptrs=(a, b), outs=(b, a), sizes=sizes, types=f32), False),
        ("one in place, one not", dict(ptrs=(a, b), outs=(a, c), sizes=sizes, types=f32), True),
        ("one input for two outputs", dict(ptrs=(a, a), outs=(b, c), sizes=sizes, types=f32), True),
        ("one input in place and for another output", dict(ptrs=(a, a), outs=(a, c), sizes=sizes, types=f32), False),
    ]


@pytest.mark.parametrize("case", overlap_cases(), ids=lambda c: c[0])
def test_tensors_that_share_memory(case):
    # where one workgroup writes what another reads or writes, the result would
    # depend on which comes first
    _, kw, fine = case
    if fine and torch.cuda.is_available():
        pytest.skip("these pass the checks and would be launched on addresses that do not exist")
    want = {ersj.ERR_HIP, ersj.ERR_OOM} if fine else {ersj.ERR_INVALID_ARG}
    assert clip(**kw) in want
    if not fine:
        assert b"share" in ersj.lib().ersj_last_error()


def test_many_tensors_side_by_side():
    n, size = 3000, 33
    ptrs = [FAKE + 4 * size * (i * 7 % n) for i in range(n)]  # in no order
    kw = dict(sizes=(size,) * n, types=(0,) * n, count=n, work_bytes=1 << 30)
    if not torch.cuda.is_available():
        assert clip(ptrs=ptrs, **kw) == ersj.ERR_HIP
    ptrs[2000] += 4
    assert clip(ptrs=ptrs, **kw) == ersj.ERR_INVALID_ARG
