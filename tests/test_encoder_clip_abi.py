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
