"""C ABI checks of the encoder operators that need no GPU: the library exports
every entry point of include/ersj_encoder.h and rejects bad arguments before
making any HIP call; the binding rejects bad tensors."""
import ctypes
import os
import re

import pytest
import torch

import exact_range_similarity_amd as ersj
from exact_range_similarity_amd import encoder

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: validation fails first
NAN, INF = float("nan"), float("inf")


def message():
    return ersj.lib().ersj_last_error().decode()


def test_header_and_binding_agree():
    with open(os.path.join(ROOT, "include", "ersj_encoder.h")) as f:
        text = f.read()
    # comments name entry points of both headers; declarations start a line
    names = set(re.findall(r"^(?:int|uint64_t|void) (ersj_[a-z_]+)\(", text, re.M))
    assert names == set(encoder.ENCODER_SYMBOLS)
    for name in names:
        assert hasattr(ersj.lib(), name), name
    assert int(re.search(r"#define ERSJ_GRADS_WORK (\d+)", text).group(1)) == encoder.GRADS_WORK


def embed(**kw):
    a = dict(table=FAKE, table_type=0, rows=10, dim=4, ld_table=4, ids=FAKE, id_type=1, n=3, scale=1.0, pad=-1,
             out=FAKE, out_type=0, ld_out=4)
    a.update(kw)
    return ersj.lib().ersj_embed(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(table=None), dict(table=FAKE + 2), dict(table_type=3), dict(table_type=-1), dict(rows=0), dict(rows=-1),
    dict(rows=2 ** 31 - 1), dict(dim=0), dict(dim=65537), dict(ld_table=3), dict(ld_table=2 ** 41), dict(ids=None),
    dict(ids=FAKE + 4), dict(id_type=2), dict(n=-1), dict(n=2 ** 31), dict(pad=-2), dict(out=None),
    dict(out_type=7), dict(ld_out=3), dict(table_type=1, out_type=0), dict(table_type=1, out_type=2),
])
def test_embed_rejects_bad_arguments(kw):
    assert embed(**kw) == ersj.ERR_INVALID_ARG
    assert message()


def embed_grad(**kw):
    a = dict(grad=FAKE, grad_type=2, ld_grad=4, ids=FAKE, id_type=1, n=3, scale=1.0, pad=-1, out=FAKE, out_type=2,
             rows=10, dim=4, ld_out=4, accumulate=0, work=FAKE, work_bytes=1 << 30)
    a.update(kw)
    return ersj.lib().ersj_embed_grad(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(grad=None), dict(grad=FAKE + 1), dict(grad_type=3), dict(ld_grad=3), dict(ids=None), dict(ids=FAKE + 4),
    dict(id_type=-1), dict(n=-1), dict(n=2 ** 31), dict(pad=-5), dict(out=None), dict(out_type=1), dict(rows=0),
    dict(rows=2 ** 31), dict(dim=0), dict(dim=1 << 20), dict(ld_out=2), dict(work=None, n=5000), dict(work=FAKE + 64),
    dict(work_bytes=16, n=5000),
])
def test_embed_grad_rejects_bad_arguments(kw):
    assert embed_grad(**kw) == ersj.ERR_INVALID_ARG
    assert message()


def norm(**kw):
    a = dict(x=FAKE, type=2, n=3, dim=4, ld_x=4, weight=FAKE, bias=FAKE, param_type=0, eps=1e-5, y=FAKE, ld_y=4,
             mean=FAKE, rstd=FAKE)
    a.update(kw)
    return ersj.lib().ersj_layer_norm(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=FAKE + 1), dict(type=4), dict(n=-1), dict(n=2 ** 31), dict(dim=0), dict(dim=65537),
    dict(ld_x=3), dict(weight=FAKE + 2), dict(bias=FAKE + 1), dict(param_type=1), dict(param_type=9), dict(eps=-1.0),
    dict(eps=NAN), dict(eps=INF), dict(y=None), dict(ld_y=3), dict(ld_y=8), dict(mean=FAKE + 2), dict(rstd=FAKE + 1),
])
def test_layer_norm_rejects_bad_arguments(kw):
    assert norm(**kw) == ersj.ERR_INVALID_ARG
    assert message()


def norm_grad(**kw):
    a = dict(gy=FAKE, ld_gy=4, x=2 * FAKE, ld_x=4, type=2, n=3, dim=4, mean=FAKE, rstd=FAKE, weight=FAKE, param_type=0,
             gx=3 * FAKE, ld_gx=4, gw=FAKE, gb=FAKE, work=FAKE, work_bytes=1 << 30)
    a.update(kw)
    return ersj.lib().ersj_layer_norm_grad(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(gy=None), dict(x=None), dict(ld_gy=3), dict(ld_x=1), dict(type=3), dict(n=-1), dict(dim=0), dict(mean=None),
    dict(rstd=None), dict(mean=FAKE + 2), dict(weight=FAKE + 1), dict(param_type=1), dict(ld_gx=3), dict(gw=FAKE + 1),
    dict(gb=FAKE + 2), dict(work=None, n=5000), dict(work=FAKE + 8), dict(work_bytes=7, n=5000), dict(gx=FAKE, ld_gx=6),
    dict(gx=2 * FAKE, ld_gx=6),
])
def test_layer_norm_grad_rejects_bad_arguments(kw):
    assert norm_grad(**kw) == ersj.ERR_INVALID_ARG
    assert message()


def create(count=2, ptrs=(FAKE, FAKE), outs=None, sizes=(4, 5), types=(0, 2), out=True):
    h = ctypes.c_void_p(77)
    n = len(ptrs) if ptrs is not None else 2
    rc = ersj.lib().ersj_grads_create(
        count, None if ptrs is None else (ctypes.c_void_p * n)(*ptrs),
        None if outs is None else (ctypes.c_void_p * n)(*outs),
        None if sizes is None else (ctypes.c_int64 * n)(*sizes),
        None if types is None else (ctypes.c_int32 * n)(*types), None, ctypes.byref(h) if out else None)
    return rc, h


@pytest.mark.parametrize("kw", [
    dict(count=0), dict(count=-3), dict(count=65537), dict(ptrs=None), dict(sizes=None), dict(types=None),
    dict(ptrs=(FAKE, None)), dict(ptrs=(FAKE, FAKE + 1)), dict(outs=(None, FAKE)), dict(outs=(FAKE + 2, FAKE)),
    dict(sizes=(4, -1)), dict(sizes=(4, 2 ** 41)), dict(types=(0, 3)),
    dict(sizes=(2 ** 40, 2 ** 40), count=2),
])
def test_grads_create_rejects_bad_arguments(kw):
    rc, h = create(**kw)
    assert rc == ersj.ERR_INVALID_ARG
    assert h.value is None
    assert message()


def test_grads_null_paths():
    L = ersj.lib()
    assert create(out=False)[0] == ersj.ERR_INVALID_ARG
    assert L.ersj_grads_clip(None, 1.0, None, FAKE, encoder.GRADS_WORK, None) == ersj.ERR_INVALID_ARG
    L.ersj_grads_free(None)


def test_grads_clip_rejects_bad_arguments():
    L = ersj.lib()
    # a set without elements needs no device memory
    rc, h = create(ptrs=(None, None), sizes=(0, 0))
    assert rc == ersj.OK
    for args in ((-1.0, None, FAKE, 16384), (NAN, None, FAKE, 16384), (1.0, FAKE + 2, FAKE, 16384),
                 (1.0, None, None, 16384), (1.0, None, FAKE + 4, 16384), (1.0, None, FAKE, 16383)):
        assert L.ersj_grads_clip(h, *args, None) == ersj.ERR_INVALID_ARG
        assert message()
    L.ersj_grads_free(h)


def test_work_sizes():
    L = ersj.lib()
    for n, rows, dim in ((-1, 5, 5), (2 ** 31, 5, 5), (5, 0, 5), (5, 2 ** 31, 5), (5, 5, 0), (5, 5, 65537)):
        assert L.ersj_embed_grad_work(n, rows, dim) == 0
    for n, dim in ((-1, 5), (2 ** 31, 5), (5, 0), (5, 65537)):
        assert L.ersj_layer_norm_grad_work(n, dim) == 0
    # the largest sizes do not overflow
    assert L.ersj_embed_grad_work(2 ** 31 - 1, 2 ** 31 - 2, 65536) > 2 ** 34
    assert L.ersj_layer_norm_grad_work(2 ** 31 - 1, 65536) >= 2 * 65536 * 4


def test_binding_rejects_host_tensors_and_types():
    w, ids = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(TypeError):
        ersj.embed(w, ids)
    with pytest.raises(TypeError):
        ersj.embed(w.double(), ids)
    with pytest.raises(TypeError):
        ersj.embed_grad(torch.zeros(3, 8), ids, 4)
    with pytest.raises(TypeError):
        ersj.layer_norm(w)
    with pytest.raises(TypeError):
        ersj.layer_norm(w.to(torch.int32))
    with pytest.raises(TypeError):
        ersj.layer_norm_grad(w, w.half(), w[:, 0], w[:, 0])
    with pytest.raises(TypeError):
        ersj.clip_grads([w], 1.0)
    with pytest.raises(ValueError):
        ersj.clip_grads([], 1.0)


def test_row_spacing():
    f = encoder._rows
    x = torch.zeros(6, 10)
    assert f(x, "x") == (6, 10)
    assert f(x[:, :7], "x") == (6, 10)
    assert f(x.reshape(2, 3, 10)[:, :, 2:9], "x") == (6, 10)
    assert f(x[0], "x") == (1, 10)
    assert f(x[:1, :3], "x") == (1, 3)
    assert f(torch.zeros(0, 5), "x") == (0, 5)
    assert f(torch.zeros(3, 1, 5)[:, 0], "x") == (3, 5)
    for bad in (x.t(), x[:, ::2], x.reshape(2, 3, 10)[:, :2, :4], torch.zeros(1, 10).expand(6, 10),
                torch.zeros(10, 1).expand(10, 6)):
        with pytest.raises(ValueError):
            f(bad, "x")
    with pytest.raises(ValueError):
        f(x, "x", 11)


def test_hip_failure_without_a_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; this checks the no-device error path")
    for rc in (embed(), embed_grad(), embed_grad(n=5000), norm(), norm_grad(), norm_grad(n=5000)):
        assert rc in (ersj.ERR_HIP, ersj.ERR_OOM)
    rc, h = create()
    assert rc in (ersj.ERR_HIP, ersj.ERR_OOM) and h.value is None


def test_empty_calls_do_nothing():
    # nothing to write: no launch, so no device is needed either
    assert embed(n=0, ids=None, out=None) == ersj.OK
    assert norm(n=0, x=None, y=None, mean=None, rstd=None) == ersj.OK
    assert norm_grad(n=0, gy=None, x=None, mean=None, rstd=None, gw=None, gb=None, work=None, work_bytes=0) == ersj.OK
