"""C ABI checks of the feed-forward operators that need no GPU: bad arguments are
refused before any HIP call; the binding refuses bad tensors and makes its
autograd nodes on the given stream."""
import os
import re

import pytest
import torch

import exact_range_similarity_amd as ersj
from exact_range_similarity_amd import encoder, feedforward

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: validation fails first
NAN, INF = float("nan"), float("inf")


def message():
    return ersj.lib().ersj_last_error().decode()


def refused(rc):
    assert rc == ersj.ERR_INVALID_ARG
    assert message()


def test_constants_agree_with_the_header():
    with open(os.path.join(ROOT, "include", "ersj_encoder.h")) as f:
        text = f.read()
    assert int(re.search(r"#define ERSJ_PACK_BLOCK (\d+)", text).group(1)) == encoder.PACK_BLOCK
    names = dict(re.findall(r"ERSJ_(SILU|GELU|GELU_TANH) = (\d)", text))
    assert {k.lower(): int(v) for k, v in names.items()} == feedforward.ACTIVATIONS


def pack(**kw):
    a = dict(x=FAKE, type=2, n=3, dim=4, ld_x=4, codes=FAKE, scales=FAKE)
    a.update(kw)
    return ersj.lib().ersj_pack_rows(*a.values(), None)


def unpack(**kw):
    a = dict(codes=FAKE, scales=FAKE, n=3, dim=4, x=FAKE, type=2, ld_x=4)
    a.update(kw)
    return ersj.lib().ersj_unpack_rows(*a.values(), None)


@pytest.mark.parametrize("call", [pack, unpack])
@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=FAKE + 1), dict(type=3), dict(type=-1), dict(n=-1), dict(n=2 ** 31), dict(dim=0),
    dict(dim=65537), dict(ld_x=3), dict(ld_x=2 ** 41), dict(codes=None), dict(scales=None),
    dict(n=2 ** 31 - 1, dim=65536, ld_x=65536),
])
def test_pack_and_unpack_reject_bad_arguments(call, kw):
    refused(call(**kw))


def norm_pack(**kw):
    a = dict(x=FAKE, type=2, n=3, dim=4, ld_x=4, weight=FAKE, bias=FAKE, param_type=0, eps=1e-5, y=FAKE, ld_y=4,
             mean=FAKE, rstd=FAKE, codes=FAKE, scales=FAKE)
    a.update(kw)
    return ersj.lib().ersj_layer_norm_pack(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(type=4), dict(n=-1), dict(dim=0), dict(ld_x=3), dict(weight=FAKE + 2), dict(param_type=1),
    dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(y=None), dict(ld_y=8), dict(mean=FAKE + 2), dict(rstd=FAKE + 1),
    dict(codes=None), dict(scales=None),
])
def test_layer_norm_pack_rejects_bad_arguments(kw):
    refused(norm_pack(**kw))


def norm_grad_packed(**kw):
    a = dict(gy=FAKE, ld_gy=4, codes=FAKE, scales=FAKE, type=2, n=3, dim=4, mean=FAKE, rstd=FAKE, weight=FAKE,
             param_type=0, gx=FAKE, ld_gx=4, gw=FAKE, gb=FAKE, work=FAKE, bytes=1 << 30)
    a.update(kw)
    return ersj.lib().ersj_layer_norm_grad_packed(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(gy=None), dict(gy=FAKE + 1), dict(ld_gy=3), dict(codes=None), dict(scales=None), dict(type=5), dict(n=-1),
    dict(dim=0), dict(mean=None), dict(rstd=None), dict(mean=FAKE + 1), dict(weight=FAKE + 2), dict(param_type=1),
    dict(gx=FAKE + 1), dict(ld_gx=3), dict(gx=FAKE, ld_gx=8), dict(gw=FAKE + 2), dict(work=None, n=5000),
    dict(work=FAKE + 64, n=5000), dict(bytes=16, n=5000), dict(dim=40000, ld_gy=40000, ld_gx=40000, bytes=1000),
    dict(dim=40000, ld_gy=40000, ld_gx=40000, gw=None, gb=None, work=None, bytes=0),
])
def test_layer_norm_grad_packed_rejects_bad_arguments(kw):
    refused(norm_grad_packed(**kw))


def gated(**kw):
    a = dict(x=FAKE, type=2, n=3, dim=8, ld_x=8, gate=FAKE, ld_gate=8, up=FAKE, ld_up=8, hidden=16, act=0, h=FAKE,
             ld_h=16, work=FAKE, bytes=1 << 30)
    a.update(kw)
    return ersj.lib().ersj_gated(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=FAKE + 1), dict(type=3), dict(n=-1), dict(n=2 ** 30 + 1), dict(dim=0), dict(dim=65537),
    dict(ld_x=7), dict(gate=None), dict(gate=FAKE + 1), dict(ld_gate=7), dict(up=None), dict(ld_up=7), dict(hidden=0),
    dict(hidden=65537), dict(act=3), dict(act=-1), dict(h=None), dict(h=FAKE + 1), dict(ld_h=15), dict(ld_h=2 ** 21),
    dict(type=0, work=None), dict(type=0, work=FAKE + 64), dict(type=0, bytes=100), dict(dim=7, ld_x=7, bytes=0),
    dict(x=FAKE + 2, bytes=0), dict(ld_up=16, bytes=0),
])
def test_gated_rejects_bad_arguments(kw):
    refused(gated(**kw))


def gated_grad(**kw):
    a = dict(gh=FAKE, ld_gh=16, x=FAKE, ld_x=8, codes=None, scales=None, type=2, n=3, dim=8, gate=FAKE, ld_gate=8,
             up=FAKE, ld_up=8, hidden=16, act=0, gx=FAKE, ld_gx=8, ggate=FAKE, ld_ggate=8, gup=FAKE, ld_gup=8,
             work=FAKE, bytes=1 << 30)
    a.update(kw)
    return ersj.lib().ersj_gated_grad(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(gh=None), dict(gh=FAKE + 1), dict(ld_gh=15), dict(x=None), dict(x=FAKE + 1), dict(ld_x=7), dict(type=9),
    dict(codes=FAKE, scales=FAKE), dict(scales=FAKE), dict(x=None, codes=FAKE), dict(x=None, scales=FAKE), dict(n=-1),
    dict(n=2 ** 30 + 1), dict(dim=0), dict(gate=None), dict(up=FAKE + 1), dict(ld_gate=7), dict(hidden=0), dict(act=7),
    dict(gx=FAKE + 1), dict(ld_gx=7), dict(ld_gx=2 ** 21), dict(ggate=FAKE + 1), dict(ld_ggate=2 ** 21),
    dict(gup=FAKE + 1), dict(ld_gup=7), dict(work=None), dict(work=FAKE + 128), dict(bytes=10),
])
def test_gated_grad_rejects_bad_arguments(kw):
    refused(gated_grad(**kw))


def test_work_of_refused_sizes_is_none():
    L = ersj.lib()
    ok = (FAKE, 2, 3, 8, 8, FAKE, 8, FAKE, 8, 16)
    assert L.ersj_gated_work(*ok) == 0  # everything is read in place
    assert L.ersj_gated_work(FAKE, 0, 3, 8, 8, FAKE, 8, FAKE, 8, 16) > 0
    assert L.ersj_gated_work(FAKE, 0, 0, 8, 8, FAKE, 8, FAKE, 8, 16) == 0
    for at, bad in ((1, 3), (2, -1), (2, 2 ** 30 + 1), (3, 0), (3, 65537), (9, 0), (9, 65537)):
        args = list(ok)
        args[at] = bad
        assert L.ersj_gated_work(*args) == 0
        assert L.ersj_gated_grad_work(*args, 1, 1, 1) == 0
    assert L.ersj_gated_grad_work(*ok, 1, 1, 1) > 0
    assert L.ersj_layer_norm_grad_packed_work(7, 10, 10) == 0
    assert L.ersj_layer_norm_grad_packed_work(2, -1, 10) == 0
    assert L.ersj_layer_norm_grad_packed_work(2, 10, 65536) >= 10 * 65536 * 2


def test_empty_calls_need_no_device():
    # nothing is launched for no rows
    assert pack(n=0, x=None, codes=None, scales=None) == 0
    assert unpack(n=0, x=None, codes=None, scales=None) == 0
    assert norm_pack(n=0, x=None, y=None, codes=None, scales=None) == 0
    assert gated(n=0, x=None, h=None, work=None, bytes=0) == 0
    assert gated_grad(n=0, gh=None, x=None, ggate=None, gup=None) == 0
    assert gated_grad(gx=None, ggate=None, gup=None) == 0


def test_binding_refuses_what_is_not_on_the_gpu():
    x, w = torch.zeros(3, 8), torch.zeros(16, 8)
    for call in (lambda: ersj.gated(x, w, w), lambda: ersj.gated_grad(torch.zeros(3, 16), x, w, w),
                 lambda: ersj.pack_rows(x), lambda: ersj.layer_norm_pack(x),
                 lambda: ersj.unpack_rows(ersj.PackedRows(torch.zeros(3, 8, dtype=torch.int8),
                                                          torch.zeros(3, 1, dtype=torch.uint8), torch.float32))):
        with pytest.raises(TypeError, match="GPU"):
            call()
    for call in (lambda: ersj.gated(x.double(), w, w), lambda: ersj.gated("x", w, w), lambda: ersj.pack_rows(x.int()),
                 lambda: ersj.unpack_rows(x), lambda: ersj.gated_grad(x.half(), x, w, w)):
        with pytest.raises((TypeError, AttributeError)):
            call()


def test_packed_rows_are_checked():
    codes, scales = torch.zeros(3, 40, dtype=torch.int8), torch.zeros(3, 2, dtype=torch.uint8)
    assert ersj.PackedRows(codes, scales, torch.float16).shape == (3, 40)
    for c, s, t in ((codes.float(), scales, torch.float16), (codes, scales.int(), torch.float16),
                    (codes, scales[:, :1], torch.float16), (codes, scales[:2], torch.float16),
                    (codes.t(), scales, torch.float16), (codes[:, :0], scales[:, :0], torch.float16),
                    (codes, scales, torch.float64), (codes, None, torch.float16)):
        with pytest.raises((ValueError, TypeError)):
            ersj.PackedRows(c, s, t)


@pytest.mark.parametrize("op", ["gated", "gated packed", "layer_norm packed"])
def test_the_node_is_made_on_the_given_stream(op, monkeypatch):
    inside, seen = [], []

    def run_elsewhere(device, stream, tensors, call):
        inside.append(stream)
        try:
            return call()
        finally:
            inside.pop()

    class Node:
        @staticmethod
        def apply(*args):
            seen.append(list(inside))
            return "result"

    for m in (encoder, feedforward):
        monkeypatch.setattr(m, "_elsewhere", lambda device, stream: stream is not None)
        monkeypatch.setattr(m, "_run_elsewhere", run_elsewhere)
    monkeypatch.setattr(feedforward, "_Gated", Node)
    monkeypatch.setattr(encoder, "_LayerNormPacked", Node)
    x, w = torch.zeros(4, 8), torch.zeros(6, 8, requires_grad=True)
    call = {"gated": lambda **kw: ersj.gated(x, w, w, **kw),
            "gated packed": lambda **kw: ersj.gated(x, w, w, pack=True, **kw),
            "layer_norm packed": lambda **kw: ersj.layer_norm(w, pack=True, **kw)}[op]
    assert call(stream="side") == "result" and seen == [["side"]]
    seen.clear()
    assert call() == "result" and seen == [[]]
    with pytest.raises(ValueError, match="out cannot be given"):
        call(out=torch.zeros(4, 6))
