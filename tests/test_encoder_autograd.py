"""How the binding of the encoder operators meets autograd, as far as it shows
without a GPU."""
import pytest
import torch

import exact_range_similarity_amd as ersj
from exact_range_similarity_amd import encoder


@pytest.mark.parametrize("op", ["embed", "layer_norm"])
def test_the_node_is_made_on_the_given_stream(op, monkeypatch):
    # autograd runs a node's backward pass on the stream that was current when
    # the node was made; what the forward pass saved was allocated on the given one
    inside, seen = [], []

    def run_elsewhere(device, stream, tensors, call):
        inside.append(stream)
        try:
            return call()
        finally:
            inside.pop()
            seen.append([t for t in tensors if t is not None])

    class Node:
        @staticmethod
        def apply(*args):
            seen.append(list(inside))
            return "result"

    monkeypatch.setattr(encoder, "_elsewhere", lambda device, stream: stream is not None)
    monkeypatch.setattr(encoder, "_run_elsewhere", run_elsewhere)
    monkeypatch.setattr(encoder, "_Embed", Node)
    monkeypatch.setattr(encoder, "_LayerNorm", Node)
    w = torch.zeros(4, 8, requires_grad=True)
    ids = torch.zeros(3, dtype=torch.int64)
    call, inputs = {"embed": (lambda **kw: ersj.embed(w, ids, **kw), [w, ids]),
                    "layer_norm": (lambda **kw: ersj.layer_norm(w, w[0], **kw), None)}[op]
    assert call(stream="side") == "result"
    assert seen[0] == ["side"]
    if inputs is not None:  # the inputs outlive the stream's use of them
        assert len(seen[1]) == 2 and all(a is b for a, b in zip(seen[1], inputs))
    seen.clear()
    assert call() == "result"
    assert seen == [[]]


@pytest.mark.parametrize("op", ["embed", "layer_norm"])
def test_spaced_gradients_are_not_copied(op, monkeypatch):
    # the kernels take rows that are spaced; only what they cannot take is copied
    seen = []
    monkeypatch.setattr(encoder, "embed_grad", lambda grad, *a: seen.append(grad))
    monkeypatch.setattr(encoder, "layer_norm_grad", lambda grad, *a: seen.append(grad) or (None, None, None))

    class Ctx:
        args = (9, torch.float32, 1.0, None)
        saved_tensors = (torch.zeros(6), None, None, None)
        needs_input_grad = (True, False, False, False)
        bias_dtype = None

    def backward(grad):
        node = {"embed": lambda: encoder._Embed.backward(Ctx, grad),
                "layer_norm": lambda: encoder._LayerNorm.backward(Ctx, grad, None, None)}[op]
        node()
        return seen.pop()

    wide = torch.randn(6, 20)
    for grad in (wide, wide[:, 3:11], wide[1:2, :5], wide.view(2, 3, 20)[:, :, 4:7]):
        got = backward(grad)
        assert got.data_ptr() == grad.data_ptr() and got.stride() == grad.stride()
    for grad in (torch.ones(()).expand(6, 8), wide[:1].expand(6, 20), wide.t(), wide[:, ::2], wide.view(2, 3, 20)[:, :2]):
        got = backward(grad)
        assert got.is_contiguous() and torch.equal(got, grad)
