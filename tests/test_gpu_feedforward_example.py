"""examples/train_encoder.py with a gated block: the operators together in a model
that is trained, and the gradients of that model."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_train_encoder_with_a_block():
    import train_encoder

    quality, losses, norms = train_encoder.train(texts=1000, topics=50, vocab=2000, batch=32, steps=6, hidden=96,
                                                 log=lambda s: print(s, flush=True))
    assert bool(torch.isfinite(losses).all()) and bool(torch.isfinite(norms).all()) and bool((norms > 0).all())
    assert all(0 <= v <= 1 for pair in quality for v in pair)


def test_gradients_of_the_model():
    import train_encoder

    import exact_range_similarity_amd as ersj

    encoder = train_encoder.Encoder(300, 64, 299, 3, hidden=96)
    g = torch.Generator(device="cuda").manual_seed(4)
    with torch.no_grad():
        encoder.block[2].copy_(torch.randn((64, 96), generator=g, device="cuda") * 0.1)
    ids = torch.randint(0, 299, (20, 12), generator=g, device="cuda")
    ids[:, 9:] = 299
    target = torch.randn((20, 64), generator=g, device="cuda")
    (encoder(ids) * target).sum().backward()

    # the same model in 64 bits, plain torch, with the values that are held in the
    # place of those that the backward pass keeps
    leaves = [p.detach().double().requires_grad_() for p in encoder.parameters()]
    table, weight, bias, gate, up, down = leaves

    def swap(t, value):  # ``value`` forward, the gradient to t
        return t + (value - t).detach()

    # the held values take the place of the rows in the backward pass alone, which
    # plain torch cannot say; they are at most 1/127 of a run's largest off
    rows = table[ids] * 8.0 * (ids != 299).unsqueeze(-1)
    rows = swap(rows, rows.to(torch.bfloat16).double())
    mean = rows.mean(dim=-1, keepdim=True)
    y = (rows - mean) * ((rows - mean).square().mean(dim=-1, keepdim=True) + 1e-5).rsqrt() * weight + bias
    h = torch.nn.functional.gelu(y @ gate.t()) * (y @ up.t())
    y = y + h @ down.t()
    kept = (ids != 299).unsqueeze(-1)
    total = (y * kept).sum(dim=1)
    out = total / total.norm(dim=1, keepdim=True)
    (out * target.double()).sum().backward()
    for name, p, ref in zip(("table", "weight", "bias", "gate", "up", "down"), encoder.parameters(), leaves):
        off = float((p.grad.double() - ref.grad).norm() / ref.grad.norm())
        # bf16 rows and products (2^-8 each, a handful of them) and rows held in 8 bits (1/127)
        assert off < 6 * 2.0 ** -8 + 1 / 127, f"{name}: {off}"
    # without the table's padding row nothing reaches it
    assert bool((encoder.table.grad[299] == 0).all())
    # clipped together, with the 16-bit matrices of the block among them
    norm = ersj.clip_grads([p.grad for p in encoder.parameters()], 1e-3)
    assert float(norm) > 1e-3
