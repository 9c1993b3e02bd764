"""examples/train_encoder.py on a small corpus: the encoder's operators, their
gradients, the clipping and the self-join together."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_train_encoder():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import train_encoder

    max_norm = 0.5
    kw = dict(texts=2000, topics=100, vocab=4000, batch=64, steps=40, max_norm=max_norm, log=lambda s: print(s, flush=True))
    quality, losses, norms = train_encoder.train(**kw)
    (p0, r0), (p1, r1) = quality
    assert p0 < 0.1 and r0 < 0.1  # untrained vectors say nothing of the topics
    assert p1 > 0.9 and r1 > 0.3
    assert bool(torch.isfinite(losses).all()) and float(losses[-1]) < 0.5 * float(losses[0])
    assert float(norms[0]) > max_norm  # the first steps are clipped
