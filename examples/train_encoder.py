"""Train a token-table encoder and join the vectors it makes.

A text's vector is the mean of its normalised token rows, scaled to unit
length: embed -> layer_norm -> mean over the text -> unit length.  With
``--hidden`` a gated feed-forward block is added to the rows before the mean, and
what the backward pass needs of the forward pass is kept in 8 bits.  Training
draws pairs of texts of one topic together and apart from the other texts of
the batch, clips the gradients by their global norm and takes a step; the
exact epsilon self-join then finds all pairs of texts whose vectors lie within
a given distance.  Synthetic topics stand in for a corpus.

    python examples/train_encoder.py [--texts 20000] [--steps 200] [--hidden 192]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import exact_range_similarity_amd as ersj


class Corpus:
    """Texts of ragged lengths: a share of each text's tokens comes from its
    topic's own few, the rest from a vocabulary all texts use.  The last id pads."""

    def __init__(self, texts, topics, vocab, length, seed, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.padding = vocab - 1
        self.topic = torch.arange(texts, device=device) % topics
        own = torch.randint(0, vocab - 1, (topics, 40), generator=g, device=device)
        pick = torch.randint(0, 40, (texts, length), generator=g, device=device)
        common = (torch.rand((texts, length), generator=g, device=device).pow(4) * (vocab - 1)).long()
        from_topic = torch.rand((texts, length), generator=g, device=device) < 0.25
        ids = torch.where(from_topic, own[self.topic].gather(1, pick), common)
        lengths = torch.randint(length // 2, length + 1, (texts, 1), generator=g, device=device)
        ids[torch.arange(length, device=device)[None, :] >= lengths] = self.padding
        self.ids = ids
        self.texts_of = torch.argsort(self.topic, stable=True).view(topics, -1)

    def pairs(self, batch, g):
        """Rows of two texts each of ``batch`` different topics."""
        topics = torch.randperm(self.texts_of.shape[0], generator=g, device=g.device)[:batch]
        members = torch.randint(0, self.texts_of.shape[1], (2, len(topics)), generator=g, device=g.device)
        return self.texts_of[topics, members[0]], self.texts_of[topics, members[1]]


class Encoder:
    def __init__(self, vocab, dim, padding, seed, hidden=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.table = torch.randn((vocab, dim), generator=g, device=device).mul_(dim ** -0.5).requires_grad_()
        self.weight = torch.ones(dim, device=device, requires_grad=True)
        self.bias = torch.zeros(dim, device=device, requires_grad=True)
        self.padding, self.scale = padding, dim ** 0.5
        self.block = None
        if hidden:  # both projections up, one down that begins at zero
            up = [torch.randn((hidden, dim), generator=g, device=device).mul_(dim ** -0.5) for _ in range(2)]
            self.block = [w.to(torch.bfloat16).requires_grad_()
                          for w in (*up, torch.zeros((dim, hidden), device=device))]

    def parameters(self):
        return [self.table, self.weight, self.bias] + (self.block or [])

    def __call__(self, ids):
        rows = ersj.embed(self.table, ids, self.scale, self.padding, torch.bfloat16)
        rows, _, _ = ersj.layer_norm(rows, self.weight, self.bias, pack=self.block is not None)
        if self.block:
            gate, up, down = self.block
            rows = rows + ersj.gated(rows, gate, up, "gelu", pack=True) @ down.t()
        kept = (ids != self.padding).unsqueeze(-1)
        total = (rows.float() * kept).sum(dim=1)
        return total / total.norm(dim=1, keepdim=True).clamp_min(1e-12)


def vectors(encoder, ids, chunk=4096):
    with torch.no_grad():
        return torch.cat([encoder(ids[i:i + chunk]) for i in range(0, len(ids), chunk)])


def join_quality(x, topic, eps):
    """(precision, recall) of the joined pairs as pairs of one topic, self pairs left out."""
    hits = found = 0
    for part in ersj.self_join(x.contiguous(), eps):
        a, b = part[:, 0].long(), part[:, 1].long()
        other = a != b
        found += int(other.sum())
        hits += int((other & (topic[a] == topic[b])).sum())
    count = torch.bincount(topic)
    wanted = int((count * (count - 1)).sum())
    return (hits / found if found else 1.0), hits / wanted


def train(texts=20000, topics=500, vocab=32768, dim=64, length=48, batch=256, steps=200, rate=60.0, max_norm=0.5,
          eps=0.9, seed=0, hidden=0, log=print):
    corpus = Corpus(texts, topics, vocab, length, seed)
    encoder = Encoder(vocab, dim, corpus.padding, seed + 1, hidden)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    target = torch.arange(min(batch, topics), device="cuda")
    quality = [join_quality(vectors(encoder, corpus.ids), corpus.topic, eps)]
    log(f"before: precision {quality[0][0]:.3f} recall {quality[0][1]:.3f} at eps {eps}")
    clipping, losses, norms = None, [], []
    for step in range(steps):
        first, second = corpus.pairs(batch, g)
        logits = encoder(corpus.ids[first]) @ encoder(corpus.ids[second]).t() / 0.1
        loss = torch.nn.functional.cross_entropy(logits, target)
        loss.backward()
        if clipping is None:  # the gradients keep their memory from here on
            clipping = ersj.GradSet([p.grad for p in encoder.parameters()])
        norm = ersj.clip_grads(clipping, max_norm)
        with torch.no_grad():
            for p in encoder.parameters():
                p.sub_(p.grad, alpha=rate if p is encoder.table else rate * 0.001)
                p.grad.zero_()
        losses.append(loss.detach())
        norms.append(norm)
        if step % 50 == 0 or step == steps - 1:
            log(f"step {step}: loss {float(losses[-1]):.4f} gradient norm {float(norm):.4f}")
    quality.append(join_quality(vectors(encoder, corpus.ids), corpus.topic, eps))
    log(f"after: precision {quality[1][0]:.3f} recall {quality[1][1]:.3f} at eps {eps}")
    return quality, torch.stack(losses), torch.stack(norms)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--texts", type=int, default=20000)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--dim", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=0)
    args = ap.parse_args()
    train(texts=args.texts, steps=args.steps, dim=args.dim, hidden=args.hidden)
