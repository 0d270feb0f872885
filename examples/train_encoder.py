"""A late-interaction encoder trained and searched with this package's operators, end to end.

Texts are packed: one [n_tokens, ...] array, with offsets between the texts. A step encodes
documents and queries (rotary positions and attention over packed texts), scores every query
against every document (maxsim), takes the cross-entropy of the matching document, goes back
through all of it and clips the gradients by their global norm. Afterwards the documents are
encoded once more, without gradients, and a query is answered: encode, score, best five.

    python examples/train_encoder.py --steps 200

The texts are random: a query holds tokens of the document it belongs to, three in four replaced
by their partner under one permutation of the vocabulary, which is what there is to learn.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import maxsim_scoring_fwd_amd as ms  # noqa: E402

BF16 = torch.bfloat16
TEMPERATURE = 20.0  # of the mean over a query's tokens of their best cosine


def linear(x: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    return F.linear(x, w.to(x.dtype))


class Layer(torch.nn.Module):
    def __init__(self, hidden: int, heads: int, kv_heads: int, inner: int):
        super().__init__()
        self.heads, self.kv_heads, self.d = heads, kv_heads, hidden // heads
        rows = (heads + 2 * kv_heads) * self.d

        def weight(n, m):
            return torch.nn.Parameter(torch.randn(n, m) * m ** -0.5)

        self.qkv, self.out = weight(rows, hidden), weight(hidden, hidden)
        self.up, self.down = weight(inner, hidden), weight(hidden, inner)
        freq = 10000.0 ** (-torch.arange(self.d // 2, dtype=torch.float64) / (self.d // 2))
        self.register_buffer("freq", freq.float())

    def forward(self, x: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
        # query and key heads lie side by side, so one call turns both
        turned = self.heads + self.kv_heads
        y = linear(F.rms_norm(x, x.shape[-1:]), self.qkv).unflatten(-1, (-1, self.d))
        qk = ms.rotary(y[:, :turned], self.freq, offsets)
        o = ms.attention(qk[:, :self.heads], qk[:, self.heads:], y[:, turned:], offsets)
        x = x + linear(o.flatten(-2), self.out)
        return x + linear(F.gelu(linear(F.rms_norm(x, x.shape[-1:]), self.up)), self.down)


class Encoder(torch.nn.Module):
    """Tokens [n_tokens] of packed texts -> unit vectors [n_tokens, width] in bf16."""

    def __init__(self, vocab: int, hidden: int = 256, heads: int = 4, kv_heads: int = 2,
                 layers: int = 2, width: int = 128):
        super().__init__()
        self.table = torch.nn.Parameter(torch.randn(vocab, hidden))
        self.layers = torch.nn.ModuleList(Layer(hidden, heads, kv_heads, 4 * hidden)
                                          for _ in range(layers))
        self.project = torch.nn.Parameter(torch.randn(width, hidden) * hidden ** -0.5)

    def forward(self, tokens: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
        x = self.table[tokens].to(BF16)
        for layer in self.layers:
            x = layer(x, offsets)
        return F.normalize(linear(x, self.project).float(), dim=-1).to(BF16)


def offsets_of(lengths: torch.Tensor) -> torch.Tensor:
    return F.pad(lengths.cumsum(0), (1, 0)).cuda()


def batch(n: int, vocab: int, query: int, rng: torch.Generator):
    """n documents of 20 to 180 tokens, and n queries that hold tokens of theirs or the partners."""
    lengths = torch.randint(20, 181, (n,), generator=rng)
    docs = torch.randint(vocab, (int(lengths.sum()),), generator=rng)
    queries = torch.cat([d[torch.randint(len(d), (query,), generator=rng)]
                         for d in docs.split(lengths.tolist())])
    partner = torch.randperm(vocab, generator=torch.Generator().manual_seed(0))
    other = torch.rand(len(queries), generator=rng) < 0.75
    return (docs.cuda(), offsets_of(lengths), torch.where(other, partner[queries], queries).cuda(),
            offsets_of(torch.full((n,), query)))


def loss_of(encoder: Encoder, docs, doc_offsets, queries, query_offsets, query: int) -> torch.Tensor:
    D = encoder(docs, doc_offsets)
    Q = encoder(queries, query_offsets)
    scores = torch.stack([ms.maxsim(q, D, doc_offsets) for q in Q.split(query)])
    return F.cross_entropy(scores * (TEMPERATURE / query), torch.arange(len(scores), device=scores.device))


def train(steps: int, docs: int = 32, query: int = 32, vocab: int = 300, max_norm: float = 1.0,
          report=print):
    """The losses of the steps, and the encoder."""
    torch.manual_seed(0)
    rng = torch.Generator().manual_seed(1)
    encoder = Encoder(vocab).cuda()
    optimizer = torch.optim.AdamW(encoder.parameters(), lr=1e-3)
    losses = []
    for step in range(steps):
        loss = loss_of(encoder, *batch(docs, vocab, query, rng), query)
        optimizer.zero_grad()
        loss.backward()
        norm = ms.maxsim_clip_grad_norm([p.grad for p in encoder.parameters()], max_norm)
        optimizer.step()
        losses.append(float(loss.detach()))
        if step % 20 == 0 or step == steps - 1:
            report(f"step {step}: loss {losses[-1]:.3f}, gradient norm {float(norm):.3f}")
    return losses, encoder


@torch.no_grad()
def search(encoder: Encoder, docs: int = 200, query: int = 32, vocab: int = 300, k: int = 5):
    """How many of 20 queries find their document first among `docs`, and the last one's best k."""
    texts, doc_offsets, queries, _ = batch(docs, vocab, query, torch.Generator().manual_seed(2))
    D = encoder(texts, doc_offsets)
    one = offsets_of(torch.tensor([query]))
    found = 0
    for i in range(20):
        Q = encoder(queries[i * query:(i + 1) * query], one)
        scores, index = ms.maxsim_topk(ms.maxsim_score(Q, D, doc_offsets), k)
        found += int(index[0]) == i
    return found, index.tolist()


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=200)
    a = p.parse_args()
    _, encoder = train(a.steps)
    found, best = search(encoder)
    print(f"{found} of 20 queries find their document first among 200; the last one's best: {best}")


if __name__ == "__main__":
    main()
