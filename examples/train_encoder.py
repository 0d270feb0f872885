"""A late-interaction encoder trained and searched with this package's operators, end to end.

Texts are packed: one [n_tokens, ...] array, with offsets between the texts. A step encodes
documents and queries (norms with the residual's addition, rotary positions and attention over
packed texts), scores every query against every document (maxsim), takes the cross-entropy of the
matching document, goes back through all of it and clips the gradients by their global norm.
Afterwards the documents are encoded once more, without gradients, and a query is answered: encode,
score, best five; with --index int8 or mx4 from an index of 8-bit or 4-bit vectors.

    python examples/train_encoder.py --steps 200

With --masked the encoder first learns to fill in tokens that were taken out of the documents, with
dropout before every addition: the cross entropy over the vocabulary of those tokens alone.

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


def another(drop: dict) -> dict:
    """The dropout of the next place that drops: a call number of its own."""
    return dict(drop, call=drop["call"] + 1) if drop else drop


class Layer(torch.nn.Module):
    def __init__(self, hidden: int, heads: int, kv_heads: int, inner: int):
        super().__init__()
        self.heads, self.kv_heads, self.d = heads, kv_heads, hidden // heads
        rows = (heads + 2 * kv_heads) * self.d

        def weight(n, m):
            return torch.nn.Parameter(torch.randn(n, m) * m ** -0.5)

        self.qkv, self.out = weight(rows, hidden), weight(hidden, hidden)
        self.up, self.down = weight(inner, hidden), weight(hidden, inner)
        self.norm_in = torch.nn.Parameter(torch.ones(hidden))
        self.norm_mid = torch.nn.Parameter(torch.ones(hidden))
        freq = 10000.0 ** (-torch.arange(self.d // 2, dtype=torch.float64) / (self.d // 2))
        self.register_buffer("freq", freq.float())

    def forward(self, update: torch.Tensor, x, offsets: torch.Tensor, drop: dict):
        """The next update of the tokens' states, the states with this layer's first two, and the dropout
        of the next place."""
        y, x = ms.rms_norm(update, self.norm_in, x, **drop)
        drop = another(drop)
        # query and key heads lie side by side, so one call turns both
        turned = self.heads + self.kv_heads
        y = linear(y, self.qkv).unflatten(-1, (-1, self.d))
        qk = ms.rotary(y[:, :turned], self.freq, offsets)
        o = ms.attention(qk[:, :self.heads], qk[:, self.heads:], y[:, turned:], offsets)
        y, x = ms.rms_norm(linear(o.flatten(-2), self.out), self.norm_mid, x, **drop)
        return linear(F.gelu(linear(y, self.up)), self.down), x, another(drop)


class Encoder(torch.nn.Module):
    """Tokens [n_tokens] of packed texts -> unit vectors [n_tokens, width] in bf16."""

    def __init__(self, vocab: int, hidden: int = 256, heads: int = 4, kv_heads: int = 2,
                 layers: int = 2, width: int = 128):
        super().__init__()
        self.table = torch.nn.Parameter(torch.randn(vocab, hidden))
        self.layers = torch.nn.ModuleList(Layer(hidden, heads, kv_heads, 4 * hidden)
                                          for _ in range(layers))
        self.project = torch.nn.Parameter(torch.randn(width, hidden) * hidden ** -0.5)
        self.last = torch.nn.Parameter(torch.ones(hidden))

    def states(self, tokens: torch.Tensor, offsets: torch.Tensor, dropout: float = 0.0, rng=None):
        """The tokens' states after the last layer's norm."""
        drop = dict(dropout=dropout, rng=rng, call=0) if dropout else {}
        update, x = self.table[tokens].to(BF16), None
        for layer in self.layers:
            update, x, drop = layer(update, x, offsets, drop)
        return ms.rms_norm(update, self.last, x, **drop)[0]

    def forward(self, tokens: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
        y = self.states(tokens, offsets)
        return F.normalize(linear(y, self.project).float(), dim=-1).to(BF16)

    def masked_loss(self, tokens: torch.Tensor, offsets: torch.Tensor, labels: torch.Tensor,
                    dropout: float = 0.0, rng=None) -> torch.Tensor:
        """Mean cross entropy of the tokens with a label (the others have -100)."""
        y = self.states(tokens, offsets, dropout, rng)
        loss = ms.linear_cross_entropy(y, self.table.to(y.dtype), labels, scale=y.shape[-1] ** -0.5)
        return loss.sum() / (labels >= 0).sum()


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


def masked_batch(n: int, vocab: int, rng: torch.Generator):
    """Documents with 15 in 100 tokens replaced by token 0, and labels for those alone. A document is a
    walk along one permutation of the vocabulary, so that a token tells its neighbours."""
    lengths = torch.randint(20, 181, (n,), generator=rng)
    after = torch.randperm(vocab, generator=torch.Generator().manual_seed(4))
    walk = torch.empty(int(lengths.max()), n, dtype=torch.int64)
    walk[0] = torch.randint(vocab, (n,), generator=rng)
    for i in range(1, len(walk)):
        walk[i] = after[walk[i - 1]]
    docs = torch.cat([walk[:k, i] for i, k in enumerate(lengths.tolist())])
    out = torch.rand(len(docs), generator=rng) < 0.15
    labels = torch.where(out, docs, torch.full_like(docs, -100))
    return torch.where(out, torch.zeros_like(docs), docs).cuda(), offsets_of(lengths), labels.cuda()


def learn_masked(encoder: Encoder, steps: int, docs: int = 32, vocab: int = 300, dropout: float = 0.1,
                 report=print):
    """The losses of the steps, which change the encoder."""
    rng = torch.Generator().manual_seed(5)
    masks = torch.tensor([1234, 0], device="cuda")  # key and step of the dropout
    optimizer = torch.optim.AdamW(encoder.parameters(), lr=1e-3)  # the projection has no gradient
    losses = []
    for step in range(steps):
        loss = encoder.masked_loss(*masked_batch(docs, vocab, rng), dropout, masks)
        optimizer.zero_grad()
        loss.backward()
        ms.maxsim_clip_grad_norm([p.grad for p in encoder.parameters()], 1.0)
        optimizer.step()
        masks[1] += 1  # after the backward, which makes the step's masks again
        losses.append(float(loss.detach()))
        if step % 20 == 0 or step == steps - 1:
            report(f"masked step {step}: loss {losses[-1]:.3f}")
    return losses


def train(steps: int, docs: int = 32, query: int = 32, vocab: int = 300, max_norm: float = 1.0,
          report=print, masked: int = 0):
    """The losses of the steps, and the encoder, after `masked` steps of filling in tokens."""
    torch.manual_seed(0)
    rng = torch.Generator().manual_seed(1)
    encoder = Encoder(vocab).cuda()
    learn_masked(encoder, masked, docs, vocab, report=report)
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


class Index:
    """Documents' token vectors as they are, in 8 bits or in 4."""

    def __init__(self, D: torch.Tensor, offsets: torch.Tensor, kind: str = "bf16"):
        self.kind, self.offsets = kind, offsets
        self.stored = self.store(D)

    def store(self, x: torch.Tensor):
        if self.kind == "int8":
            # unit vectors: the norm scales them all alike, which changes no order
            return ms.maxsim_rms_norm_i8(x, torch.ones(x.shape[-1], device=x.device))[:2]
        return ms.maxsim_quantize_mx4(x) if self.kind == "mx4" else (x,)

    def scores(self, Q: torch.Tensor) -> torch.Tensor:
        score = {"bf16": ms.maxsim_score, "int8": ms.maxsim_score_i8, "mx4": ms.maxsim_score_mx4}[self.kind]
        return score(*self.store(Q), *self.stored, self.offsets)


@torch.no_grad()
def search(encoder: Encoder, docs: int = 200, query: int = 32, vocab: int = 300, k: int = 5,
           index: str = "bf16"):
    """How many of 20 queries find their document first among `docs`, and the last one's best k."""
    texts, doc_offsets, queries, _ = batch(docs, vocab, query, torch.Generator().manual_seed(2))
    store = Index(encoder(texts, doc_offsets), doc_offsets, index)
    one = offsets_of(torch.tensor([query]))
    found = 0
    for i in range(20):
        Q = encoder(queries[i * query:(i + 1) * query], one)
        scores, best = ms.maxsim_topk(store.scores(Q), k)
        found += int(best[0]) == i
    return found, best.tolist()


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--masked", type=int, default=0, help="steps of filling in tokens before")
    p.add_argument("--index", choices=["bf16", "int8", "mx4"], default="bf16")
    a = p.parse_args()
    _, encoder = train(a.steps, masked=a.masked)
    found, best = search(encoder, index=a.index)
    print(f"{found} of 20 queries find their document first among 200; the last one's best: {best}")


if __name__ == "__main__":
    main()
