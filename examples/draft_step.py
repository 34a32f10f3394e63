"""Drafted decoding with the library's operators, on a small model with random weights.

    python examples/draft_step.py

A prompt is read into a paged cache; then tokens are decoded one by one, and once
more by checking drafted trees of tokens, several of them a step.  Both ways give
the same text.  A layer is

    q, k, v = w4_linear(norm(x));  q = rotary_append(...);  a = tree_attention(...)
    x += w4_linear(a);  x += decode_layer(down, relu(w4_linear(norm(x))))

with the last product on a sparse matrix in the dual-view blocked format, and the
logits go through penalize_logits.
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dynamic_sparsity_spmspv_gb300 as dbs  # noqa: E402

DT, DEV = torch.float16, "cuda"
HIDDEN, HEADS, KV_HEADS, DIM, FFN, VOCAB, LAYERS, GROUP = 512, 8, 2, 64, 1024, 2051, 2, 64
PAGE, PAGES = 16, 24


class CSR:
    """A random sparse matrix, a tenth of it filled."""

    def __init__(self, rng, m, n):
        full = np.where(rng.random((m, n)) < 0.1, rng.normal(0, (0.1 * n)**-0.5, (m, n)), 0).astype(np.float32)
        rows, cols = np.nonzero(full)
        self.m, self.n, self.vals, self.col_idx = m, n, full[rows, cols], cols.astype(np.int32)
        self.row_ptr = np.concatenate([[0], np.cumsum(np.bincount(rows, minlength=m))]).astype(np.int64)


class Linear:
    """4-bit weights with a scale for each group of inputs."""

    def __init__(self, rng, m, n):
        self.codes = torch.from_numpy(rng.integers(0, 256, (m, n // 2)).astype(np.uint8)).to(DEV)
        self.scales = torch.from_numpy(rng.uniform(0.15, 0.25, (m, n // GROUP)).astype(np.float32)).to(DEV, DT) * n**-0.5

    def __call__(self, x):
        return dbs.w4_linear(x, self.codes, self.scales, group=GROUP)


def norm(x):
    f = x.float()
    return (f * (f.square().mean(-1, keepdim=True) + 1e-6).rsqrt()).to(DT)


class Model:
    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        self.embedding = torch.from_numpy(rng.normal(0, 1, (VOCAB, HIDDEN))).to(DEV, DT)
        self.table = dbs.rotary_table(PAGE * PAGES, DIM)
        self.layers = []
        for _ in range(LAYERS):
            down = dbs.DBMatrix.from_csr(CSR(rng, HIDDEN, FFN))
            self.layers.append((Linear(rng, (HEADS + 2 * KV_HEADS) * DIM, HIDDEN), Linear(rng, HIDDEN, HEADS * DIM),
                                Linear(rng, FFN, HIDDEN), down, dbs.Workspace(down)))
        self.head = Linear(rng, VOCAB, HIDDEN)


class Sequence:
    """The tokens of one text and its cache: pages in an order of their own."""

    def __init__(self, model, prompt, seed):
        self.model, self.tokens, self.prompt = model, [], len(prompt)
        self.pages = torch.from_numpy(np.random.default_rng(seed).permutation(PAGES).astype(np.int32)).to(DEV)[None]
        shape = (PAGES, PAGE, KV_HEADS, DIM)
        self.cache = [(torch.zeros(shape, dtype=DT, device=DEV), torch.zeros(shape, dtype=DT, device=DEV)) for _ in range(LAYERS)]
        self.step(prompt[:-1], list(range(-1, len(prompt) - 2)))            # a chain: each token's parent is the one before
        self.tokens = list(prompt[:-1])
        self.last = prompt[-1]

    def entries(self, at):
        """Cache entries of positions in the text."""
        at = torch.as_tensor(at, device=DEV)
        return (self.pages[0, at // PAGE] * PAGE + at % PAGE).to(torch.int32)

    def step(self, tokens, parents):
        """Logits [tokens, vocab] of drafted tokens, each with a parent among them (-1: the text).  They are in the cache
        behind the text, in their order."""
        m, n, before = self.model, len(tokens), len(self.tokens)
        paths = []
        for t, p in enumerate(parents):
            paths.append((paths[p] if p >= 0 else []) + [t])
        bits = np.zeros((1, n, (n + 63) // 64), np.uint64)
        for t, path in enumerate(paths):
            for i in path:
                bits[0, t, i // 64] |= np.uint64(1) << np.uint64(i % 64)
        tree = torch.from_numpy(bits.view(np.int64)).to(DEV)
        positions = torch.tensor([before + len(p) - 1 for p in paths], dtype=torch.int32, device=DEV)
        slots = self.entries(np.arange(before, before + n))
        lens = torch.tensor([before + n], dtype=torch.int32, device=DEV)

        x = m.embedding[torch.tensor(tokens, device=DEV)]
        for (qkv, out, up, down, ws), (kc, vc) in zip(m.layers, self.cache):
            q, k, v = qkv(norm(x)).unflatten(1, (-1, DIM)).split([HEADS, KV_HEADS, KV_HEADS], 1)
            q = dbs.rotary_append(q, k, v, m.table, positions, kc, vc, slots)
            a = dbs.tree_attention(q[None], kc, vc, lens, tree, page_table=self.pages)
            x = x + out(a[0].flatten(1))
            f = up(norm(x)).relu().float()
            x = x + torch.stack([dbs.decode_layer(down, row, 0.0, ws=ws) for row in f]).to(DT)
        logits = m.head(norm(x))

        # the tokens up to and with each drafted one
        seen = [self.tokens + [tokens[i] for i in path] for path in paths]
        history = torch.full((n, max(map(len, seen))), -1, dtype=torch.int32)
        for t, s in enumerate(seen):
            history[t, :len(s)] = torch.tensor(s, dtype=torch.int32)
        rows = torch.ones(n, device=DEV)
        return dbs.penalize_logits(logits, history=history.to(DEV), history_lens=torch.tensor([len(s) for s in seen], dtype=torch.int32, device=DEV),
                                   prompt_lens=torch.full((n,), self.prompt, dtype=torch.int32, device=DEV), repetition=1.1 * rows,
                                   frequency=0.05 * rows)

    def keep(self, path):
        """Takes the drafted tokens on `path` into the text: their entries move to its end."""
        before = len(self.tokens)
        src, dst = self.entries([before + t for t in path]).long(), self.entries([before + i for i in range(len(path))]).long()
        for pair in self.cache:
            for c in pair:
                flat = c.view(-1, KV_HEADS, DIM)
                flat[dst] = flat[src]

    def advance(self, drafts, parents):
        """One step: the last token and drafted ones behind it (a parent of 0: the last token).  Returns the tokens that
        follow, one more than were drafted rightly, and the logits that chose them."""
        tokens = [self.last] + drafts
        logits = self.step(tokens, [-1] + parents)
        best = logits.argmax(-1).tolist()
        path = [0]
        while True:
            next_ = [t for t, p in enumerate(parents, 1) if p == path[-1] and tokens[t] == best[path[-1]]]
            if not next_:
                break
            path.append(next_[0])
        self.keep(path)
        self.tokens += [tokens[t] for t in path]
        self.last = best[path[-1]]
        return [best[t] for t in path], logits[path]


def main(count=24):
    model, prompt = Model(1), np.random.default_rng(2).integers(0, VOCAB, 40).tolist()
    single, text, logits = Sequence(model, prompt, 3), [], []
    while len(text) < count:
        t, l = single.advance([], [])
        text += t
        logits.append(l)

    # Trees of a main line, drafted from the text just found (a guess in four is wrong), with a wrong sibling at each token.
    rng, drafted, got, steps = np.random.default_rng(4), Sequence(model, prompt, 5), [], 0
    got_logits = []
    while len(got) < count:
        drafts, parents, at = [], [], 0
        for right in text[len(got):len(got) + 5]:
            drafts += [(right + 1) % VOCAB, right if rng.random() < 0.75 else (right + 2) % VOCAB]
            parents += [at, at]
            at = len(drafts)
        t, l = drafted.advance(drafts, parents)
        got += t
        got_logits.append(l)
        steps += 1
    got_logits, logits = torch.cat(got_logits)[:count], torch.cat(logits)
    print(f"{count} tokens one by one, and in {steps} steps of drafted trees: {'the same' if got[:count] == text else 'another'} text")
    return text, got[:count], steps, logits, got_logits


if __name__ == "__main__":
    main()
