"""A paged key-value cache and a small decoder on it: the serving operators run
together as a server runs them, with a Command for the elementwise part.

    python -m elementwise_tensor_commands_amd.decode [--steps N] [--beams N]

prefills a few prompts of different lengths in one packed batch, forks each into
beams, decodes with a beam search's reordering, ends a sequence, packs the live
pages together halfway, and prints the time of a step, eager and replayed from a
HIP graph.  Weights are random: it shows the calls, not a language.
"""
from __future__ import annotations

import argparse
import math
import sys

from . import (Command, page_assign, page_compact, page_copy, paged_attention, rope_append, rope_frequencies)


class PagedCache:
    """Keys and values of ``rows`` sequences in ``n`` pages of ``page`` slots, the
    same pages in every layer, with the tables that say whose they are.

    pages [rows, cols], lens [rows] and refs [n] are the current tables (int32, on
    the GPU).  Nothing here waits for the GPU or reads from it; ``stats`` holds
    what the last ``step`` (pages wanted, given) or ``compact`` (live, moved)
    counted, for a server that looks at it now and then."""

    def __init__(self, layers, n, page, heads, d, rows, cols, dv=None, dtype=None, device="cuda"):
        import torch
        dtype = dtype or torch.bfloat16

        def table(*shape, fill=0):
            return torch.full(shape, fill, dtype=torch.int32, device=device)

        self.page = page
        self.k = [torch.zeros(n, page, heads, d, dtype=dtype, device=device) for _ in range(layers)]
        self.v = [torch.zeros(n, page, heads, dv or d, dtype=dtype, device=device) for _ in range(layers)]
        self.pages, self.lens, self.refs = table(rows, cols, fill=-1), table(rows), table(n)
        self._pages, self._lens, self._refs = table(rows, cols, fill=-1), table(rows), table(n)
        self.src, self.dst = table(max(rows, n // 2)), table(max(rows, n // 2))
        self.stats = table(2)
        self.rows = rows

    def step(self, parent, add):
        """Every row takes over row parent[r]'s sequence (-1: starts empty) and
        grows by add[r] positions, whose slots the coming ``append`` fills."""
        src, dst = self.src[:self.rows], self.dst[:self.rows]
        page_assign(self.pages, self.lens, self.refs, parent, add, self.page, self._pages, self._lens, self.refs, src,
                    dst, self.stats)
        page_copy(self.k + self.v, src, dst)
        # copied back rather than swapped: a captured step finds them in their places
        self.pages.copy_(self._pages)
        self.lens.copy_(self._lens)

    def append(self, layer, q, k, v, pos, row, freq, q_out, layout="half"):
        """Turn q into q_out, and k and v into the slots of positions pos of rows row."""
        rope_append(q, k, v, pos, row, self.pages, freq, q_out, self.k[layer], self.v[layer], layout=layout)

    def attend(self, layer, q, out, pages=None, lens=None, window=0):
        """Attention of one query token a row over what the rows hold, or over other
        tables and lengths: a prompt's token t of row r has r's pages and length t + 1."""
        paged_attention(q, self.k[layer], self.v[layer], self.pages if pages is None else pages,
                        self.lens if lens is None else lens, out, window=window)

    def compact(self):
        """Move the live pages to the lowest ids (then the end of the pools is free)."""
        page_compact(self.pages, self.refs, self.pages, self._refs, self.src, self.dst, self.stats)
        page_copy(self.k + self.v, self.src, self.dst)
        self.refs.copy_(self._refs)


class Decoder:
    """A decoder of attention layers with random weights: x + attention(x) in each
    layer, the logits a product with the embedding."""

    def __init__(self, layers=2, vocab=1000, hq=8, hk=2, d=64, rows=12, n=256, page=16, cols=32, dtype=None, seed=0,
                 device="cuda"):
        import torch
        dtype = dtype or torch.bfloat16
        g = torch.Generator().manual_seed(seed)
        width = hq * d

        def weight(a, b):
            return (torch.randn(a, b, generator=g) / math.sqrt(a)).to(dtype).to(device)

        self.hq, self.hk, self.d, self.vocab = hq, hk, d, vocab
        self.embedding = torch.randn(vocab, width, generator=g).to(dtype).to(device)
        self.qkv = [weight(width, (hq + 2 * hk) * d) for _ in range(layers)]
        self.o = [weight(width, width) for _ in range(layers)]
        self.freq = rope_frequencies(d).to(device)
        self.cache = PagedCache(layers, n, page, hk, d, rows, cols, dtype=dtype, device=device)
        names = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float32: "f32"}
        self.add = Command()                       # out = x + y, in place in x
        x, y = self.add.load(names[dtype]), self.add.load(names[dtype])
        self.add.store(self.add.add(x, y))

    def forward(self, tokens, pos, row, pages=None, lens=None):
        """Logits [T, vocab] of T tokens at positions pos of rows row, whose slots the
        cache has; pages and lens: what each token attends to (by default token t is
        row t's newest)."""
        import torch
        hq, hk, d = self.hq, self.hk, self.d
        x = self.embedding[tokens]
        for layer in range(len(self.o)):
            h = torch.matmul(x, self.qkv[layer]).view(len(tokens), hq + 2 * hk, d)
            q, k, v = h[:, :hq], h[:, hq:hq + hk], h[:, hq + hk:]
            self.cache.append(layer, q, k, v, pos, row, self.freq, q)          # q turned in place
            out = torch.empty(len(tokens), hq, d, dtype=x.dtype, device=x.device)
            self.cache.attend(layer, q, out, pages, lens)
            y = torch.matmul(out.view(len(tokens), hq * d), self.o[layer])
            self.add.launch(x.view(-1), y.view(-1), x.view(-1))
        return torch.matmul(x, self.embedding.t())

    def prefill(self, prompts):
        """Start row r with the tokens prompts[r] (rows without any, and rows beyond,
        are empty): one packed batch.  Returns the logits after the last token of each
        prompt that has one."""
        import torch
        c, device = self.cache, self.embedding.device
        count = [len(p) for p in prompts]
        room = c.pages.shape[1] * c.page
        if len(count) > c.rows or max(count, default=0) > room:
            raise ValueError("%d prompts of up to %d tokens: there is room for %d of %d" % (
                len(count), max(count, default=0), c.rows, room))
        whole = count + [0] * (c.rows - len(count))

        def ints(a):
            return torch.tensor(a, dtype=torch.int32, device=device)

        c.step(ints([-1] * c.rows), ints(whole))
        row = ints([r for r, p in enumerate(prompts) for _ in p])
        pos = ints([i for p in prompts for i in range(len(p))])
        tokens = torch.tensor([t for p in prompts for t in p], dtype=torch.int64, device=device)
        # a token attends to its own row's pages up to itself
        logits = self.forward(tokens, pos, row, c.pages[row.long()], pos + 1)
        ends, at = [], 0
        for n in count:
            at += n
            if n:
                ends.append(at - 1)
        return logits[torch.tensor(ends, dtype=torch.int64, device=device)]

    def decode(self, tokens, parent, alive):
        """One step of every row: row r goes on from row parent[r] with tokens[r]
        (int64); rows where alive [rows] (int32) is 0 end.  A row whose table is full
        keeps what it has: its token sees that, and is not written.  Returns the logits."""
        import torch
        c = self.cache
        parent = torch.where((alive > 0) & (parent < c.rows), parent, -1)
        pos = torch.where(parent >= 0, c.lens[parent.clamp(min=0).long()], 0)
        c.step(parent, alive)
        rows = torch.arange(c.rows, dtype=torch.int32, device=tokens.device)
        return self.forward(tokens, pos, torch.where(c.lens > pos, rows, -1))


def next_beams(logits, alive, beams):
    """A beam search's choice in every group of ``beams`` rows: all of them go on from
    the group's row that scored highest of those alive, the i-th with its i-th best
    token.  Returns the parents [rows] (int32) and tokens [rows] (int64)."""
    import torch
    score = logits.amax(-1).masked_fill(alive == 0, -math.inf).view(-1, beams)
    best = torch.arange(0, len(logits), beams, device=logits.device) + score.argmax(-1)
    left, tokens = logits[best], []
    for _ in range(beams):
        tokens.append(left.argmax(-1))
        left = left.scatter(-1, tokens[-1][:, None], -math.inf)
    return best.repeat_interleave(beams).to(torch.int32), torch.stack(tokens, 1).flatten()


PROMPTS = (37, 120, 5, 64)      # tokens


def arguments(argv):
    """(steps of each half, eager and replayed; beams; table columns, of 16 positions,
    that hold the longest sequence)."""
    def positive(text):
        if int(text) < 1:
            raise ValueError
        return int(text)

    ap = argparse.ArgumentParser(prog="decode", description="A small decoder on the serving operators: times of a step.")
    ap.add_argument("--steps", type=positive, default=64, help="decode steps, half of them replayed from a graph")
    ap.add_argument("--beams", type=positive, default=4, help="beams of each of %d prompts" % len(PROMPTS))
    a = ap.parse_args(argv)
    return (a.steps + 1) // 2, a.beams, max(32, -(-(max(PROMPTS) + 1 + 2 * ((a.steps + 1) // 2)) // 16))


def main(argv):
    import torch
    half, beams, cols = arguments(argv)
    rows = len(PROMPTS) * beams
    m = Decoder(rows=rows, n=rows * (cols + 1), cols=cols)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, m.vocab, (n,), generator=g).tolist() for n in PROMPTS]
    # a prompt fills the first beam of its group; the others fork from it at the first step
    m.prefill([prompts[r // beams] if r % beams == 0 else [] for r in range(rows)])
    alive = torch.ones(rows, dtype=torch.int32, device="cuda")
    parent = torch.arange(rows, dtype=torch.int32, device="cuda") // beams * beams     # each row's group's first
    tokens = torch.randint(0, m.vocab, (rows,), generator=g).cuda()

    def step():
        p, t = next_beams(m.decode(tokens, parent, alive), alive, beams)
        parent.copy_(p)
        tokens.copy_(t)

    def timed(name, f, n):
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            f()
        b.record()
        torch.cuda.synchronize()
        print("%s: %.1f us a step" % (name, a.elapsed_time(b) / n * 1e3), flush=True)

    step()
    timed("eager", step, half)
    alive[rows - 1] = 0                            # one sequence ends
    m.cache.compact()
    print("live pages %d, moved %d" % tuple(m.cache.stats.tolist()), flush=True)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    timed("replayed", graph.replay, half)
    print("lengths", m.cache.lens.tolist())
    return 0


if __name__ == "__main__":
    sys.exit(main(sys.argv[1:]))
