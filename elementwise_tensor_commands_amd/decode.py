"""A paged key-value cache and a small decoder on it: the serving operators run
together as a server runs them, with a Command for the elementwise part.

    python -m elementwise_tensor_commands_amd.decode [--steps N] [--beams N]

prefills a few prompts of different lengths in one packed batch, forks each into
beams, decodes with a beam search's reordering, ends a sequence, packs the live
pages together halfway, and prints the time of a step, eager and replayed from a
HIP graph.  Weights are random: it shows the calls, not a language.

A ``Decoder`` also checks trees of drafted tokens (``verify``), reads only the pages
that a query may care for (``decode(take=...)``) and keeps rows within a budget of
pages (``decode(budget=...)``).
"""
from __future__ import annotations

import argparse
import math
import sys

from . import (Command, page_assign, page_bounds, page_compact, page_copy, page_evict, page_mass, page_select,
               paged_attention, rope, rope_append, rope_frequencies, slot_move, tree_accept, tree_attention)


class PagedCache:
    """Keys and values of ``rows`` sequences in ``n`` pages of ``page`` slots, the
    same pages in every layer, with the tables that say whose they are.

    pages [rows, cols], lens [rows] and refs [n] are the current tables (int32, on
    the GPU).  Nothing here waits for the GPU or reads from it; ``stats`` holds
    what the last ``step`` (pages wanted, given) or ``compact`` (live, moved)
    counted, for a server that looks at it now and then.

    select: the least and largest keys of every page are kept too (by ``bound``, after every
    append), for ``attend_some``; weigh: the weight that attention gave to every column of the
    tables, for ``evict``."""

    def __init__(self, layers, n, page, heads, d, rows, cols, dv=None, dtype=None, device="cuda", select=False, weigh=False):
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
        # a page's bounds are copied with it
        self.bounds = [torch.zeros(n, heads, 2, d, dtype=dtype, device=device) for _ in range(layers if select else 0)]
        self.mass = torch.zeros(rows, cols, device=device) if weigh else None
        self.count = table(rows)
        # as masses: of a row's columns the last are the least
        self.order = -torch.arange(cols, dtype=torch.float32, device=device).repeat(rows, 1)

    def step(self, parent, add):
        """Every row takes over row parent[r]'s sequence (-1, or what is no row: starts empty)
        and grows by add[r] positions, whose slots the coming ``append`` fills."""
        import torch
        src, dst = self.src[:self.rows], self.dst[:self.rows]
        page_assign(self.pages, self.lens, self.refs, parent, add, self.page, self._pages, self._lens, self.refs, src,
                    dst, self.stats)
        page_copy(self.k + self.v + self.bounds, src, dst)
        if self.mass is not None:
            from_row = (parent >= 0) & (parent < self.rows)
            self.mass.copy_(torch.where(from_row[:, None], self.mass[torch.where(from_row, parent, 0).long()], 0.0))
        # copied back rather than swapped: a captured step finds them in their places
        self.pages.copy_(self._pages)
        self.lens.copy_(self._lens)

    def append(self, layer, q, k, v, pos, row, freq, q_out, layout="half"):
        """Turn q into q_out, and k and v into the slots of positions pos of rows row."""
        rope_append(q, k, v, pos, row, self.pages, freq, q_out, self.k[layer], self.v[layer], layout=layout)

    def bound(self, layer, since):
        """Keep up the bounds of pages with positions since [rows] .. lens - 1, which were
        appended after the last call; nothing without ``select``."""
        if self.bounds:
            page_bounds(self.k[layer], self.pages, self.lens, since, self.bounds[layer])

    def attend(self, layer, q, out, pages=None, lens=None, window=0):
        """Attention of one query token a row over what the rows hold, or over other
        tables and lengths: a prompt's token t of row r has r's pages and length t + 1."""
        paged_attention(q, self.k[layer], self.v[layer], self.pages if pages is None else pages,
                        self.lens if lens is None else lens, out, window=window)

    def attend_some(self, layer, q, out, since, take):
        """``attend`` over the ``take`` pages of each row and kv head that q may care for
        most; since [rows]: the positions from there on were appended after the last ``bound``."""
        import torch
        heads = self.k[layer].shape[2]
        self.bound(layer, since)
        pages = torch.empty(self.rows, heads, take, dtype=torch.int32, device=q.device)
        lens = torch.empty(self.rows, heads, dtype=torch.int32, device=q.device)
        page_select(q, self.bounds[layer], self.pages, self.lens, self.page, pages, lens, first=min(1, take - 1), last=1)
        paged_attention(q, self.k[layer], self.v[layer], pages, lens, out)

    def attend_weighed(self, layer, q, out, decay=1.0):
        """``attend`` that adds the weight every page got to ``decay`` times what it had."""
        import torch
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        paged_attention(q, self.k[layer], self.v[layer], self.pages, self.lens, out, lse=lse)
        page_mass(q, self.k[layer], self.pages, self.lens, lse, self.mass, self.mass, decay=decay)

    def evict(self, budget):
        """Take the pages of least weight out of rows that hold more than budget [rows],
        but for the first and the last; ``count`` says how many."""
        page_evict(self.pages, self.lens, self.refs, self.mass, budget, self.page, self.pages, self.refs, self.count,
                   first=1, last=1)

    def attend_tree(self, layer, q, parent, lens, out):
        """Attention of trees of tokens, q [rows, T, hq, d], that lie at positions lens + i."""
        tree_attention(q, self.k[layer], self.v[layer], self.pages, lens, parent, out)

    def keep(self, path, old, lens):
        """Of the tokens at positions old + i keep those of a path: they move to old, old +
        1, ..., rows end at lens, and the pages past that are free again.  (Rejected keys
        never enter the bounds: these are kept up from here.)"""
        slot_move(self.k + self.v, self.pages, old, path)
        import torch
        # as many pages as they hold up to there (holes hold none): the last ones go
        budget = ((self.pages >= 0) & (-self.order < (lens + (self.page - 1))[:, None] // self.page)).sum(1, dtype=torch.int32)
        page_evict(self.pages, self.lens, self.refs, self.order, budget, self.page, self.pages, self.refs, self.count,
                   first=0, last=0)
        self.lens.copy_(lens)
        for layer in range(len(self.bounds)):
            self.bound(layer, old)

    def compact(self):
        """Move the live pages to the lowest ids (then the end of the pools is free)."""
        page_compact(self.pages, self.refs, self.pages, self._refs, self.src, self.dst, self.stats)
        page_copy(self.k + self.v + self.bounds, self.src, self.dst)
        self.refs.copy_(self._refs)


class Decoder:
    """A decoder of attention layers with random weights: x + attention(x) in each
    layer, the logits a product with the embedding."""

    def __init__(self, layers=2, vocab=1000, hq=8, hk=2, d=64, rows=12, n=256, page=16, cols=32, dtype=None, seed=0,
                 device="cuda", select=False, weigh=False):
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
        self.cache = PagedCache(layers, n, page, hk, d, rows, cols, dtype=dtype, device=device, select=select, weigh=weigh)
        names = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float32: "f32"}
        self.add = Command()                       # out = x + y, in place in x
        x, y = self.add.load(names[dtype]), self.add.load(names[dtype])
        self.add.store(self.add.add(x, y))

    def forward(self, tokens, pos, row, pages=None, lens=None, attend=None):
        """Logits [T, vocab] of T tokens at positions pos of rows row, whose slots the
        cache has; pages and lens: what each token attends to (by default token t is
        row t's newest); attend(layer, q, out) in place of the cache's."""
        import torch
        hq, hk, d = self.hq, self.hk, self.d
        x = self.embedding[tokens]
        for layer in range(len(self.o)):
            h = torch.matmul(x, self.qkv[layer]).view(len(tokens), hq + 2 * hk, d)
            q, k, v = h[:, :hq], h[:, hq:hq + hk], h[:, hq + hk:]
            self.cache.append(layer, q, k, v, pos, row, self.freq, q)          # q turned in place
            out = torch.empty(len(tokens), hq, d, dtype=x.dtype, device=x.device)
            if attend is None:
                self.cache.attend(layer, q, out, pages, lens)
            else:
                attend(layer, q, out)
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
        for layer in range(len(c.bounds)):
            c.bound(layer, ints([0] * c.rows))
        ends, at = [], 0
        for n in count:
            at += n
            if n:
                ends.append(at - 1)
        return logits[torch.tensor(ends, dtype=torch.int64, device=device)]

    def decode(self, tokens, parent, alive, take=0, budget=None):
        """One step of every row: row r goes on from row parent[r] with tokens[r]
        (int64); rows where alive [rows] (int32) is 0 end.  A row whose table is full
        keeps what it has: its token sees that, and is not written.  take: how many pages of
        each kv head are read (0: all; of a decoder with ``select``).  budget [rows]
        (int32; of one with ``weigh``, and not with take): how many pages a row keeps after it.
        Returns the logits."""
        import torch
        c = self.cache
        if take and budget is not None:
            raise ValueError("take and budget: pages that a step does not read get no weight to keep them by")
        if take < 0:
            raise ValueError("take is a number of pages, or 0")
        if take and not c.bounds:
            raise ValueError("take is of a decoder with select")
        if budget is not None and c.mass is None:
            raise ValueError("budget is of a decoder with weigh")
        parent = torch.where((alive > 0) & (parent < c.rows), parent, -1)
        pos = torch.where(parent >= 0, c.lens[parent.clamp(min=0).long()], 0)
        c.step(parent, alive)
        rows = torch.arange(c.rows, dtype=torch.int32, device=tokens.device)

        def attend(layer, q, out):
            if take:
                c.attend_some(layer, q, out, pos, take)
                return
            c.bound(layer, pos)
            if budget is None:
                c.attend(layer, q, out)
            else:
                c.attend_weighed(layer, q, out, 0.9 if layer == 0 else 1.0)

        logits = self.forward(tokens, pos, torch.where(c.lens > pos, rows, -1), attend=attend)
        if budget is not None:
            c.evict(budget)
        return logits

    def verify(self, tokens, parent, alive):
        """One step that checks a tree of drafted tokens in every row: tokens [rows, T]
        (int32, T <= 256), token 0 the row's newest, which ``decode`` would be given; token
        i > 0 a guess of what follows token parent[r, i] < i (int32; -1 for token 0, any other
        number: padding).  Rows keep the longest path of guesses that are what the model goes
        on with (greedily) and lose the others; guesses may begin alike.  Rows where alive is 0
        end.  A token without a slot, since the table is full or no page was free, is padding:
        a row that has none for token 0 stays as it is.  Returns path [rows, T] (the tokens
        kept, ascending, then -1: none of a row that stays or has ended) and last [rows], the
        next newest (-1 of those).  (The weights of a decoder with ``weigh`` are those of
        ``decode`` with a budget alone.)"""
        import torch
        c, device = self.cache, tokens.device
        rows, t = tokens.shape
        if t > 256 or rows != c.rows:
            raise ValueError("trees of up to 256 tokens in each of %d rows, got %s" % (c.rows, tuple(tokens.shape)))
        parent = parent.expand(rows, t)
        hq, hk, d = self.hq, self.hk, self.d
        every = torch.arange(rows, dtype=torch.int32, device=device)
        old = torch.where(alive > 0, c.lens, 0)
        c.step(torch.where(alive > 0, every, -1), alive * t)
        slot = old[:, None] + torch.arange(t, dtype=torch.int32, device=device)
        # rows that have ended, and tokens without a slot (the table is full, or no page was free), are padding
        there = (alive > 0)[:, None] & (slot < c.pages.shape[1] * c.page)
        there &= c.pages.gather(1, torch.where(there, slot // c.page, 0).long()) >= 0
        parent = torch.where(there, parent, -2)
        parent, depth = tree_depths(parent)
        parent = merge_alike(tokens, parent)
        pos, slot = (old[:, None] + depth).view(1, -1), slot.reshape(-1)
        row = torch.where(parent >= -1, every[:, None], -1).view(-1)
        x = self.embedding[torch.where(parent >= -1, tokens, 0).view(-1).long()]    # (padding's may be anything)
        for layer in range(len(self.o)):
            h = torch.matmul(x, self.qkv[layer]).view(rows * t, hq + 2 * hk, d)
            turned = h[None, :, :hq + hk]
            rope(turned, pos, self.freq, turned)    # by its depth; its slot is another place
            q, k, v = h[:, :hq], h[:, hq:hq + hk], h[:, hq + hk:]
            c.append(layer, q, k, v, slot, row, self.freq[:0], q)
            out = torch.empty(rows, t, hq, d, dtype=x.dtype, device=device)
            c.attend_tree(layer, q.unflatten(0, (rows, t)), parent, old, out)
            y = torch.matmul(out.view(rows * t, hq * d), self.o[layer])
            self.add.launch(x.view(-1), y.view(-1), x.view(-1))
        follow = torch.matmul(x, self.embedding.t()).argmax(-1).to(torch.int32).view(rows, t)
        path, lens, last = torch.empty_like(parent), torch.empty_like(old), torch.empty_like(old)
        tree_accept(tokens, parent, follow, old, path, lens, last)
        c.keep(path, old, lens)
        return path, last


def tree_depths(parent):
    """Of trees given by parents [rows, T] (int32): the same with -2 for every token that is
    padding, as ``tree_attention`` takes it (its parent is neither -1 nor a token before it, or
    it is below such a one), and how many tokens of its tree are above each."""
    import torch
    t = parent.shape[1]
    parent = torch.where((parent >= -1) & (parent < torch.arange(t, device=parent.device)), parent, -2)
    depth, up = (parent >= 0).to(torch.int32), parent.long()
    for _ in range(t.bit_length()):                 # steps up the tree, doubling
        at = up.clamp(min=0)
        depth = depth + torch.where(up >= 0, depth.gather(1, at), 0)
        up = torch.where(up >= 0, up.gather(1, at), up)
    return torch.where(up == -2, -2, parent), depth


def merge_alike(tokens, parent):
    """Parents [rows, T] (of ``tree_depths``) with tokens merged whose paths from the root on are
    alike: what is below such a token follows the first of them, and the others are padding.
    Then a token's followers differ, and only one of them can be right."""
    import torch
    t = parent.shape[1]
    up, real = parent.long(), parent > -2
    # alike[r, i, j]: the last 1, 2, 4, ... tokens of the paths to i and j are the same, or all of both
    alike = (tokens[:, :, None] == tokens[:, None]) & real[:, :, None] & real[:, None]
    for _ in range(t.bit_length()):
        at, more = up.clamp(min=0), up >= 0
        above = alike.gather(1, at[:, :, None].expand(-1, -1, t)).gather(2, at[:, None].expand(-1, t, -1))
        alike = alike & torch.where(more[:, :, None] & more[:, None], above, more[:, :, None] == more[:, None])
        up = torch.where(more, up.gather(1, at), up)
    first = (torch.arange(t, 0, -1, dtype=torch.int32, device=parent.device) * alike).argmax(2) if t else parent.long()
    merged = torch.where(parent >= 0, first.gather(1, parent.clamp(min=0).long()), parent).to(parent.dtype)
    return torch.where(real & (first != torch.arange(t, device=parent.device)), -2, merged)


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
