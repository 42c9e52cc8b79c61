"""Cases of the serving operators: rotary positions, rotary positions with the
write into a paged key-value cache, attention of one new token over that cache,
and the bookkeeping of its pages (assign, compact, copy).

``run`` computes one call in elementary torch operations (``own`` False) or
through the library (``own`` True) on what ``prepare`` made; ``exact`` is the
operators' definition in 64 bits, written apart from both.

The cache: k_cache [N, page, kv heads, d], v_cache [N, page, kv heads, dv]; row
r of a batch holds positions 0 .. lens[r] - 1, position p in slot p % page of
cache page pages[r, p // page].  An id outside 0 .. N - 1 is a hole: nothing is
written there and its positions take no part in attention.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases.

def listed():
    return [
        # The query and key heads of a packed projection, rotated in one call for a batch of prompts.
        dict(name="rope_prompt", op="rope", b=4, t=4096, h=40, d=128, r=128, extra=8, layout="half", dtype="bf16",
             inverse=False, far=0, mscale=1.0),
        # The gradient through a partly rotated head of odd width, at positions a million tokens in.
        dict(name="rope_grad", op="rope", b=2, t=511, h=12, d=81, r=40, extra=0, layout="interleaved", dtype="f32",
             inverse=True, far=1000003, mscale=1.1),
        # One decode step of 64 sequences: every row's new token into the cache.
        dict(name="append_token", op="append", rows=64, top=1, hq=32, hk=8, d=128, dv=128, r=128, page=16, p=64,
             layout="half", dtype="bf16", pad=0),
        # Ragged prompts of 16 sequences packed into one batch, with padding tokens.
        dict(name="append_prompt", op="append", rows=16, top=1000, hq=32, hk=4, d=128, dv=96, r=64, page=32, p=48,
             layout="interleaved", dtype="f16", pad=37),
        # One sequence's next token: the smallest call of a decode loop.
        dict(name="attn_token", op="attention", b=1, hq=32, hk=8, d=128, dv=128, page=16, top=777, window=0,
             dtype="bf16"),
        # A serving batch with lengths from nothing to 8192.
        dict(name="attn_batch", op="attention", b=64, hq=32, hk=8, d=128, dv=128, page=16, top=8192, window=0,
             dtype="bf16"),
        # Two long documents: few rows, everything along the cache.
        dict(name="attn_long", op="attention", b=2, hq=16, hk=2, d=128, dv=128, page=64, top=262143, window=0,
             dtype="f16"),
        # One key head a query head, odd sizes, and a window whose older pages have been given back.
        dict(name="attn_window", op="attention", b=9, hq=12, hk=12, d=80, dv=64, page=17, top=4095, window=1000,
             dtype="f32"),
        # A beam search's step: 8 requests of 4 beams, states reordered, the partial pages copied.
        dict(name="fork_beams", op="fork", groups=8, width=4, p=64, page=16, h=2, d=64, n=2048, share=30, busy=1.0,
             prompt=0, dtype="bf16"),
        # A server's step: most rows grow by one token, some fork, end or start with a prompt.
        dict(name="fork_serve", op="fork", groups=128, width=4, p=1024, page=8, h=2, d=64, n=131072, share=100,
             busy=0.2, prompt=500, dtype="bf16"),
        # Packing a small cache's live pages to its start.
        dict(name="compact_small", op="compact", rows=8, p=40, n=509, live=250, moves=120, page=16, h=2, d=64,
             dtype="f32"),
        # Packing a large one: a quarter of the pages move.
        dict(name="compact_large", op="compact", rows=128, p=192, n=32768, live=16384, moves=8192, page=16, h=4,
             d=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    layout = rng.choice(["half", "interleaved"])
    if op == "rope":
        b, t, d = _log(rng, 1, 8), _log(rng, 1, 4096), rng.choice([64, 64, 80, 96, 128, 128, rng.randint(33, 255)])
        h = max(1, min(_log(rng, 1, 40), 40000000 // (b * t * d)))
        r = rng.choice([d // 2 * 2, d // 2 * 2, rng.randint(1, d // 2) * 2])
        return dict(op=op, b=b, t=t, h=h, d=d, r=r, extra=rng.choice([0, 1, 8]), layout=layout, dtype=dtype,
                    inverse=rng.random() < 0.5, far=rng.choice([0, rng.randint(1000, 2000000)]),
                    mscale=rng.choice([1.0, 1.25]))
    hk = _log(rng, 1, 8)
    hq = hk * rng.choice([1, 2, 3, 4, 8, 16])
    d = rng.choice([64, 80, 96, 128, 128, 192, rng.randint(33, 200)])
    dv = rng.choice([d, d, 64, 128])
    page = rng.choice([1, 16, 16, 32, 64, rng.randint(2, 100)])
    if op == "append":
        rows, top = _log(rng, 1, 64), rng.choice([1, _log(rng, 2, 400)])
        p = -(-max(2 * top, rng.randint(64, 512)) // page)
        while rows * p * page * hk * max(d, dv) > 60000000 and rows > 1:
            rows = (rows + 1) // 2
        return dict(op=op, rows=rows, top=top, hq=hq, hk=hk, d=d, dv=dv, r=rng.choice([d // 2 * 2, d // 4 * 2]),
                    page=page, p=p, layout=layout, dtype=dtype, pad=rng.choice([0, rng.randint(1, 50)]))
    if op == "attention":
        b, top = _log(rng, 1, 64), _log(rng, 1, 65536)
        while b * top * hk * (d + dv) * (2 if dtype == "f32" else 1) > 500000000:
            b, top = max(1, b // 2), (top + 1) // 2
        return dict(op=op, b=b, hq=hq, hk=hk, d=d, dv=dv, page=page, top=top,
                    window=rng.choice([0, 0, rng.randint(1, top)]), dtype=dtype)
    if op == "fork":
        p, page = _log(rng, 8, 1024), rng.choice([4, 8, 16])
        groups, width = _log(rng, 1, 128), rng.randint(1, 6)
        n = _log(rng, 512, 131072)
        share = min(p // 2, n // (2 * groups * width))
        return dict(op=op, groups=groups, width=width, p=p, page=page, h=2, d=rng.choice([32, 64]), n=n, share=share,
                    busy=rng.uniform(0.1, 1.0), prompt=rng.randint(0, p * page // 4), dtype=dtype)
    n = _log(rng, 256, 32768)
    live = rng.randint(n // 8, n - n // 8)
    rows = _log(rng, 1, 128)
    return dict(op=op, rows=rows, p=-(-live // rows) + rng.randint(0, 40), n=n, live=live,
                moves=rng.randint(0, min(live, n - live)), page=rng.choice([8, 16]), h=rng.choice([1, 2, 4]),
                d=rng.choice([64, 80, 128]) // (2 if dtype == "f32" else 1), dtype=dtype)


# ---------------------------------------------------------------------------
# What a case's name alone decides: lengths and who forks from whom.

def _rng(case):
    return random.Random(" ".join("%s=%s" % kv for kv in sorted(case.items()) if kv[0] != "name"))


def _lens(case, b, top):
    """Lengths of b rows: the first the longest, one of four or more empty, the others spread."""
    rng = _rng(case)
    lens = [top] + [rng.randint(1, top) for _ in range(b - 1)]
    if b >= 4:
        lens[b // 2] = 0
    return lens


def _fork_plan(case):
    """Lengths before the step, parents and new tokens of every row."""
    rng = _rng(case)
    rows, page = case["groups"] * case["width"], case["page"]
    most = case["share"] * page
    lens, parent, add = [], [], []
    for g in range(case["groups"]):
        own_len = rng.randint(1, max(1, most))
        for w in range(case["width"]):
            r = g * case["width"] + w
            lens.append(own_len)
            busy = rng.random() < case["busy"]
            kind = rng.random()
            if not busy or kind < 0.2:
                parent.append(r)
            elif kind < 0.8:
                parent.append(g * case["width"] + rng.randrange(case["width"]))
            else:
                parent.append(-1)
            add.append(1 if parent[r] >= 0 else rng.choice([0, case["prompt"]]))
    assert len(lens) == rows
    return lens, parent, add


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op == "rope":
        n = case["b"] * case["t"] * case["h"]
        return dict(bytes=2 * n * case["d"] * e + 4 * case["b"] * case["t"], flops=3 * n * case["r"])
    if op == "append":
        t = sum(_append_counts(case))
        per = case["hq"] * case["d"] + case["hk"] * (case["d"] + case["dv"])
        return dict(bytes=t * (2 * per * e + 8), flops=3 * t * (case["hq"] + case["hk"]) * case["r"])
    if op == "attention":
        w = case["window"]
        keys = sum(min(x, w) if w else x for x in _lens(case, case["b"], case["top"]))
        per = case["d"] + case["dv"]
        return dict(bytes=keys * case["hk"] * per * e + case["b"] * case["hq"] * (per * e + 4),
                    flops=2 * keys * case["hq"] * per)
    page_bytes = case["page"] * case["h"] * case["d"] * e
    if op == "fork":
        lens, parent, add = _fork_plan(case)
        rows = len(lens)
        copies = sum(1 for r in range(rows) if parent[r] not in (r, -1) and lens[parent[r]] % case["page"])
        return dict(bytes=8 * case["n"] + 8 * rows * case["p"] + 28 * rows + 4 * copies * page_bytes, flops=0)
    return dict(bytes=8 * case["n"] + 8 * case["rows"] * case["p"] + 4 * case["moves"] * page_bytes + 4 * case["n"],
                flops=0)


def _append_counts(case):
    """New tokens of each row, 1 to top."""
    rng = _rng(case)
    return [rng.randint((case["top"] + 1) // 2, case["top"]) for _ in range(case["rows"])]


# ---------------------------------------------------------------------------
# Inputs.

def _freq(r, base=10000.0):
    """Inverse frequencies of a rotary part of width r, in radians a position."""
    return torch.tensor([base ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64)


def _randn(g, *shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype) if np.prod(shape) < 1 << 22 \
        else torch.empty(shape, device="cuda", dtype=dtype).normal_(generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    pick = np.random.RandomState(seed & 0x7FFFFFFF)
    dt, op = DTYPES[case["dtype"]], case["op"]

    def ints(a):
        return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()

    s = dict(case=case)
    if op == "rope":
        b, t, h, d = case["b"], case["t"], case["h"], case["d"]
        packed = _randn(g, b, t, (h + case["extra"]) * d, dtype=dt)
        start = pick.randint(0, 50, size=(b, 1)) + case["far"]
        s.update(x=packed[:, :, :h * d].unflatten(2, (h, d)), pos=ints(start + np.arange(t)[None]),
                 freq=_freq(case["r"]).cuda(), out=torch.empty(b, t, h, d, dtype=dt, device="cuda"))
        return s
    if op == "append":
        rows, page, p = case["rows"], case["page"], case["p"]
        n = rows * p + 3
        pages = pick.permutation(n)[:rows * p].reshape(rows, p)
        row, pos = [], []
        for r, c in enumerate(_append_counts(case)):
            first = pick.randint(0, p * page - c + 1)
            row.append(np.full(c, r))
            pos.append(first + np.arange(c))
        row.append(np.full(case["pad"], -1))
        pos.append(np.zeros(case["pad"]))
        row, pos = np.concatenate(row), np.concatenate(pos)
        t, hq, hk, d, dv = len(row), case["hq"], case["hk"], case["d"], case["dv"]
        s.update(q=_randn(g, t, hq, d, dtype=dt), k=_randn(g, t, hk, d, dtype=dt), v=_randn(g, t, hk, dv, dtype=dt),
                 row=ints(row), pos=ints(pos), pages=ints(pages), freq=_freq(case["r"]).cuda(),
                 q_out=torch.empty(t, hq, d, dtype=dt, device="cuda"), k_cache=_randn(g, n, page, hk, d, dtype=dt),
                 v_cache=_randn(g, n, page, hk, dv, dtype=dt))
        return s
    if op == "attention":
        b, hq, hk, d, dv, page = (case[k] for k in ("b", "hq", "hk", "d", "dv", "page"))
        lens = _lens(case, b, case["top"])
        used = [-(-x // page) for x in lens]
        p = max(used) + 1
        n = sum(used) + 2
        ids = pick.permutation(n)
        pages, at = np.full((b, p), -1), 0
        for r in range(b):
            pages[r, :used[r]] = ids[at:at + used[r]]
            at += used[r]
            if case["window"]:                     # pages wholly before the window have been given back
                pages[r, :max(0, lens[r] - case["window"]) // page] = -1
        # queries of different sharpness: near-uniform weights in some heads, a few keys' in others
        sharp = torch.linspace(0.5, 3.0, hq, device="cuda")[:, None]
        s.update(q=(_randn(g, b, hq, d, dtype=torch.float32) * sharp).to(dt),
                 k_cache=_randn(g, n, page, hk, d, dtype=dt), v_cache=_randn(g, n, page, hk, dv, dtype=dt),
                 pages=ints(pages), lens=ints(lens), out=torch.empty(b, hq, dv, dtype=dt, device="cuda"),
                 lse=torch.empty(b, hq, dtype=torch.float32, device="cuda"))
        # a last page's unused slots hold whatever the memory held
        for r in range(b):
            if lens[r] % page:
                s["k_cache"][pages[r, lens[r] // page], lens[r] % page:] = math.nan
                s["v_cache"][pages[r, lens[r] // page], lens[r] % page:] = math.nan
        return s
    n, p, page, h, d = (case[k] for k in ("n", "p", "page", "h", "d"))
    if op == "fork":
        lens, parent, add = _fork_plan(case)
        rows = len(lens)
        pages, refs = np.full((rows, p), -1), np.zeros(n, np.int64)
        ids, at = pick.permutation(n), 0
        for r in range(rows):
            first, used = r - r % case["width"], -(-lens[r] // page)
            common = used // 2 if r != first else 0    # the first half came from a common prompt
            pages[r, :common] = pages[first, :common]
            pages[r, common:used] = ids[at:at + used - common]
            at += used - common
            refs[pages[r, :used]] += 1
        copies = rows
        s.update(lens=ints(lens), parent=ints(parent), add=ints(add),
                 lens_out=torch.empty(rows, dtype=torch.int32, device="cuda"))
    else:
        rows, live, moves = case["rows"], case["live"], case["moves"]
        ids = np.concatenate([pick.permutation(live)[:live - moves], live + pick.permutation(n - live)[:moves]])
        ids = pick.permutation(ids)
        pages, refs = np.full(rows * p, -1), np.zeros(n, np.int64)
        pages[:live] = ids
        extra = pick.randint(0, live, size=max(0, rows * p - live) // 3)       # shared pages
        pages[live:live + len(extra)] = ids[extra]
        np.add.at(refs, pages[pages >= 0], 1)
        pages = pick.permutation(pages).reshape(rows, p)
        copies = n // 2
    s.update(pages=ints(pages), refs=ints(refs), pools=[_randn(g, n, page, h, d, dtype=dt) for _ in range(2)],
             pages_out=torch.empty(rows, p, dtype=torch.int32, device="cuda"),
             refs_out=torch.empty(n, dtype=torch.int32, device="cuda"),
             src=torch.empty(copies, dtype=torch.int32, device="cuda"),
             dst=torch.empty(copies, dtype=torch.int32, device="cuda"),
             stats=torch.empty(2, dtype=torch.int32, device="cuda"))
    return s


# ---------------------------------------------------------------------------
# One pass.

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import elementwise_tensor_commands_amd as ecmd
    case = s["case"]
    op = case["op"]
    if op == "rope":
        ecmd.rope(s["x"], s["pos"], s["freq"], s["out"], layout=case["layout"], mscale=case["mscale"],
                  inverse=case["inverse"])
        return s["out"]
    if op == "append":
        ecmd.rope_append(s["q"], s["k"], s["v"], s["pos"], s["row"], s["pages"], s["freq"], s["q_out"], s["k_cache"],
                         s["v_cache"], layout=case["layout"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "attention":
        ecmd.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["lens"], s["out"], lse=s["lse"],
                             window=case["window"])
        return s["out"], s["lse"]
    if op == "fork":
        ecmd.page_assign(s["pages"], s["lens"], s["refs"], s["parent"], s["add"], case["page"], s["pages_out"],
                         s["lens_out"], s["refs_out"], s["src"], s["dst"], s["stats"])
        ecmd.page_copy(s["pools"], s["src"], s["dst"])
        return s["pages_out"], s["lens_out"], s["refs_out"], s["src"], s["dst"], s["stats"], s["pools"]
    ecmd.page_compact(s["pages"], s["refs"], s["pages_out"], s["refs_out"], s["src"], s["dst"], s["stats"])
    ecmd.page_copy(s["pools"], s["src"], s["dst"])
    return s["pages_out"], s["refs_out"], s["src"], s["dst"], s["stats"], s["pools"]


def _rotate(x, pos, freq, layout, mscale=1.0, inverse=False):
    """x [..., heads, d] rotated by pos [...]; the angles in 64 bits, the products in 32, one rounding."""
    angle = pos.double()[..., None] * freq
    cos, sin = (angle.cos() * mscale).float()[..., None, :], (angle.sin() * mscale).float()[..., None, :]
    if inverse:
        sin = -sin
    r = 2 * freq.numel()
    y = x[..., :r].float()
    a, b = (y[..., :r // 2], y[..., r // 2:]) if layout == "half" else (y[..., 0::2], y[..., 1::2])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([u, v], -1) if layout == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([y.to(x.dtype), x[..., r:]], -1)


def _copy_pages(pools, src, dst):
    """Page dst[i] of every pool from its page src[i]; pairs of -1 repeat the first real one."""
    real = src >= 0
    first = real.int().argmax()
    a = torch.where(real, src, src[first]).clamp(min=0).long()
    b = torch.where(real, dst, dst[first]).clamp(min=0).long()
    for pool in pools:
        pool[b] = pool[a]


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "rope":
        return _rotate(s["x"], s["pos"], s["freq"], case["layout"], case["mscale"], case["inverse"])
    if op == "append":
        q = _rotate(s["q"], s["pos"], s["freq"], case["layout"])
        k = _rotate(s["k"], s["pos"], s["freq"], case["layout"])
        row, pos, page, pages = s["row"].long(), s["pos"].long(), case["page"], s["pages"]
        n = s["k_cache"].shape[0]
        ok = (row >= 0) & (row < pages.shape[0]) & (pos >= 0) & (pos < pages.shape[1] * page)
        row, pos = torch.where(ok, row, 0), torch.where(ok, pos, 0)
        at = pages[row, pos // page].long()
        ok &= (at >= 0) & (at < n)
        tok = torch.where(ok, torch.arange(len(ok), device=ok.device), ok.int().argmax())   # padding repeats a real token
        s["k_cache"][at[tok], pos[tok] % page] = k[tok]
        s["v_cache"][at[tok], pos[tok] % page] = s["v"][tok]
        return q, s["k_cache"], s["v_cache"]
    if op == "attention":
        q, pages, lens = s["q"].float(), s["pages"].long(), s["lens"].long()
        b, hq, d = q.shape
        n, page, hk, dv = s["v_cache"].shape
        ok = (pages >= 0) & (pages < n)
        at = pages.clamp(0, n - 1)
        pos = torch.arange(pages.shape[1] * page, device=q.device)
        mask = (pos < lens[:, None]) & ok.repeat_interleave(page, 1)
        if case["window"]:
            mask &= pos >= lens[:, None] - case["window"]
        k = s["k_cache"][at].flatten(1, 2).transpose(1, 2).float()               # [b, hk, positions, d]
        v = torch.where(mask[:, None, :, None], s["v_cache"][at].flatten(1, 2).transpose(1, 2).float(), 0.0)
        score = torch.matmul(q.view(b, hk, hq // hk, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
        score = torch.where(mask[:, None, None], score, -math.inf)
        top = score.amax(-1, keepdim=True)
        p = (score - torch.where(top == -math.inf, 0.0, top)).exp()
        total = p.sum(-1, keepdim=True)
        out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
        return out.view(b, hq, dv).to(s["q"].dtype), (top + total.log()).view(b, hq)
    pages, refs, n = s["pages"].long(), s["refs"].long(), case["n"]
    ids = torch.arange(n, device=pages.device)
    rows, p = pages.shape
    if op == "fork":
        page, parent = case["page"], s["parent"].long()
        old = s["lens"].long().clamp(0, p * page)
        me, col = torch.arange(rows, device=pages.device), torch.arange(p, device=pages.device)
        has = (parent >= 0) & (parent < rows)
        par = parent.clamp(0, rows - 1)
        length = torch.where(has, old[par], 0)
        new = (length + s["add"].clamp(min=0)).clamp(max=p * page)
        keep = torch.where(has & (par == me), (length + page - 1) // page, length // page)[:, None]
        total = ((new + page - 1) // page)[:, None]
        fresh = (col >= keep) & (col < total)
        rank = fresh.flatten().cumsum(0).view(rows, p) - 1
        free = refs == 0
        order = torch.argsort(free.logical_not(), stable=True)                    # free pages first, ascending
        have, want = free.sum(), fresh.sum()
        given = torch.where(rank < have, order[rank.clamp(0, n - 1)], -1)
        kept = torch.where(col < keep, pages[par], -1)
        out = torch.where(fresh, given, torch.where((kept >= 0) & (kept < n), kept, -1))
        delta = torch.zeros(n, dtype=torch.long, device=pages.device)
        was = (col < ((old + page - 1) // page)[:, None]) & (pages >= 0) & (pages < n)
        spare = torch.arange(rows * p, device=pages.device).view(rows, p) % n    # where nothing is counted, spread out
        delta.index_add_(0, torch.where(was, pages, spare).flatten(), -was.long().flatten())
        delta.index_add_(0, torch.where(out >= 0, out, spare).flatten(), (out >= 0).long().flatten())
        last = (length // page).clamp(max=p - 1)
        a, b = pages[par, last], out[me, last]
        copy = has & (par != me) & (length % page != 0) & (a >= 0) & (a < n) & (b >= 0)
        src, dst = torch.where(copy, a, -1).int(), torch.where(copy, b, -1).int()
        stats = torch.stack([want, torch.minimum(want, have)]).int()
        _copy_pages(s["pools"], src, dst)
        return out.int(), new.int(), (refs + delta).int(), src, dst, stats, s["pools"]
    live = refs > 0
    k = live.sum()
    high, low = live & (ids >= k), ~live & (ids < k)
    moves = high.sum()
    src = torch.argsort(high.logical_not(), stable=True)[:n // 2]
    dst = torch.argsort(low.logical_not(), stable=True)[:n // 2]
    to = torch.where(high, dst[(high.cumsum(0) - 1).clamp(min=0)], ids)
    comes = torch.where(low, src[(low.cumsum(0) - 1).clamp(min=0)], ids)
    at = pages.clamp(0, n - 1)
    out = torch.where((pages >= 0) & (pages < n) & live[at], to[at], -1).int()
    real = torch.arange(n // 2, device=pages.device) < moves
    src, dst = torch.where(real, src, -1).int(), torch.where(real, dst, -1).int()
    _copy_pages(s["pools"], src, dst)
    return (out, torch.where(ids < k, refs[comes], 0).int(), src, dst, torch.stack([k, moves]).int(), s["pools"])


# ---------------------------------------------------------------------------
# The definition in 64 bits.

def _turned(x, pos, freq, layout, mscale=1.0, inverse=False):
    """Pairs as complex numbers, multiplied by mscale * exp(+-i angle)."""
    angle = pos.double().unsqueeze(-1) * freq
    unit = torch.polar(torch.full_like(angle, mscale), -angle if inverse else angle).unsqueeze(-2)
    y, r = x.double().clone(), 2 * freq.numel()
    if layout == "half":
        z = torch.complex(y[..., :r // 2], y[..., r // 2:r]) * unit
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:r:2], y[..., 1:r:2]) * unit
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _turned(s["x"], s["pos"], s["freq"], case["layout"], case["mscale"], case["inverse"])
    if op == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        k = _turned(s["k"], s["pos"], s["freq"], case["layout"])
        real = s["row"] >= 0
        row, pos = s["row"][real].long(), s["pos"][real].long()
        flat = s["pages"][row, pos // case["page"]].long() * case["page"] + pos % case["page"]
        kc.flatten(0, 1)[flat], vc.flatten(0, 1)[flat] = k[real], s["v"][real].double()
        return _turned(s["q"], s["pos"], s["freq"], case["layout"]), kc, vc
    if op == "attention":
        b, hq, d = s["q"].shape
        group, w = hq // case["hk"], case["window"]
        out, lse = [], []
        for r, length in enumerate(_lens(case, b, case["top"])):
            q = s["q"][r].double().unflatten(0, (case["hk"], group))
            lo = max(0, length - w) if w else 0
            pos = torch.arange(lo, length, device="cuda")
            at = s["pages"][r, pos // case["page"]].long()
            k = s["k_cache"][at, pos % case["page"]].double().permute(1, 2, 0)
            v = s["v_cache"][at, pos % case["page"]].double().transpose(0, 1)
            score = torch.bmm(q, k.contiguous()) / math.sqrt(d)
            out.append(torch.bmm(score.softmax(-1), v.contiguous()).flatten(0, 1))
            lse.append(score.logsumexp(-1).flatten())
        return torch.stack(out), torch.stack(lse)
    pages, refs, n, page = s["pages"].tolist(), s["refs"].tolist(), case["n"], case["page"]
    src, dst = [], []
    if op == "fork":
        free = [i for i in range(n) if refs[i] == 0]
        table, lens, wanted, given = [], [], 0, 0
        old, parent, add = _fork_plan(case)
        left = list(refs)
        for r in range(len(old)):
            for j in range(-(-old[r] // page)):
                left[pages[r][j]] -= 1
        for r, par in enumerate(parent):
            length = old[par] if par >= 0 else 0
            new = min(length + add[r], case["p"] * page)
            held = pages[par][:-(-length // page) if par == r else length // page] if par >= 0 else []
            pair = (-1, -1)
            for j in range(len(held), -(-new // page)):
                wanted += 1
                got = free[given] if given < len(free) else -1
                given += got >= 0
                if j * page < length and got >= 0:
                    pair = (pages[par][j], got)
                held = held + [got]
            src.append(pair[0])
            dst.append(pair[1])
            lens.append(new)
            for i in held:
                if i >= 0:
                    left[i] += 1
            table.append(held + [-1] * (case["p"] - len(held)))
        answer = [table, lens, left, src, dst, [wanted, given]]
    else:
        live = [i for i in range(n) if refs[i] > 0]
        to = {i: i for i in live}
        src = [i for i in live if i >= len(live)]
        dst = [i for i in range(len(live)) if refs[i] <= 0]
        to.update(zip(src, dst))
        left = [0] * n
        for i in live:
            left[to[i]] = refs[i]
        table = [[to.get(i, -1) for i in row] for row in pages]
        stats, fill = [len(live), len(src)], [-1] * (n // 2 - len(src))
        answer = [table, left, src + fill, dst + fill, stats]
    pools = []
    for pool in s["pools"]:
        after = pool.clone()
        for a, b in zip(src, dst):
            if a >= 0:
                after[b] = pool[a]
        pools.append(after)
    return (*[torch.tensor(x, dtype=torch.int32) for x in answer], pools)
