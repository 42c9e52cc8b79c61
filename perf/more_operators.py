"""Cases of the further serving operators over a paged key-value cache: attention
for a tree of drafted tokens, the choice of its accepted path with the move of
their slots, attention over pages that a cheap score selects, and the eviction of
pages by accumulated attention weight.

``run`` computes one call in elementary torch operations (``own`` False) or
through the library (``own`` True) on what ``prepare`` made; ``exact`` is the
operators' definition in 64 bits, written apart from both.

The cache: k_cache [N, page, kv heads, d], v_cache [N, page, kv heads, dv];
position p of row r lies in slot p % page of cache page pages[r, p // page].  An
id outside 0 .. N - 1 is a hole: nothing is written there and its positions take
no part in attention.
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
        # One sequence, a handful of guesses: the smallest check of drafted tokens.
        dict(name="tree_token", op="tree", b=1, t=8, hq=32, hk=8, d=128, dv=128, page=16, top=777, window=0,
             dtype="f16"),
        # A serving batch, 64 drafted tokens a row, contexts from nothing to 8192.
        dict(name="tree_batch", op="tree", b=16, t=64, hq=32, hk=8, d=128, dv=128, page=16, top=8192, window=0,
             dtype="bf16"),
        # One key head a query head, odd sizes, and a window whose older pages have been given back.
        dict(name="tree_window", op="tree", b=5, t=23, hq=12, hk=12, d=80, dv=64, page=17, top=2047, window=1000,
             dtype="f32"),
        # What one sequence's check leaves: four guesses of five tokens, one layer.
        dict(name="accept_token", op="accept", rows=1, chains=4, length=5, layers=1, page=16, p=64, h=8, d=128,
             dtype="bf16"),
        # A server's: 128 rows, eight guesses of seven tokens each, the caches of eight layers.
        dict(name="accept_batch", op="accept", rows=128, chains=8, length=7, layers=8, page=16, p=96, h=8, d=128,
             dtype="bf16"),
        # A decode step of 64 sequences that reads 64 pages of each kv head in place of up to 512.
        dict(name="sparse_batch", op="sparse", b=64, hq=32, hk=8, d=128, dv=128, page=16, top=8192, take=64, holes=0.0,
             dtype="bf16"),
        # Two long documents, some of whose pages have been evicted; few pages of many.
        dict(name="sparse_long", op="sparse", b=2, hq=16, hk=2, d=128, dv=128, page=64, top=262143, take=96, holes=0.1,
             dtype="f16"),
        # The key bounds of 16 ragged prompts, after their append.
        dict(name="bounds_prompt", op="bounds", b=16, hk=4, d=96, page=32, top=4000, dtype="f16"),
        # The weight that a step's attention gave to every page, for a batch.
        dict(name="mass_batch", op="mass", b=64, hq=32, hk=8, d=128, page=16, top=8192, window=0, dtype="bf16"),
        # The same for a few rows in a window, binary32, odd sizes.
        dict(name="mass_window", op="mass", b=3, hq=12, hk=12, d=80, page=17, top=1500, window=1000, dtype="f32"),
        # Four sequences whose pages just passed their budgets.
        dict(name="evict_few", op="evict", rows=4, p=64, n=512, first=1, last=2, keep=0.8, share=0.0),
        # A server's tables brought back to their budgets.
        dict(name="evict_serve", op="evict", rows=256, p=1024, n=163840, first=1, last=4, keep=0.6, share=0.1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "accept", "sparse", "sparse", "bounds", "mass", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    hk = _log(rng, 1, 8)
    hq = hk * rng.choice([1, 2, 3, 4, 8, 16])
    d = rng.choice([64, 80, 96, 128, 128, 192, rng.randint(33, 200)])
    dv = rng.choice([d, d, 64, 128])
    page = rng.choice([1, 16, 16, 32, 64, rng.randint(2, 100)])
    wide = 2 if dtype == "f32" else 1
    if op == "tree":
        b, t, top = _log(rng, 1, 16), _log(rng, 1, 100), _log(rng, 1, 65536)
        while b * top * hk * (d + dv) * wide > 200000000 or b * top * hq * t * (d + dv) * wide * wide > 30000000000:
            b, top, t = max(1, b // 2), (top + 1) // 2, max(1, t - 1)
        return dict(op=op, b=b, t=t, hq=hq, hk=hk, d=d, dv=dv, page=page, top=top,
                    window=rng.choice([0, 0, rng.randint(1, top)]), dtype=dtype)
    if op == "accept":
        page = rng.choice([8, 16, 32, rng.randint(2, 50)])
        rows, chains, length = _log(rng, 1, 128), rng.randint(1, 8), _log(rng, 1, 16)
        layers, p = _log(rng, 1, 8), -(-rng.randint(200, 1500) // page)
        while rows * p * page * layers * hk * d > 400000000:
            rows, layers = (rows + 1) // 2, max(1, layers - 1)
        return dict(op=op, rows=rows, chains=chains, length=length, layers=layers, page=page, p=p, h=hk, d=d,
                    dtype=dtype)
    if op == "sparse":
        page = rng.choice([8, 16, 16, 32, 64])
        b, top = _log(rng, 1, 64), _log(rng, 200, 131072)
        while b * top * hk * (d + dv) * wide > 400000000:
            b, top = max(1, b // 2), (top + 1) // 2
        return dict(op=op, b=b, hq=hq, hk=hk, d=d, dv=dv, page=page, top=top,
                    take=_log(rng, 4, max(5, top // page)), holes=rng.choice([0.0, 0.0, 0.2]), dtype=dtype)
    if op == "bounds":
        page = rng.choice([8, 16, 32, 64, rng.randint(2, 100)])
        b, top = _log(rng, 1, 16), _log(rng, 1, 8192)
        while b * top * hk * d * wide > 200000000:
            b, top = max(1, b // 2), (top + 1) // 2
        return dict(op=op, b=b, hk=hk, d=d, page=page, top=top, dtype=dtype)
    if op == "mass":
        page = rng.choice([8, 16, 16, 32, 64, rng.randint(2, 100)])
        b, top = _log(rng, 1, 64), _log(rng, 1, 65536)
        while b * top * hk * d * wide > 200000000:
            b, top = max(1, b // 2), (top + 1) // 2
        return dict(op=op, b=b, hq=hq, hk=hk, d=d, page=page, top=top,
                    window=rng.choice([0, 0, rng.randint(1, top)]), dtype=dtype)
    rows, p = _log(rng, 1, 256), _log(rng, 8, 1024)
    return dict(op=op, rows=rows, p=p, n=rows * p + rng.randint(0, 4096), first=rng.randint(0, 2),
                last=rng.randint(0, 4), keep=rng.uniform(0.1, 1.0), share=rng.choice([0.0, 0.1, 0.3]))


# ---------------------------------------------------------------------------
# What a case's name alone decides: lengths, trees, budgets.

def _rng(case):
    return random.Random(" ".join("%s=%s" % kv for kv in sorted(case.items()) if kv[0] != "name"))


def _lens(case, b, top):
    """Lengths of b rows: the first the longest, one of four or more empty, the others spread."""
    rng = _rng(case)
    lens = [top] + [rng.randint(1, top) for _ in range(b - 1)]
    if b >= 4:
        lens[b // 2] = 0
    return lens


def _trees(case):
    """Every row's parents: deep trees of up to t tokens; rows with fewer end with padding (-2)."""
    rng = _rng(case)
    out = []
    for r in range(case["b"]):
        n = case["t"] if r == 0 else rng.randint((case["t"] + 1) // 2, case["t"])
        row = [-1] + [i - 1 if rng.random() < 0.5 else rng.randint(max(0, i - 8), i - 1) for i in range(1, n)]
        out.append(row + [-2] * (case["t"] - n))
    return out


def _guesses(case):
    """Of every row: its length, which guess turns out right and how far (a token more: the first)."""
    rng = _rng(case)
    room = case["p"] * case["page"] - 1 - case["chains"] * case["length"]
    return [(rng.randint(0, max(0, room)), rng.randrange(case["chains"]), rng.randint(0, case["length"]))
            for _ in range(case["rows"])]


def _held(case):
    """Columns in use and the budget of every row."""
    rng = _rng(case)
    used = [case["p"]] + [rng.randint(0, case["p"]) for _ in range(case["rows"] - 1)]
    return used, [max(1, round(x * rng.uniform(case["keep"], 1.1))) for x in used]


def work(case):
    op = case["op"]
    if op == "evict":
        used, _ = _held(case)
        entries = case["rows"] * case["p"]
        return dict(bytes=4 * sum(used) * 2 + 4 * entries + 8 * case["n"] + 12 * case["rows"], flops=sum(used))
    e = 4 if case["dtype"] == "f32" else 2
    if op == "accept":
        t = 1 + case["chains"] * case["length"]
        slot = case["h"] * case["d"] * e
        moved = sum(far for _, chain, far in _guesses(case) if chain)
        return dict(bytes=12 * case["rows"] * t + 16 * case["rows"] + 4 * case["rows"] * t
                    + 2 * case["layers"] * 2 * moved * slot, flops=0)
    lens = _lens(case, case["b"], case["top"])
    if op == "bounds":
        keys, pages = sum(lens), sum(-(-x // case["page"]) for x in lens)
        per = case["hk"] * case["d"]
        return dict(bytes=(keys + 2 * pages) * per * e + 4 * pages, flops=2 * keys * per)
    w = case.get("window", 0)
    if op == "tree":
        per, keys, pairs = case["d"] + case["dv"], 0, 0
        for x, parents in zip(lens, _trees(case)):
            n, depth = sum(p >= -1 for p in parents), []
            for p in parents[:n]:
                depth.append(depth[p] + 1 if p >= 0 else 0)
            keys += (min(x, w) if w else x) + n
            pairs += sum(min(x + y + 1, w) if w else x + y + 1 for y in depth)
        tokens = case["b"] * case["t"] * case["hq"]
        return dict(bytes=keys * case["hk"] * per * e + tokens * (per * e + 4), flops=2 * pairs * case["hq"] * per)
    if op == "mass":
        keys = sum(min(x, w) if w else x for x in lens)
        pages = sum(-(-x // case["page"]) for x in lens)
        return dict(bytes=keys * case["hk"] * case["d"] * e + case["b"] * case["hq"] * (case["d"] * e + 4) + 8 * pages,
                    flops=2 * keys * case["hq"] * case["d"])
    per, pages, keys = case["d"] + case["dv"], 0, 0
    for x in lens:
        used = -(-x // case["page"])
        pages += used
        keys += min(x, case["take"] * case["page"])
    return dict(bytes=pages * case["hk"] * 2 * case["d"] * e + keys * case["hk"] * per * e
                + case["b"] * case["hq"] * (per * e + 4),
                flops=(2 * pages * case["d"] * 2 + 2 * keys * per) * case["hq"])


# ---------------------------------------------------------------------------
# Inputs.

def _randn(g, *shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype) if np.prod(shape) < 1 << 22 \
        else torch.empty(shape, device="cuda", dtype=dtype).normal_(generator=g)


def _ints(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def _empty(*shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _tables(pick, page, lens, spare=2):
    """Pages of rows with these lengths, at random places of a cache a little larger: the table and n."""
    used = [-(-x // page) for x in lens]
    n, at = sum(used) + spare, 0
    ids, pages = pick.permutation(n), np.full((len(lens), max(used) + 1), -1)
    for r, u in enumerate(used):
        pages[r, :u] = ids[at:at + u]
        at += u
    return pages, n


def _queries(g, *shape, dtype):
    """Queries [..., hq, d] of different sharpness: near-uniform weights in some heads, a few keys' in others."""
    sharp = torch.linspace(0.5, 3.0, shape[-2], device="cuda")[:, None]
    return (_randn(g, *shape, dtype=torch.float32) * sharp).to(dtype)


def _garbage(caches, pages, lens, page):
    """A last page's unused slots hold whatever the memory held."""
    for r, x in enumerate(lens):
        if x % page and pages[r, x // page] >= 0:
            for c in caches:
                c[pages[r, x // page], x % page:] = math.nan


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    pick = np.random.RandomState(seed & 0x7FFFFFFF)
    op = case["op"]
    s = dict(case=case)
    if op == "evict":
        rows, p, n = case["rows"], case["p"], case["n"]
        used, budget = _held(case)
        pages, refs, at, ids = np.full((rows, p), -1), np.zeros(n, np.int64), 0, pick.permutation(n)
        for r in range(rows):
            pages[r, :used[r]] = ids[at:at + used[r]]
            at += used[r]
            common = int(min(used[r], used[r - 1]) * case["share"]) if r % 4 else 0
            pages[r, :common] = pages[r - 1, :common]          # a common prompt
            gone = pick.rand(used[r]) < 0.05                   # evicted before
            pages[r, :used[r]][gone] = -1
            np.add.at(refs, pages[r][pages[r] >= 0], 1)
        mass = torch.randn((rows, p), generator=g, device="cuda").mul_(2).exp_()
        mass[torch.rand((rows, p), generator=g, device="cuda") < 0.1] = 0.0      # never attended to
        page = 16
        lens = [max(0, u * page - pick.randint(0, page)) for u in used]
        s.update(pages=_ints(pages), lens=_ints(lens), refs=_ints(refs), mass=mass, budget=_ints(budget), page=page,
                 pages_out=_empty(rows, p), refs_out=_empty(n), count=_empty(rows))
        return s
    dt, page, d = DTYPES[case["dtype"]], case["page"], case["d"]
    if op == "accept":
        rows, p, h = case["rows"], case["p"], case["h"]
        chains, length = case["chains"], case["length"]
        t, n = 1 + chains * length, rows * p + 1
        pages = pick.permutation(n)[:rows * p].reshape(rows, p)
        parent = [-1] + [0 if i % length == 0 else i for i in range(chains * length)]
        tokens = pick.randint(0, 50000, size=(rows, t))
        follow = pick.randint(50000, 100000, size=(rows, t))           # no drafted token
        lens = []
        for r, (x, chain, far) in enumerate(_guesses(case)):
            lens.append(x)
            at = 0
            for i in range(far):
                follow[r, at] = tokens[r, 1 + chain * length + i]
                at = 1 + chain * length + i
        s.update(tokens=_ints(tokens), parent=_ints([parent] * rows), follow=_ints(follow), lens=_ints(lens),
                 pages=_ints(pages), path=_empty(rows, t), lens_out=_empty(rows), last=_empty(rows),
                 pools=[_randn(g, n, page, h, d, dtype=dt) for _ in range(2 * case["layers"])])
        return s
    b, hk = case["b"], case["hk"]
    lens = _lens(case, b, case["top"])
    if op == "tree":
        hq, dv, t, w = case["hq"], case["dv"], case["t"], case["window"]
        trees = _trees(case)
        full = [x + sum(q >= -1 for q in tree) for x, tree in zip(lens, trees)]
        pages, n = _tables(pick, page, full)
        for r in range(b):
            if w:                                      # pages wholly before the window have been given back
                pages[r, :max(0, lens[r] + 1 - w) // page] = -1
        k, v = _randn(g, n, page, hk, d, dtype=dt), _randn(g, n, page, hk, dv, dtype=dt)
        _garbage((k, v), pages, full, page)
        s.update(q=_queries(g, b, t, hq, d, dtype=dt), k_cache=k, v_cache=v, pages=_ints(pages), lens=_ints(lens),
                 parent=_ints(trees), out=_empty(b, t, hq, dv, dtype=dt), lse=_empty(b, t, hq, dtype=torch.float32))
        return s
    pages, n = _tables(pick, page, lens)
    if case.get("window"):
        for r in range(b):
            pages[r, :max(0, lens[r] - case["window"]) // page] = -1
    if case.get("holes"):
        for r in range(b):
            last = max(0, lens[r] - 1) // page
            pages[r, 1:last][pick.rand(max(0, last - 1)) < case["holes"]] = -1
    k = _randn(g, n, page, hk, d, dtype=dt)
    if op == "bounds":
        _garbage((k,), pages, lens, page)
        s.update(k_cache=k, pages=_ints(pages), lens=_ints(lens), since=_ints([0] * b),
                 bounds=torch.zeros(n, hk, 2, d, dtype=dt, device="cuda"))
        return s
    hq = case["hq"]
    q = _queries(g, b, hq, d, dtype=dt)
    if op == "mass":
        _garbage((k,), pages, lens, page)
        s.update(q=q, k_cache=k, pages=_ints(pages), lens=_ints(lens), out=_empty(*pages.shape, dtype=torch.float32),
                 mass=torch.rand(pages.shape, generator=g, device="cuda"))
        lse = torch.full((b, hq), -math.inf, device="cuda")
        for r, x in enumerate(lens):                   # the attention before left these
            lo = max(0, x - case["window"]) if case["window"] else 0
            if x > lo:
                pos = torch.arange(lo, x, device="cuda")
                keys = k[s["pages"][r, pos // page].long(), pos % page].float().permute(1, 2, 0).contiguous()
                score = torch.bmm(q[r].float().view(hk, hq // hk, d), keys) / math.sqrt(d)
                lse[r] = score.logsumexp(-1).flatten()
        s.update(lse=lse)
        return s
    # sparse: the keys of a page lie around a centre of its own; the newest position's are not in the bounds yet
    k += _randn(g, n, 1, hk, d, dtype=dt)
    v = _randn(g, n, page, hk, case["dv"], dtype=dt)
    bounds = torch.stack([k.amin(1), k.amax(1)], 2)
    for r, x in enumerate(lens):
        held = (x - 1) % page
        if x and held:
            part = k[pages[r, (x - 1) // page], :held]
            bounds[pages[r, (x - 1) // page]] = torch.stack([part.amin(0), part.amax(0)], 1)
    _garbage((k, v), pages, lens, page)
    take = case["take"]
    s.update(q=q, k_cache=k, v_cache=v, pages=_ints(pages), lens=_ints(lens),
             since=_ints([max(0, x - 1) for x in lens]), bounds=bounds, picked=_empty(b, hk, take),
             picked_lens=_empty(b, hk), out=_empty(b, hq, case["dv"], dtype=dt),
             lse=_empty(b, hq, dtype=torch.float32))
    return s


# ---------------------------------------------------------------------------
# One pass.

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import elementwise_tensor_commands_amd as ecmd
    case = s["case"]
    op = case["op"]
    if op == "tree":
        ecmd.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["lens"], s["parent"], s["out"],
                            lse=s["lse"], window=case["window"])
        return s["out"], s["lse"]
    if op == "accept":
        ecmd.tree_accept(s["tokens"], s["parent"], s["follow"], s["lens"], s["path"], s["lens_out"], s["last"])
        ecmd.slot_move(s["pools"], s["pages"], s["lens"], s["path"])
        return s["path"], s["lens_out"], s["last"], s["pools"]
    if op == "bounds":
        ecmd.page_bounds(s["k_cache"], s["pages"], s["lens"], s["since"], s["bounds"])
        return s["bounds"]
    if op == "sparse":
        ecmd.page_bounds(s["k_cache"], s["pages"], s["lens"], s["since"], s["bounds"])
        ecmd.page_select(s["q"], s["bounds"], s["pages"], s["lens"], case["page"], s["picked"], s["picked_lens"],
                         first=1, last=2)
        ecmd.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["picked"], s["picked_lens"], s["out"],
                             lse=s["lse"])
        return s["bounds"], s["picked"], s["picked_lens"], s["out"], s["lse"]
    if op == "mass":
        ecmd.page_mass(s["q"], s["k_cache"], s["pages"], s["lens"], s["lse"], s["mass"], s["out"], decay=0.95,
                       window=case["window"])
        return s["out"]
    ecmd.page_evict(s["pages"], s["lens"], s["refs"], s["mass"], s["budget"], s["page"], s["pages_out"],
                    s["refs_out"], s["count"], first=case["first"], last=case["last"])
    return s["pages_out"], s["refs_out"], s["count"]


def _attend(q, k, v, mask):
    """q [b, hk, m, d] over k [b, hk, x, d] and v under mask [b, 1 or hk, m, x], in 32 bits: out and lse."""
    score = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(q.shape[-1]))
    score = torch.where(mask, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top == -math.inf, 0.0, top)).exp()
    total = p.sum(-1, keepdim=True)
    v = torch.where(mask.any(2)[..., None], v, 0.0)
    return torch.matmul(p, v) / torch.where(total == 0, 1.0, total), (top + total.log()).squeeze(-1)


def _reach(parent):
    """[b, i, j]: j is i or above it; and which tokens are none (padding, or below it)."""
    b, t = parent.shape
    at = torch.arange(t, device=parent.device)
    fine = (parent >= 0) & (parent < at)
    up = ((parent[:, :, None] == at) & fine[:, :, None]).float() + torch.eye(t, device=parent.device)
    steps = 1
    while steps < t:
        up = (torch.matmul(up, up) > 0).float()
        steps *= 2
    up = up > 0
    return up, ~(up & ~(fine | (parent == -1))[:, None]).any(-1)


def _widen(s):
    """Bounds of the pages with positions since .. lens - 1: from their first slot, or with what was known."""
    k, pages, lens, since, bounds = s["k_cache"], s["pages"].long(), s["lens"].long(), s["since"].long(), s["bounds"]
    n, page = k.shape[:2]
    cols = 1 if s["case"]["op"] == "sparse" else pages.shape[1]
    col = since[:, None] // page + torch.arange(cols, device=k.device)
    at = pages.gather(1, col.clamp(max=pages.shape[1] - 1))
    start = torch.maximum(col * page, since[:, None])
    real = (start < lens[:, None]) & (col < pages.shape[1]) & (at >= 0) & (at < n)
    pos = col[..., None] * page + torch.arange(page, device=k.device)
    new = (pos >= start[..., None]) & (pos < lens[:, None, None])
    x = k[at.clamp(0, n - 1)]                                                     # [b, cols, page, hk, d]
    lo = torch.where(new[..., None, None], x, math.inf).amin(2)
    hi = torch.where(new[..., None, None], x, -math.inf).amax(2)
    old, add = bounds[at.clamp(0, n - 1)], (start > col * page)[..., None, None]
    lo = torch.where(add, torch.minimum(lo, old[..., 0, :]), lo)
    hi = torch.where(add, torch.maximum(hi, old[..., 1, :]), hi)
    one = real.flatten().int().argmax()                   # where nothing is to do, a real page's again
    to = torch.where(real.flatten(), at.flatten(), at.flatten()[one])
    value = torch.stack([lo, hi], 3).flatten(0, 1)
    value = torch.where(real.flatten()[:, None, None, None], value, value[one])
    bounds[to] = value.to(bounds.dtype)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "accept":
        tokens, parent, follow = s["tokens"], s["parent"].long(), s["follow"]
        rows, t = tokens.shape
        at, me = torch.arange(t, device=tokens.device), torch.arange(rows, device=tokens.device)
        cur = torch.where(parent[:, 0] == -1, 0, -1)
        path, last = [], torch.full((rows,), -1, dtype=torch.int32, device=tokens.device)
        for _ in range(case["length"] + 1):               # no path is longer
            path.append(cur)
            here = cur >= 0
            want = follow[me, cur.clamp(min=0)]
            last = torch.where(here, want, last)
            fits = here[:, None] & (parent == cur[:, None]) & (tokens == want[:, None]) & (at > cur[:, None])
            cur = torch.where(fits.any(1), fits.int().argmax(1), -1)
        path = torch.stack(path + [torch.full_like(cur, -1)] * (t - len(path)), 1)
        lens, page = s["lens"].long(), s["pools"][0].shape[1]
        n, limit = s["pools"][0].shape[0], s["pages"].shape[1] * page
        a, b = lens[:, None] + path, lens[:, None] + at
        move = (path > at) & (a < limit)
        pa = s["pages"].long().gather(1, a.clamp(0, limit - 1) // page)
        pb = s["pages"].long().gather(1, b.clamp(0, limit - 1) // page)
        move &= (pa >= 0) & (pa < n) & (pb >= 0) & (pb < n)
        sa, sb = (pa * page + a % page)[:, 1:].flatten(), (pb * page + b % page)[:, 1:].flatten()
        move = move[:, 1:].flatten()
        for pool in s["pools"]:
            flat = pool.view(n * page, *pool.shape[2:])
            x = torch.where(move[:, None, None], flat[sa], flat[sb])
            flat[sb] = x
        return path.int(), (lens + (path >= 0).sum(1)).int(), last, s["pools"]
    if op == "evict":
        pages, lens, refs, page = s["pages"].long(), s["lens"].long(), s["refs"].long(), s["page"]
        rows, p = pages.shape
        n = refs.numel()
        col = torch.arange(p, device=pages.device)
        used = ((lens.clamp(0, p * page) + page - 1) // page)[:, None]
        held = (col < used) & (pages >= 0) & (pages < n)
        loose = held & (col >= case["first"]) & (col < used - case["last"])
        over = held.sum(1) - s["budget"].clamp(min=0)
        key = torch.where(loose, s["mass"], math.inf)
        order = torch.sort(key, dim=1, stable=True).indices
        rank = torch.empty_like(order).scatter_(1, order, col.expand(rows, p))
        gone = loose & (rank < over[:, None])
        out = torch.where(gone | ~((pages >= 0) & (pages < n)), -1, pages)
        drop = torch.zeros(n, dtype=torch.long, device=pages.device)
        spare = torch.arange(rows * p, device=pages.device).view(rows, p) % n    # where nothing is counted, spread out
        drop.index_add_(0, torch.where(gone, pages, spare).flatten(), gone.long().flatten())
        return out.int(), (refs - drop).int(), gone.sum(1).int()
    if op == "bounds":
        _widen(s)
        return s["bounds"]
    q, pages, lens = s["q"], s["pages"].long(), s["lens"].long()
    n, page, hk, d = s["k_cache"].shape
    b, hq = q.shape[0], q.shape[-2]
    group = hq // hk
    if op == "tree":
        t, w = q.shape[1], case["window"]
        ok = (pages >= 0) & (pages < n)
        at = pages.clamp(0, n - 1)
        pos = torch.arange(pages.shape[1] * page, device=q.device)
        up, valid = _reach(s["parent"].long())
        depth = up.sum(-1) - 1
        mask = (pos < lens[:, None])[:, None].expand(b, t, len(pos))
        slot = pos - lens[:, None]                                              # of the tree, where 0 .. t - 1
        inside = (slot >= 0) & (slot < t)
        above = up.gather(2, slot.clamp(0, t - 1)[:, None].expand(b, t, len(pos)))
        if w:
            mask = mask & (pos >= (lens[:, None] + depth + 1 - w)[..., None])
            other = depth.gather(1, slot.clamp(0, t - 1))
            above = above & (depth[..., None] - other[:, None] < w)
        mask = (mask | (above & inside[:, None])) & ok.repeat_interleave(page, 1)[:, None] & valid[..., None]
        k = s["k_cache"][at].flatten(1, 2).transpose(1, 2).float()              # [b, hk, positions, d]
        v = s["v_cache"][at].flatten(1, 2).transpose(1, 2).float()
        qs = q.float().view(b, t, hk, group, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
        out, lse = _attend(qs, k, v, mask.repeat_interleave(group, 1)[:, None])
        out = out.view(b, hk, t, group, -1).permute(0, 2, 1, 3, 4).reshape(b, t, hq, -1)
        return out.to(q.dtype), lse.view(b, hk, t, group).permute(0, 2, 1, 3).reshape(b, t, hq)
    ok = (pages >= 0) & (pages < n)
    at = pages.clamp(0, n - 1)
    if op == "mass":
        pos = torch.arange(pages.shape[1] * page, device=q.device)
        mask = (pos < lens[:, None]) & ok.repeat_interleave(page, 1)
        if case["window"]:
            mask &= pos >= lens[:, None] - case["window"]
        k = s["k_cache"][at].flatten(1, 2).transpose(1, 2).float()
        score = torch.matmul(q.float().view(b, hk, group, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
        lse = s["lse"].view(b, hk, group, 1)
        weight = torch.where(mask[:, None, None], (score - lse).exp(), 0.0)
        return s["mass"] * 0.95 + weight.sum((1, 2)).view(b, -1, page).sum(-1)
    _widen(s)
    take = case["take"]
    used = (lens + page - 1) // page
    col = torch.arange(pages.shape[1], device=q.device)
    held = ok & (col < used[:, None])
    lo, hi = s["bounds"][at].double().permute(3, 0, 2, 1, 4)                    # [b, hk, cols, d]
    qs = q.double().view(b, hk, group, d)
    score = (torch.matmul(qs.clamp(min=0), hi.transpose(2, 3).contiguous())
             + torch.matmul(qs.clamp(max=0), lo.transpose(2, 3).contiguous())).amax(2)
    always = (col < 1) | (col >= used[:, None] - 2)
    score = torch.where(always[:, None], math.inf, score)
    score = torch.where(held[:, None], score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, col.expand(order.shape).contiguous())
    chosen = held[:, None] & (rank < take)
    front = torch.argsort(chosen.logical_not().int(), dim=-1, stable=True)[..., :take]      # ascending columns
    if front.shape[-1] < take:
        front = torch.nn.functional.pad(front, (0, take - front.shape[-1]))
    count = chosen.sum(-1)
    there = torch.arange(take, device=q.device) < count[..., None]
    picked = torch.where(there, pages[:, None].expand(order.shape).gather(2, front), -1)
    final = front.gather(2, (count - 1).clamp(min=0)[..., None]).squeeze(-1)
    full = torch.where(final == (used - 1)[:, None], (lens - (used - 1) * page)[:, None], page)
    picked_lens = torch.where(count > 0, (count - 1) * page + full, 0)
    head = torch.arange(hk, device=q.device)[None, :, None]
    k = s["k_cache"][picked.clamp(min=0), :, head].flatten(2, 3).float()        # [b, hk, take * page, d]
    v = s["v_cache"][picked.clamp(min=0), :, head].flatten(2, 3).float()
    mask = torch.arange(take * page, device=q.device) < picked_lens[..., None]
    out, lse = _attend(q.float().view(b, hk, group, d), k, v, mask[:, :, None].expand(b, hk, group, take * page))
    return (s["bounds"], picked.int(), picked_lens.int(), out.flatten(1, 2).to(q.dtype), lse.flatten(1, 2))


# ---------------------------------------------------------------------------
# The definition in 64 bits.

def _softmax_over(q, k, v):
    """q [hk, m, d], k [x, hk, d], v [x, hk, dv], every pair counting: out [hk, m, dv] and lse [hk, m]."""
    score = torch.bmm(q, k.permute(1, 2, 0).contiguous()) / math.sqrt(q.shape[-1])
    return torch.bmm(score.softmax(-1), v.transpose(0, 1).contiguous()), score.logsumexp(-1)


def _exact_tree(case, s):
    b, t, hq, d = s["q"].shape
    hk, page, w = case["hk"], case["page"], case["window"]
    out = torch.zeros(b, t, hq, case["dv"], dtype=torch.float64, device="cuda")
    lse = torch.full((b, t, hq), -math.inf, dtype=torch.float64, device="cuda")
    for r, (x, parents) in enumerate(zip(_lens(case, b, case["top"]), _trees(case))):
        n = sum(p >= -1 for p in parents)
        lo = max(0, x + 1 - w) if w else 0
        lo -= lo % page                                   # from the first page that is there
        lo = max(lo, 0)
        pos = torch.arange(lo, x + n, device="cuda")
        at = s["pages"][r, pos // page].long()
        k, v = s["k_cache"][at, pos % page].double(), s["v_cache"][at, pos % page].double()
        chains = []
        for i in range(n):
            chain, j = [], i
            while j >= 0:
                chain.append(j)
                j = parents[j]
            chains.append(chain)
        see = torch.zeros(n, x + n - lo, dtype=torch.bool)
        for i, chain in enumerate(chains):
            first = x + len(chain) - w if w else 0        # the oldest position that the window holds
            see[i, max(0, first - lo):x - lo] = True
            for j in chain[:w] if w else chain:
                see[i, x - lo + j] = True
        see = see.cuda()
        q = s["q"][r, :n].double().view(n, hk, hq // hk, d).transpose(0, 1).flatten(1, 2)
        score = torch.bmm(q, k.permute(1, 2, 0).contiguous()) / math.sqrt(d)
        score = score.masked_fill(~see.repeat_interleave(hq // hk, 0), -math.inf)
        o = torch.bmm(score.softmax(-1), v.transpose(0, 1).contiguous())
        out[r, :n] = o.view(hk, n, hq // hk, -1).transpose(0, 1).flatten(1, 2)
        lse[r, :n] = score.logsumexp(-1).view(hk, n, hq // hk).transpose(0, 1).flatten(1, 2)
    return out, lse


def _exact_accept(case, s):
    rows, t = s["tokens"].shape
    page, length = case["page"], case["length"]
    path, lens_out, last, moves = [], [], [], []
    follow, table = s["follow"].tolist(), s["pages"].tolist()
    for r, (x, chain, far) in enumerate(_guesses(case)):
        row = [0] + [1 + chain * length + i for i in range(far)]
        moves += [(table[r][(x + j) // page], (x + j) % page, table[r][(x + i) // page], (x + i) % page)
                  for i, j in enumerate(row) if i != j]
        path.append(row + [-1] * (t - len(row)))
        lens_out.append(x + len(row))
        last.append(follow[r][row[-1]])
    pools = []
    m = torch.tensor(moves, dtype=torch.long, device="cuda").view(-1, 4)
    for pool in s["pools"]:
        after = pool.clone()
        after[m[:, 2], m[:, 3]] = pool[m[:, 0], m[:, 1]]
        pools.append(after)
    return (*[torch.tensor(x, dtype=torch.int32) for x in (path, lens_out, last)], pools)


def _exact_evict(case, s):
    pages, refs, mass = s["pages"].tolist(), s["refs"].tolist(), s["mass"].tolist()
    lens, budget, count, n = s["lens"].tolist(), s["budget"].tolist(), [], case["n"]
    for r, row in enumerate(pages):
        used = -(-lens[r] // s["page"])
        held = [j for j in range(used) if 0 <= row[j] < n]
        loose = sorted((j for j in held if case["first"] <= j < used - case["last"]), key=lambda j: (mass[r][j], j))
        gone = loose[:max(0, len(held) - budget[r])]
        for j in gone:
            refs[row[j]] -= 1
            row[j] = -1
        count.append(len(gone))
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (pages, refs, count))


def _exact_bounds(case, s, since):
    """Of the pages with positions since .. : least and largest of all the keys that they hold, others as they are."""
    bounds, page = s["bounds"].double(), case["page"]
    for r, x in enumerate(_lens(case, case["b"], case["top"])):
        for j in range(since(x) // page, -(-x // page)):
            i = int(s["pages"][r, j])
            if i >= 0:
                keys = s["k_cache"][i, :min(page, x - j * page)].double()
                bounds[i] = torch.stack([keys.amin(0), keys.amax(0)], 1)
    return bounds


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tree":
        return _exact_tree(case, s)
    if op == "accept":
        return _exact_accept(case, s)
    if op == "evict":
        return _exact_evict(case, s)
    if op == "bounds":
        return _exact_bounds(case, s, lambda x: 0)
    b, hq, d = s["q"].shape
    hk, page = case["hk"], case["page"]
    lens = _lens(case, b, case["top"])
    if op == "mass":
        out = s["mass"].double() * 0.95
        for r, x in enumerate(lens):
            lo = max(0, x - case["window"]) if case["window"] else 0
            pos = torch.arange(lo, x, device="cuda")
            if not len(pos):
                continue
            k = s["k_cache"][s["pages"][r, pos // page].long(), pos % page].double()
            q = s["q"][r].double().unflatten(0, (hk, hq // hk))
            score = torch.bmm(q, k.permute(1, 2, 0).contiguous()) / math.sqrt(d)
            weight = torch.exp(score - s["lse"][r].double().view(hk, hq // hk, 1)).sum((0, 1))
            out[r].index_add_(0, pos // page, weight)
        return out
    bounds = _exact_bounds(case, s, lambda x: max(0, x - 1))
    take, group = case["take"], hq // hk
    picked = torch.full((b, hk, take), -1, dtype=torch.int32)
    picked_lens = torch.zeros(b, hk, dtype=torch.int32)
    out = torch.zeros(b, hq, case["dv"], dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    for r, x in enumerate(lens):
        used = -(-x // page)
        row = s["pages"][r, :used].long()
        cols = (row >= 0).nonzero().flatten()
        if not len(cols):
            continue
        q = s["q"][r].double().view(hk, group, 1, d)
        lo, hi = (bounds[row[cols], :, i].transpose(0, 1)[:, None] for i in (0, 1))
        score = torch.where(q >= 0, q * hi, q * lo).sum(-1).amax(1).cpu()           # [hk, columns]
        columns = cols.tolist()
        for h in range(hk):
            ranked = sorted(range(len(columns)),
                            key=lambda i: (not (columns[i] < 1 or columns[i] >= used - 2), -score[h, i].item()))
            mine = sorted(columns[i] for i in ranked[:take])
            picked[r, h, :len(mine)] = torch.tensor([int(row[j]) for j in mine], dtype=torch.int32)
            held = [min(page, x - j * page) for j in mine]
            picked_lens[r, h] = sum(held)
            at = torch.cat([torch.arange(j * page, j * page + c) for j, c in zip(mine, held)]).cuda()
            k = s["k_cache"][row[at // page], at % page, h].double()[:, None]
            v = s["v_cache"][row[at // page], at % page, h].double()[:, None]
            o, l = _softmax_over(q[h].view(1, group, d), k, v)
            out[r, h * group:(h + 1) * group], lse[r, h * group:(h + 1) * group] = o[0], l[0]
    return bounds, picked, picked_lens, out, lse
