"""Definitions, as plain loops in 64 bits on the CPU, of the operators on trees of
drafted tokens and on pages worth reading or keeping, with bounds on how far a
kernel that rounds as include/ecmd_serving.h says may be from them.  Shares no
code with the library."""
import math

import torch

from serving_oracle import half_step, tiny

U = 2.0 ** -24


def attend(q, k, v, scale, split, least):
    """Of query vectors q [m, d] over keys k [x, d] and values v [x, dv], x >= 1: out, lse and
    their bounds (float64).  split: how far a weight's parts may be from it, relative; least:
    relative to the largest weight."""
    s, size = q @ k.t() * scale, q.abs() @ k.abs().t() * abs(scale)
    w = torch.softmax(s, -1)
    out, lse = w @ v, torch.logsumexp(s, -1)
    top = s.amax(-1)
    # a score: d products and sums, three multiplications, the distance to the maximum; then
    # exp2, within 2^-22, and the weight's parts
    ds = size.amax(-1) * (q.shape[1] + 2) * 2 * U + (s.abs().amax(-1) + (top - s.amin(-1))) * 4 * U
    dw = 2 * ds + 2 * 2.0 ** -22 + split
    sums = k.shape[0] * 2 * U + 64 * U          # each side's sum, in any order, and the joins
    eo = (w @ v.abs()) * (dw + 2 * sums)[:, None] + w.amax(-1, keepdim=True) * v.abs().sum(0) * least
    el = ds + 2.0 ** -21 + sums + lse.abs() * 4 * U
    return out, lse, eo, el


SPLIT = {torch.bfloat16: 2.0 ** -14, torch.float16: 2.0 ** -20, torch.float32: 0.0}
LEAST = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -34, torch.float32: 0.0}


def above(parents):
    """For each token the tokens it attends to, itself first, then up; None: padding."""
    chains = []
    for i, p in enumerate(parents):
        if p == -1:
            chains.append([i])
        elif 0 <= p < i and chains[p] is not None:
            chains.append([i] + chains[p])
        else:
            chains.append(None)
    return chains


def tree(q, k_cache, v_cache, pages, lens, parent, scale, window=0):
    """out, lse and their bounds (float64)."""
    b, t, hq, d = q.shape
    n, page, hk, dv = v_cache.shape
    held, group = pages.shape[1] * page, hq // hk
    out, eo = torch.zeros(b, t, hq, dv, dtype=torch.float64), torch.zeros(b, t, hq, dv, dtype=torch.float64)
    lse, el = torch.full((b, t, hq), -math.inf, dtype=torch.float64), torch.zeros(b, t, hq, dtype=torch.float64)
    for r in range(b):
        length = int(lens[r])
        if length < 0:
            continue
        for i, chain in enumerate(above([int(x) for x in parent[r]])):
            if chain is None:
                continue
            first = max(0, length + len(chain) - window) if window else 0
            at = list(range(first, min(length, held))) + [length + x for x in (chain[:window] if window else chain)]
            at = [(int(pages[r, x // page]), x % page) for x in at if x < held]
            at = [x for x in at if 0 <= x[0] < n]
            if not at:
                continue
            at = torch.tensor(at)
            for g in range(hk):
                kk, vv = k_cache[at[:, 0], at[:, 1], g].double(), v_cache[at[:, 0], at[:, 1], g].double()
                heads = slice(g * group, (g + 1) * group)
                o, l, e, f = attend(q[r, i, heads].double(), kk, vv, scale, SPLIT[q.dtype], LEAST[q.dtype])
                out[r, i, heads], lse[r, i, heads], el[r, i, heads] = o, l, f
                eo[r, i, heads] = e + o.abs() * half_step(q.dtype) + tiny(q.dtype)
    return out, lse, eo, el


def accept(tokens, parent, follow, lens):
    rows, t = tokens.shape
    path, lens_out, last = [], [], []
    for r in range(rows):
        p, row, after = [int(x) for x in parent[r]], [], -1
        cur = 0 if t and p[0] == -1 and lens[r] >= 0 else None
        while cur is not None:
            row.append(cur)
            after = int(follow[r, cur])
            cur = next((c for c in range(cur + 1, t) if p[c] == cur and int(tokens[r, c]) == after), None)
        path.append(row + [-1] * (t - len(row)))
        lens_out.append(min(int(lens[r]) + len(row), 2 ** 31 - 1))
        last.append(after)
    return path, lens_out, last


def move(pools, pages, lens, path):
    """The pools after it (copies)."""
    pools = [p.clone() for p in pools]
    cols, page = pages.shape[1], pools[0].shape[1]
    for r in range(pages.shape[0]):
        length = int(lens[r])
        if length < 0:
            continue
        for i, x in enumerate(int(x) for x in path[r]):
            if x < 0:
                break
            a, b = length + x, length + i
            if x <= i or a >= cols * page:
                continue
            ia, ib = int(pages[r, a // page]), int(pages[r, b // page])
            for p in pools:
                if 0 <= ia < len(p) and 0 <= ib < len(p):
                    p[ib, b % page] = p[ia, a % page]
    return pools


def bounds(k_cache, pages, lens, since, old):
    """Bounds after it (a copy); NaN counts as nothing."""
    new = old.clone()
    n, page = k_cache.shape[:2]
    for r in range(pages.shape[0]):
        lo, hi = max(int(since[r]), 0), min(int(lens[r]), pages.shape[1] * page)
        for c in range(lo // page, -(-hi // page) if hi > lo else 0):
            i = int(pages[r, c])
            if not 0 <= i < n:
                continue
            a, b = max(lo, c * page), min(hi, (c + 1) * page)
            x = k_cache[i, a - c * page:b - c * page].double()
            least = torch.where(x.isnan(), math.inf, x).amin(0)
            most = torch.where(x.isnan(), -math.inf, x).amax(0)
            if a > c * page:
                was = old[i].double()
                least = torch.minimum(least, torch.where(was[:, 0].isnan(), math.inf, was[:, 0]))
                most = torch.maximum(most, torch.where(was[:, 1].isnan(), -math.inf, was[:, 1]))
            new[i] = torch.stack([least, most], 1).to(new.dtype)
    return new


def select(q, bounds, pages, lens, page, take, first, last):
    b, hq, d = q.shape
    n, hk = bounds.shape[:2]
    cols, group = pages.shape[1], hq // hk
    out, out_lens = torch.full((b, hk, take), -1, dtype=torch.int32), torch.zeros(b, hk, dtype=torch.int32)
    for r in range(b):
        hi = min(max(int(lens[r]), 0), cols * page)
        used = -(-hi // page)
        held = [c for c in range(used) if 0 <= int(pages[r, c]) < n]
        for h in range(hk):
            key = {}
            for c in held:
                x = bounds[int(pages[r, c]), h].double()
                if c < first or c >= used - last:
                    key[c] = (1, 0.0)
                    continue
                qs = q[r, h * group:(h + 1) * group].double()
                score = torch.where(qs < 0, qs * x[0], qs * x[1]).sum(-1)
                score = float(torch.where(score.isnan(), -math.inf, score).max())
                worst = bool(torch.where(qs < 0, qs * x[0], qs * x[1]).sum(-1).isnan().all())
                key[c] = (-1 if worst else 0, score)
            best = sorted(sorted(held, key=lambda c: (-key[c][0], -key[c][1], c))[:take])
            out[r, h, :len(best)] = torch.tensor([int(pages[r, c]) for c in best], dtype=torch.int32)
            out_lens[r, h] = sum(min(page, hi - c * page) for c in best)
    return out, out_lens


def mass(q, k_cache, pages, lens, lse, was, scale, decay, window=0):
    """mass_out and its bound (float64)."""
    b, hq, d = q.shape
    n, page, hk, _ = k_cache.shape
    cols, group = pages.shape[1], hq // hk
    out = was.double() * decay
    err = out.abs() * 2 * U
    for r in range(b):
        length = int(lens[r])
        for c in range(cols):
            a, z = c * page, min((c + 1) * page, length)
            if window:
                a = max(a, length - window)
            i = int(pages[r, c])
            if a >= z or not 0 <= i < n:
                continue
            total, bound = 0.0, 0.0
            for g in range(hk):
                k = k_cache[i, a - c * page:z - c * page, g].double()
                heads = slice(g * group, (g + 1) * group)
                on = ~torch.isneginf(lse[r, heads])
                qs, ls = q[r, heads].double()[on], lse[r, heads].double()[on, None]
                s, size = qs @ k.t() * scale, qs.abs() @ k.abs().t() * abs(scale)
                w = torch.exp(s - ls)
                total += float(w.sum())
                # a score: d products and sums, two multiplications; lse in base 2; their difference; exp2
                off = size * (d + 2) * 2 * U + (s.abs() + ls.abs()) * 4 * U + (s - ls).abs() * 2 * U + 2.0 ** -21
                bound += float((w * off * 1.01).sum())
            out[r, c] += total
            err[r, c] += bound + (total + abs(float(out[r, c]))) * ((z - a) * hq + 64) * 2 * U
    return out, err


def evict(pages, lens, refs, mass, budget, page, first, last):
    rows, cols = pages.shape
    n = len(refs)
    out, refs, count = [[int(x) if 0 <= int(x) < n else -1 for x in row] for row in pages], [int(x) for x in refs], []
    for r in range(rows):
        used = -(-min(max(int(lens[r]), 0), cols * page) // page)
        held = [c for c in range(used) if out[r][c] >= 0]
        key = lambda c: (math.isnan(float(mass[r, c])), 0.0 if math.isnan(float(mass[r, c])) else float(mass[r, c]), c)
        loose = sorted((c for c in held if first <= c < used - last), key=key)
        gone = loose[:max(0, len(held) - max(int(budget[r]), 0))]
        for c in gone:
            refs[out[r][c]] -= 1
            out[r][c] = -1
        count.append(len(gone))
    return out, refs, count
