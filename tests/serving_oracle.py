"""The serving operators' definitions as plain loops in 64 bits on the CPU, and
bounds on how far a kernel that rounds as include/ecmd_serving.h says may be
from them.  Shares no code with the library."""
import math

import torch


def half_step(t):
    """Half the spacing of the dtype's numbers, relative to the value."""
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the dtype's smallest subnormal."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def pairs(x, m, layout):
    return (x[..., :m], x[..., m:2 * m]) if layout == "half" else (x[..., 0:2 * m:2], x[..., 1:2 * m:2])


def rope(x, pos, freq, layout, mscale=1.0, inverse=False):
    """x [..., heads, d], pos [...] -> the turned heads, and the bound on the error."""
    y, m = x.double().clone(), freq.numel()
    w = pos.double()[..., None, None] * freq
    c, s = w.cos() * mscale, w.sin() * mscale * (-1 if inverse else 1)
    u, v = pairs(x.double(), m, layout)
    yu, yv = pairs(y, m, layout)
    a, b = u * c - v * s, v * c + u * s
    yu.copy_(a)
    yv.copy_(b)
    # cosine and sine round (half a step of binary32), so do the two products and
    # their sum; then the result rounds to the dtype
    err = torch.zeros_like(y)
    bound = (u.abs() + v.abs()) * abs(mscale) * 3.01 * 2.0 ** -24
    eu, ev = pairs(err, m, layout)
    eu.copy_(bound)
    ev.copy_(bound)
    if x.dtype != torch.float32:
        turned = (y.abs() + err) * half_step(x.dtype) + tiny(x.dtype)
        eu.add_(pairs(turned, m, layout)[0])
        ev.add_(pairs(turned, m, layout)[1])
    return y, err


def attention(q, k_cache, v_cache, pages, lens, scale, window=0):
    """out, lse and their bounds (all float64)."""
    b, hq, d = q.shape
    n, page, hk, dv = v_cache.shape
    cols = pages.shape[1]
    out, lse = torch.zeros(b, hq, dv, dtype=torch.float64), torch.full((b, hq), -math.inf, dtype=torch.float64)
    eo, el = torch.zeros_like(out), torch.zeros_like(lse)
    exact_split = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -20, torch.float32: 0.0}[q.dtype]
    u = 2.0 ** -24
    for r in range(b):
        length = int(lens[r])
        keys = []
        for x in range(max(0, length - window) if window else 0, min(length, cols * page)):
            p = int(pages[r, x // page])
            if 0 <= p < n:
                keys.append((p, x % page))
        if not keys:
            continue
        at = torch.tensor(keys)
        for h in range(hq):
            g = h // (hq // hk)
            kk, vv = k_cache[at[:, 0], at[:, 1], g].double(), v_cache[at[:, 0], at[:, 1], g].double()
            qq = q[r, h].double()
            s = kk @ qq * scale
            size = kk.abs() @ qq.abs() * abs(scale)
            w = torch.softmax(s, 0)
            out[r, h], lse[r, h] = w @ vv, torch.logsumexp(s, 0)
            # a score: d products and sums, three multiplications, the distance
            # to the maximum; then exp2, within 2^-22, and the weight's split
            ds = float(size.max()) * (d + 2) * 2 * u + float(s.abs().max() + (s.max() - s.min())) * 4 * u
            dw = 2 * ds + 2 * 2.0 ** -22 + exact_split
            sums = len(keys) * 2 * u + 64 * u       # each side's sum, in any order, and the joins
            eo[r, h] = (w @ vv.abs()) * (dw + 2 * sums) + out[r, h].abs() * half_step(q.dtype) + tiny(q.dtype)
            el[r, h] = ds + 2.0 ** -21 + sums + abs(float(lse[r, h])) * 4 * u
    return out, lse, eo, el


def assign(pages, lens, refs, parent, add, page):
    pages, refs = [list(map(int, r)) for r in pages], [int(x) for x in refs]
    rows, cols, n = len(pages), len(pages[0]) if pages else 0, len(refs)
    most = cols * page
    old = [min(max(int(x), 0), most) for x in lens]
    free = [i for i in range(n) if refs[i] == 0]
    left = list(refs)
    ok = lambda i: 0 <= i < n
    for r in range(rows):
        for j in range(-(-old[r] // page)):
            if ok(pages[r][j]):
                left[pages[r][j]] -= 1
    out, lens_out, src, dst, wanted, given = [], [], [], [], 0, 0
    for r in range(rows):
        p = int(parent[r])
        has = 0 <= p < rows
        length = old[p] if has else 0
        new = min(length + max(int(add[r]), 0), most)
        keep = (-(-length // page) if p == r else length // page) if has else 0
        row = [i if ok(i) else -1 for i in (pages[p][:keep] if has else [])]
        a, b = -1, -1
        for j in range(keep, -(-new // page)):
            wanted += 1
            got = free[given] if given < len(free) else -1
            given += got >= 0
            row.append(got)
            if j * page < length and got >= 0 and ok(pages[p][j]):
                a, b = pages[p][j], got
        for i in row:
            if i >= 0:
                left[i] += 1
        out.append(row + [-1] * (cols - len(row)))
        lens_out.append(new)
        src.append(a)
        dst.append(b)
    return out, lens_out, left, src, dst, [wanted, given]


def compact(pages, refs, capacity):
    refs = [int(x) for x in refs]
    n = len(refs)
    live = [i for i in range(n) if refs[i] > 0]
    src = [i for i in live if i >= len(live)]
    dst = [i for i in range(len(live)) if refs[i] <= 0]
    to = {i: i for i in live}
    to.update(zip(src, dst))
    left = [0] * n
    for i in live:
        left[to[i]] = refs[i]
    fill = [-1] * (capacity - len(src))
    return [[to.get(int(i), -1) for i in row] for row in pages], left, src + fill, dst + fill, [len(live), len(src)]
