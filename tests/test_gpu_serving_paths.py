"""The serving operators on the sizes at which the library takes another way than
on the small ones of test_gpu_serving.py: several kv heads to a work-group, rows
taken whole, each join of a row's segments, instances that read and write past
the caches.  Each case says which way it is for, worked out from the rules that
ecmd_serving.cpp and ecmd_kern_attention.h state, so that a case that no longer
takes it fails.  The definitions are those of serving_oracle.py, in 64 bits on
the GPU."""
import math
import random

import pytest
import torch

import elementwise_tensor_commands_amd as E
import serving_oracle as O

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
I32 = torch.int32
MUCH, STEP = 6144, 128


def ints(a):
    return torch.tensor(a, dtype=I32).cuda()


def within(got, want, bound, what=""):
    off = (got.double() - want).abs()
    off = torch.where(torch.isinf(want) & (got == want), torch.zeros_like(off), off)
    bad = ~(off <= bound)
    assert not bool(bad.any()), "%s: %d of %d off, worst %g against a bound of %g" % (
        what, int(bad.sum()), bad.numel(), float(off[bad].max()), float(bound[bad].min()))


# ---------------------------------------------------------------------------
# Attention.

def way(lens, cols, page, hq, hk, d, dv, size, window=0):
    """How the steps of these rows are dealt out and joined."""
    b, tiles = len(lens), -(-(hq // hk) // 16)
    heads, held = hk * tiles, cols * page
    keys = min(held, window) if window else held
    steps = -(-keys // STEP)
    most = max(1, steps * b)
    row_bytes = keys * (d + dv) * size
    if (steps <= 6 and row_bytes <= 256 << 10) or (steps <= 8 and row_bytes <= 512 << 10 and b * heads >= 512) or b > 2048:
        return dict(direct=True, shift=0, share=None, join=None, most=1)
    shift = 2 if heads % 4 == 0 else 1 if heads % 2 == 0 else 0
    runs, runs_much = (min(max(1, 768 // n), most, 1024) for n in (heads, heads >> shift))
    each = [-(-(min(x, held) - (max(0, min(x - window, held)) if window else 0)) // STEP) if x > 0 else 0 for x in lens]
    total, longest = sum(each), max(each)
    segments = min(max(runs, runs_much), steps)
    join = 0 if segments <= 16 else 2 if b * hq * -(-dv // 32) <= 512 else 1 if max(runs, runs_much) > 12 * b else 0
    if 128 <= b * heads <= 2048 and total * 5 >= longest * b * 4:
        return dict(direct=False, shift=0, share=0, join=join, most=1)
    much = total * heads >= MUCH
    share = -(-total // (runs_much if much else runs))
    if longest <= 2 * share and b <= (runs_much if much else runs):
        share = 0
    at, cuts = 0, [0]
    for n in each:                                                 # segments of each row
        cuts.append(0 if not n else 1 if not share else (at + n - 1) // share - at // share + 1)
        at += n
    return dict(direct=False, shift=shift if much else 0, share=share, join=join, most=max(cuts))


def slots(pages, lens, n, page, window, r):
    """Pages and slots of the positions that row r attends to."""
    x = torch.arange(max(0, lens[r] - window) if window else 0, max(0, min(lens[r], pages.shape[1] * page)), device="cuda")
    at = pages[r].long()[x // page]
    ok = (at >= 0) & (at < n)
    return at[ok], x[ok] % page


def reference(q, k, v, pages, lens, scale, window):
    """serving_oracle.attention, a row's heads at once; binary16 weights held to 2^-22 of themselves or
    2^-47 of the largest, others in 24 bits."""
    b, hq, d = q.shape
    n, page, hk, dv = v.shape
    u, (split, floor) = 2.0 ** -24, (2.0 ** -22, 2.0 ** -47) if q.dtype == torch.float16 else (0.0, 0.0)
    out = torch.zeros(b, hq, dv, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    eo, el = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(b):
        at, x = slots(pages, lens, n, page, window, r)
        if len(x) == 0:
            continue
        qq = q[r].double().view(hk, hq // hk, d)
        kk = k[at, x].double().permute(1, 2, 0).contiguous()
        vv = v[at, x].double().transpose(0, 1).contiguous()
        s = torch.matmul(qq, kk) * scale
        size = torch.matmul(qq.abs(), kk.abs()).amax(-1) * abs(scale)
        w = torch.softmax(s, -1)
        o = torch.matmul(w, vv)
        ls = torch.logsumexp(s, -1)
        ds = size * (d + 2) * 2 * u + (s.abs().amax(-1) + s.amax(-1) - s.amin(-1)) * 4 * u
        dw, sums = 2 * ds + 2 * 2.0 ** -22 + split, len(x) * 2 * u + 64 * u
        out[r], lse[r] = o.view(hq, dv), ls.view(hq)
        eo[r] = (torch.matmul(w, vv.abs()) * (dw + 2 * sums)[..., None] + floor * vv.abs().sum(1)[:, None]
                 + o.abs() * O.half_step(q.dtype) + O.tiny(q.dtype)).view(hq, dv)
        el[r] = (ds + 2.0 ** -21 + sums + ls.abs() * 4 * u).view(hq)
    return out, lse, eo, el


def attention(seed, dtype, lens, hq, hk, d, dv, page, cols, window=0, holes=0, stream=False, pool=None):
    """Rows whose tables draw from one pool of pages; stream: a pool that spans more than the caches."""
    dt, b = DT[dtype], len(lens)
    g, rng = torch.Generator(device="cuda").manual_seed(seed), random.Random(seed)
    used = max(-(-max(x, 1) // page) for x in lens)
    n = pool or min(used + 3, cols + 3)
    pages = torch.full((b, cols), -1, dtype=I32)
    for r in range(b):
        here = min(cols, -(-max(lens[r], 0) // page))
        pages[r, :here] = torch.tensor([rng.randrange(n) for _ in range(here)], dtype=I32)
    for i in range(holes):
        r = rng.randrange(b)
        pages[r, rng.randrange(max(1, min(cols, -(-max(lens[r], 1) // page))))] = [-1, n, -2147483648, 2147483647][i % 4]
    def cache(width):
        inner = page * hk * width
        step = inner if not stream else max(inner, -(-(1 << 28) // (n - 1) // dt.itemsize) + 8)
        flat = torch.empty((n - 1) * step + inner, dtype=dt, device="cuda")
        c = flat.as_strided((n, page, hk, width), (step, hk * width, width, 1))
        c.copy_(torch.randn(n, page, hk, width, generator=g, device="cuda"))
        return c
    k, v = cache(d), cache(dv)
    q = (torch.randn(b, hq, d, generator=g, device="cuda") * torch.linspace(0.5, 2.5, hq, device="cuda")[:, None]).to(dt)
    pages = pages.cuda()
    out = torch.full((b, hq, dv), math.nan, dtype=dt, device="cuda")
    lse = torch.full((b, hq), math.nan, device="cuda")
    E.paged_attention(q, k, v, pages, ints(lens), out, lse=lse, window=window)
    want, want_lse, eo, el = reference(q, k, v, pages, lens, d ** -0.5, window)
    within(out, want, eo, "out")
    within(lse, want_lse, el, "lse")
    again = torch.empty_like(out)
    E.paged_attention(q, k, v, pages, ints(lens), again, window=window)
    same = torch.equal(again, out)
    assert same
    # Every position once: with scale 0 all weights are equal, and sums of small whole numbers exact.
    v.copy_(torch.randint(-8, 9, v.shape, generator=g, device="cuda"))
    E.paged_attention(q, k, v, pages, ints(lens), out, lse=lse, scale=0.0, window=window)
    for r in range(b):
        at, x = slots(pages, lens, n, page, window, r)
        # a quotient of tensors: torch divides by a number as a product with its reciprocal
        mean = (v[at, x].double().sum(0) / torch.full((), max(1, len(x)), dtype=torch.float64, device="cuda")).float()
        same = (out[r].view(hk, hq // hk, dv) == mean.to(dt)[:, None]).all().item()
        assert same, r
        count = math.log(len(x)) if len(x) else -math.inf
        assert all(abs(z - count) <= (count + 1) * 2.0 ** -21 or z == count for z in lse[r].tolist()), r


def ragged(seed, b, lo, hi):
    rng = random.Random(seed)
    lens = [rng.randint(lo, hi) for _ in range(b)]
    lens[b // 2], lens[b // 3] = 0, 1
    return lens


@pytest.mark.parametrize("stream", [False, True], ids=["cached", "past"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("heads,shift", [((8, 4, 64, 64), 2), ((12, 6, 81, 96), 1), ((64, 2, 33, 64), 2), ((15, 3, 128, 128), 0),
                                         ((4, 2, 200, 130), 1), ((16, 4, 192, 128), 2), ((8, 8, 80, 64), 2)],
                         ids=lambda x: "-".join(map(str, x)) if isinstance(x, tuple) else str(x))
def test_attention_with_much_to_read(heads, shift, dtype, stream):
    """Ragged rows, those of a run cut and whole, with several heads to a work-group where they allow it."""
    hq, hk, d, dv = heads
    many = hk * -(-(hq // hk) // 16)
    b = 1 + 2 * MUCH // many // 50
    lens, cols, page = ragged(sum(heads), b, 1, 12700), 800, 16
    w = way(lens, cols, page, hq, hk, d, dv, DT[dtype].itemsize)
    assert not w["direct"] and w["shift"] == shift and w["share"] > 0 and w["most"] > 1
    attention(sum(heads), dtype, lens, hq, hk, d, dv, page, cols, holes=40, stream=stream)


@pytest.mark.parametrize("stream", [False, True], ids=["cached", "past"])
@pytest.mark.parametrize("dtype", list(DT))
def test_attention_runs_of_many_short_rows(dtype, stream):
    """Runs that span rows, empty ones among them, each a segment or a part of one; windows."""
    for hq, hk, d, dv, window in ((8, 4, 64, 64, 0), (6, 2, 81, 41, 1200), (5, 1, 96, 64, 0)):
        heads = hk
        lens = ragged(hk, 2000, 0, 1300)
        for r in range(100, 160):
            lens[r] = 0
        lens[1999] = 6000
        w = way(lens, 400, 17, hq, hk, d, dv, DT[dtype].itemsize, window)
        assert not w["direct"] and w["share"] > 5 and w["shift"] == {4: 2, 2: 1, 1: 0}[heads]
        attention(hk, dtype, lens, hq, hk, d, dv, 17, 400, window=window, holes=200, stream=stream)


@pytest.mark.parametrize("stream", [False, True], ids=["cached", "past"])
@pytest.mark.parametrize("dtype", list(DT))
def test_attention_rows_taken_whole(dtype, stream):
    """Rows of nearly one length; and rows that are about a run long, by one head and by several."""
    rng = random.Random(5)
    for hq, hk, d, dv in ((8, 4, 128, 128), (9, 9, 66, 80), (34, 2, 64, 64)):
        lens = [rng.randint(1540, 1700) for _ in range(64)]
        w = way(lens, 110, 16, hq, hk, d, dv, DT[dtype].itemsize)
        assert not w["direct"] and w["share"] == 0 and w["shift"] == 0
        attention(1, dtype, lens, hq, hk, d, dv, 16, 110, holes=9, stream=stream)
    lens = [rng.randint(260, 512) for _ in range(700)]
    lens[5] = lens[699] = 0
    w = way(lens, 256, 16, 8, 4, 64, 72, DT[dtype].itemsize)
    assert not w["direct"] and w["share"] == 0 and w["shift"] == 2
    attention(2, dtype, lens, 8, 4, 64, 72, 16, 256, holes=9, stream=stream)
    lens = [rng.randint(1, 250) for _ in range(30)]
    lens[7] = 0
    w = way(lens, 256, 16, 6, 2, 64, 64, DT[dtype].itemsize)
    assert not w["direct"] and w["share"] == 0 and w["shift"] == 0
    attention(3, dtype, lens, 6, 2, 64, 64, 16, 256, stream=stream)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("join,heads,b,hi", [(1, (32, 2, 64, 96), 8, 6300), (1, (32, 4, 80, 64), 9, 30000), (1, (24, 3, 96, 200), 8, 9000),
                                             (2, (4, 2, 64, 64), 3, 50000), (2, (8, 1, 128, 33), 8, 2500), (0, (32, 8, 64, 64), 70, 3000)],
                         ids=str)
def test_attention_joins(dtype, join, heads, b, hi):
    """Each way of joining a row's segments, of few and of many."""
    hq, hk, d, dv = heads
    lens = [hi] + ragged(join + b, b - 1, 1, hi)
    cols = -(-hi // 32) + 5
    w = way(lens, cols, 32, hq, hk, d, dv, DT[dtype].itemsize)
    assert not w["direct"] and w["join"] == join and w["most"] > (4 if join == 0 else 16)
    attention(b, dtype, lens, hq, hk, d, dv, 32, cols, holes=5)


@pytest.mark.parametrize("dtype", list(DT))
def test_attention_of_many_direct_rows(dtype):
    """No runs: short tables of many rows, and more rows than prefixes fit, long ones among them."""
    size = DT[dtype].itemsize
    for hq, hk, d, dv, b, cols, hi in ((8, 4, 64, 64, 200, 64, 1024), (4, 4, 33, 80, 2049, 300, 300)):
        lens = ragged(b, b, 0, hi)
        if b > 2048:
            lens[7] = 4800
        assert way(lens, cols, 16, hq, hk, d, dv, size)["direct"]
        attention(b, dtype, lens, hq, hk, d, dv, 16, cols, holes=30, stream=True)


# ---------------------------------------------------------------------------
# Rotary positions, the append and the page copies past the caches (64 MiB moved).

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_past_the_caches(dtype, layout):
    dt = DT[dtype]
    for b, t, h, d, m in ((2, 2100, 33, 128, 64), (1, 4100, 40, 130, 50), (3, 1500, 48, 83, 40), (1, 9000, 30, 72, 12)):
        b *= 2 if dt != torch.float32 else 1
        assert 2 * b * t * h * d * dt.itemsize > 64 << 20
        g = torch.Generator(device="cuda").manual_seed(d)
        x = torch.randn(b, t, (h + 1) * d, generator=g, device="cuda").to(dt)[:, :, :h * d].unflatten(2, (h, d))
        pos = torch.randint(0, 2000000, (b, t), generator=g, dtype=I32, device="cuda")
        freq = E.rope_frequencies(2 * m).cuda()
        want, bound = O.rope(x, pos, freq, layout, 1.25, d % 2 == 0)
        out = torch.full((b, t, h, d), math.nan, dtype=dt, device="cuda")
        E.rope(x, pos, freq, out, layout=layout, mscale=1.25, inverse=d % 2 == 0)
        within(out, want, bound, (b, t, h, d, m))
        E.rope(x, pos, freq, x, layout=layout, mscale=1.25, inverse=d % 2 == 0)
        same = torch.equal(x, out)
        assert same, (b, t, h, d, m)


def test_rope_of_more_tokens_than_a_launch_has_groups():
    """138 GB turned in place, where a token alone would fill a work-group: two to a group then."""
    tokens, d, m = (1 << 24) + 5, 4104, 2048
    x = torch.empty(1, tokens, 1, d, dtype=torch.float16, device="cuda")
    g = torch.Generator().manual_seed(3)
    at = torch.cat([torch.randint(0, tokens, (200,), generator=g), torch.tensor([0, 1, tokens // 2, tokens - 2, tokens - 1])]).unique().cuda()
    here = torch.randn(1, len(at), 1, d, generator=g).half().cuda()
    x[:, at] = here
    pos = torch.arange(tokens, dtype=I32, device="cuda").view(1, tokens)
    freq = E.rope_frequencies(2 * m).cuda()
    E.rope(x, pos, freq, x)
    want, bound = O.rope(here, pos[:, at], freq, "half")
    got = x[:, at].clone()
    del x, pos
    torch.cuda.empty_cache()
    within(got, want, bound)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_append_past_the_caches(dtype, layout):
    """q, k and v of one packed projection, q turned in place, and apart; whole and odd widths."""
    dt = DT[dtype]
    for hq, hk, d, dv, m in ((16, 4, 128, 128, 64), (12, 3, 90, 90, 41), (12, 3, 90, 83, 20)):
        rows, page, cols = 7, 48, 40
        tokens = rows * cols * page - 500
        assert 2 * tokens * ((hq + hk) * d + hk * dv) * dt.itemsize > 64 << 20
        g = torch.Generator(device="cuda").manual_seed(d + dv)
        n = rows * cols + 2
        pages = torch.randperm(n, generator=g, device="cuda")[:rows * cols].view(rows, cols).to(I32)
        pages[3, 7], pages[4, 0] = -1, n
        at = torch.randperm(rows * cols * page, generator=g, device="cuda")[:tokens]
        row, pos = (at // (cols * page)).to(I32), (at % (cols * page)).to(I32)
        row[::97], pos[5::101] = rows, -1                          # padding
        if dv == d:
            qkv = torch.randn(tokens, hq + 2 * hk, d, generator=g, device="cuda").to(dt)
            q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        else:
            q, k, v = (torch.randn(tokens, a, w, generator=g, device="cuda").to(dt) for a, w in ((hq, d), (hk, d), (hk, dv)))
        kc, vc = (torch.randn(n, page, hk, w, generator=g, device="cuda").to(dt) for w in (d, dv))
        freq = E.rope_frequencies(2 * m).cuda()
        q_want, q_bound = O.rope(q, pos, freq, layout, 0.9)
        k_turned, k_err = O.rope(k, pos, freq, layout, 0.9)
        k_want, k_bound, v_want = kc.double(), torch.zeros_like(kc, dtype=torch.float64), vc.clone()
        real = (row < rows) & (pos >= 0)
        page_of = pages[torch.where(real, row, 0).long(), torch.where(real, pos, 0).long() // page].long()
        real &= (page_of >= 0) & (page_of < n)
        slot = (page_of * page + pos % page)[real]
        k_want.flatten(0, 1)[slot], k_bound.flatten(0, 1)[slot] = k_turned[real], k_err[real]
        v_want.flatten(0, 1)[slot] = v[real]
        q_out = q if dv == d else torch.full_like(q, math.nan)
        E.rope_append(q, k, v, pos, row, pages, freq, q_out, kc, vc, layout=layout, mscale=0.9)
        within(q_out, q_want, q_bound, "q")
        within(kc, k_want, k_bound, "k")
        same = torch.equal(vc, v_want)
        assert same


def test_page_copy_past_the_caches():
    for shape, dt in (((3000, 16, 4, 128), torch.bfloat16), ((2200, 24, 3, 132), torch.float32)):
        n = shape[0]
        g = torch.Generator(device="cuda").manual_seed(n)
        pools = [torch.randn(shape, generator=g, device="cuda").to(dt) for _ in range(2)]
        ids = torch.randperm(n, generator=g, device="cuda").to(I32)
        src, dst = ids[:n // 2].clone(), ids[n // 2:].clone()
        src[3], dst[4], src[5] = -1, -1, n
        assert (n // 2) * 2 * 2 * pools[0][0].numel() * dt.itemsize > 64 << 20
        want = [p.clone() for p in pools]
        ok = (src >= 0) & (src < n) & (dst >= 0)
        for p in want:
            p[dst[ok].long()] = p[src[ok].long()]
        E.page_copy(pools, src, dst)
        assert all(torch.equal(a, b) for a, b in zip(pools, want))
