"""The serving operators on the GPU against the oracle's definitions in 64 bits
(serving_oracle.py), within bounds counted from the roundings that
include/ecmd_serving.h lists; whole numbers are equal."""
import math
import random

import pytest
import torch

import elementwise_tensor_commands_amd as E
import serving_oracle as O

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
I32 = torch.int32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g).to(dtype)


def ints(a):
    return torch.tensor(a, dtype=I32)


def within(got, want, bound, what=""):
    got = got.detach().cpu().double()
    off = (got - want).abs()
    off = torch.where(torch.isinf(want) & (got == want), torch.zeros_like(off), off)
    bad = ~(off <= bound)
    assert not bool(bad.any()), "%s: %d of %d off, worst %g against a bound of %g" % (
        what, int(bad.sum()), bad.numel(), float(off[bad].max()), float(bound[bad].min()))


# ---------------------------------------------------------------------------
# Rotary positions.

ROPE = [  # b, t, h, d, m
    (1, 1, 1, 2, 1), (1, 1, 1, 1, 0), (2, 3, 4, 128, 64), (3, 5, 7, 81, 20), (1, 2, 3, 80, 40), (2, 1, 40, 96, 32),
    (1, 1030, 2, 64, 32), (2, 600, 3, 33, 16), (1, 3, 2, 300, 149), (0, 3, 2, 8, 4), (2, 0, 2, 8, 4), (1, 4, 1, 4096, 2048),
    (1, 2, 5, 17, 3), (5, 9, 1, 7, 2),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope(dtype, layout):
    for case, (b, t, h, d, m) in enumerate(ROPE):
        g = gen(case)
        extra = case % 3                                           # heads beside these in a packed row
        x = randn(g, b, t, (h + extra) * d, dtype=DT[dtype])[:, :, :h * d].unflatten(2, (h, d))
        pos = torch.randint(0, 2000000 if case % 2 else 50, (b, t), generator=g, dtype=I32)
        freq = E.rope_frequencies(2 * m)
        inverse, mscale = case % 2 == 1, [1.0, 1.25, 0.7][case % 3]
        want, bound = O.rope(x, pos, freq, layout, mscale, inverse)
        xg = torch.empty(b, t, (h + extra) * d, dtype=DT[dtype], device="cuda")[:, :, :h * d].unflatten(2, (h, d))
        xg.copy_(x)
        out = torch.full((b, t, h, d), math.nan, dtype=DT[dtype], device="cuda")
        E.rope(xg, pos.cuda(), freq.cuda(), out, layout=layout, mscale=mscale, inverse=inverse)
        within(out, want, bound, (b, t, h, d, m))
        assert bool((xg.cpu() == x).all())
        E.rope(xg, pos.cuda(), freq.cuda(), xg, layout=layout, mscale=mscale, inverse=inverse)     # in place
        assert bool((xg == out).all()), (b, t, h, d, m)


def test_rope_strides_and_extremes():
    g = gen(1)
    x = randn(g, 3, 6, 4, 24, dtype=torch.bfloat16)
    base = randn(g, 6, 3, 4, 30, dtype=torch.bfloat16).cuda()
    xg = base.transpose(0, 1)[..., 3:27]                            # batch and token swapped, rows off 16 bytes
    xg.copy_(x)
    pos = ints([[-5, 0, 2147483647, -2147483648, 1 << 24, 7]]).expand(3, 6)
    freq = torch.tensor([1.0, 0.0, 1e-9, 0.5, 3.0], dtype=torch.float64)
    want, bound = O.rope(x, pos, freq, "half")
    out = torch.full((4, 3, 6, 27), 9.0, dtype=torch.bfloat16, device="cuda")
    view = out.permute(1, 2, 0, 3)[..., 1:25]
    E.rope(xg, pos.cuda(), torch.stack([freq, freq], 1).cuda()[:, 1], view)
    within(view, want, bound)
    assert bool((out[..., 0] == 9).all() and (out[..., 25:] == 9).all())     # nothing beside the view
    # infinities and NaN stay in their pair
    x = torch.ones(1, 1, 1, 12)
    x[..., 1], x[..., 2] = math.inf, math.nan
    out = torch.zeros(1, 1, 1, 12, device="cuda")
    E.rope(x.cuda(), ints([[3]]).cuda(), E.rope_frequencies(10).cuda(), out)
    assert torch.isfinite(out).flatten().tolist() == [i not in (1, 6, 2, 7) for i in range(12)]


def test_rope_inverse_undoes():
    g = gen(2)
    x = randn(g, 2, 70, 3, 64, dtype=torch.float32).cuda()
    pos = torch.randint(0, 3000000, (2, 70), generator=g, dtype=I32).cuda()
    freq = E.rope_frequencies(48).cuda()
    y, z = torch.empty_like(x), torch.empty_like(x)
    E.rope(x, pos, freq, y, layout="interleaved")
    E.rope(y, pos, freq, z, layout="interleaved", inverse=True)
    # two turns: each within 3.01 half steps of |u| + |v| <= sqrt(2) of the pair's length, twice over
    u, v = O.pairs(x, 24, "interleaved")
    length = torch.sqrt(u * u + v * v).amax().item()
    assert float((z - x).abs().max()) <= 4 * 1.5 * length * 3.01 * 2.0 ** -24


def test_a_backward_pass_notices_what_was_written():
    """A tensor that torch saved for a gradient and that a call wrote afterwards."""
    pos, freq = torch.arange(3, dtype=I32, device="cuda").view(1, 3), E.rope_frequencies(8).cuda()
    x = torch.ones(1, 3, 2, 8, device="cuda")
    w = torch.ones_like(x, requires_grad=True)
    y = (x * w).sum()
    E.rope(x, pos, freq, torch.empty_like(x))                       # only read: as before
    y.backward()
    y = (x * w).sum()
    E.rope(x, pos, freq, x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    # every output of every operator
    args, out = step_state()
    lse = torch.empty(out.shape[:2], device="cuda")
    qkv, kc, vc = torch.ones(2, 6, 8, device="cuda"), torch.zeros(4, 2, 2, 8, device="cuda"), torch.zeros(4, 2, 2, 8, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=I32, device="cuda")
    tables = [i(2, 2), i(2), i(4), i(2), i(2)], [i(2, 2), i(2), i(4), i(2), i(2), i(2)]
    compact = [i(2, 2), i(4)], [i(2, 2), i(4), i(2), i(2), i(2)]
    q_out = torch.empty(2, 2, 8, device="cuda")
    for call, ins, outs in (
            (lambda: E.paged_attention(*args, out, lse=lse), args, [out, lse]),
            (lambda: E.rope_append(qkv[:, :2], qkv[:, 2:4], qkv[:, 4:], i(2), i(2), i(1, 2), freq, q_out, kc, vc), [qkv], [q_out, kc, vc]),
            (lambda: E.page_assign(*tables[0], 2, *tables[1]), *tables), (lambda: E.page_compact(*compact[0], *compact[1]), *compact),
            (lambda: E.page_copy([kc, vc], i(1), i(1) + 1), [], [kc, vc])):
        versions = [t._version for t in [*ins, *outs]]
        call()
        assert [t._version for t in [*ins, *outs]] == versions[:len(ins)] + [n + 1 for n in versions[len(ins):]]


# ---------------------------------------------------------------------------
# The append.

APPEND = [  # tokens, rows, cols, page, hq, hk, d, dv, m
    (1, 1, 1, 1, 1, 1, 1, 1, 0), (64, 64, 4, 16, 32, 8, 128, 128, 64), (37, 3, 9, 17, 12, 4, 81, 33, 20),
    (700, 5, 40, 32, 8, 2, 96, 64, 32), (5, 2, 3, 1, 3, 3, 64, 64, 32), (0, 2, 3, 4, 2, 1, 8, 8, 4),
    (2000, 4, 33, 64, 6, 1, 40, 80, 10),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_append(dtype, layout):
    for case, (tokens, rows, cols, page, hq, hk, d, dv, m) in enumerate(APPEND):
        g, rng, dt = gen(case), random.Random(case), DT[dtype]
        n = rows * cols + 3
        ids = list(range(n))
        rng.shuffle(ids)
        pages = ints(ids[:rows * cols]).view(rows, cols)
        holes = rng.sample(range(rows * cols), rows * cols // 8)
        for k, x in enumerate(holes):
            pages.view(-1)[x] = [-1, n, -2147483648, 2147483647][k % 4]
        slots = [(r, p) for r in range(rows) for p in range(cols * page)]
        rng.shuffle(slots)
        slots = slots[:tokens]
        slots += [(rng.randrange(rows), cols * page + 5)] * (tokens - len(slots))
        for k in range(0, len(slots), 9):                            # padding of each kind
            slots[k] = [(-1, 0), (rows, 0), (0, -1), (0, cols * page), (0, 2147483647), (2147483647, 3)][k // 9 % 6]
        row, pos = ints([s[0] for s in slots]), ints([s[1] for s in slots])
        qkv = randn(g, tokens, hq + hk, d, dtype=dt)
        q, k, v = qkv[:, :hq], qkv[:, hq:], randn(g, tokens, hk, dv, dtype=dt)
        freq = E.rope_frequencies(2 * m)
        kc, vc = randn(g, n, page, hk, d, dtype=dt), randn(g, n, hk, page, dv, dtype=dt)
        q_want, q_bound = O.rope(q, pos, freq, layout, 1.1)
        k_turned, k_err = O.rope(k, pos, freq, layout, 1.1)
        k_want, k_bound, v_want = kc.double(), torch.zeros_like(kc, dtype=torch.float64), vc.double()
        for t, (r, p) in enumerate(slots):
            if not (0 <= r < rows and 0 <= p < cols * page) or not 0 <= int(pages[r, p // page]) < n:
                continue
            at = int(pages[r, p // page])
            k_want[at, p % page], k_bound[at, p % page] = k_turned[t], k_err[t]
            v_want[at, :, p % page] = v[t].double()
        qkv_g, kg, vg = qkv.cuda(), kc.cuda(), vc.cuda()
        out = torch.full((tokens, hq, d), math.nan, dtype=dt, device="cuda")
        args = (v.cuda(), pos.cuda(), row.cuda(), pages.cuda(), freq.cuda())
        E.rope_append(qkv_g[:, :hq], qkv_g[:, hq:], *args, out, kg, vg.transpose(1, 2), layout=layout, mscale=1.1)
        within(out, q_want, q_bound, ("q", case))
        within(kg, k_want, k_bound, ("k", case))
        assert bool((vg.cpu().double() == v_want).all()), case
        E.rope_append(qkv_g[:, :hq], qkv_g[:, hq:], *args, qkv_g[:, :hq], kg, vg.transpose(1, 2), layout=layout, mscale=1.1)
        assert bool((qkv_g[:, :hq] == out).all()), case              # q in place


@pytest.mark.parametrize("hq,hk,d,dv", [(0, 2, 8, 8), (2, 1, 8, 0), (0, 0, 8, 8), (3, 0, 8, 8), (2, 1, 0, 8)])
def test_append_of_nothing(hq, hk, d, dv):
    """No query heads, no kv heads, or heads without elements: the rest is done."""
    z = lambda *s: torch.ones(*s, device="cuda")
    kc, vc, out = z(4, 2, hk, d) * 0, z(4, 2, hk, dv) * 0, z(3, hq, d) * 0
    m = torch.zeros(0, dtype=torch.float64, device="cuda")
    E.rope_append(z(3, hq, d), z(3, hk, d), z(3, hk, dv), ints([0, 1, 3]).cuda(), ints([0, 0, -1]).cuda(),
                  ints([[2, 1]]).cuda(), m, out, kc, vc)
    assert bool((out == 1).all())
    for c in (kc, vc):
        assert bool((c[2] == 1).all()) and not bool(c[[0, 1, 3]].any())


# ---------------------------------------------------------------------------
# Attention.

def attention_case(seed, dt, b, hq, hk, d, dv, page, lens, window=0, holes=0, cols=None, sharp=1.5):
    """Inputs whose every slot that no row may look at is NaN."""
    g, rng = gen(seed), random.Random(seed)
    cols = cols or max(1, max(-(-max(x, 1) // page) for x in lens))
    n = b * cols + 2
    ids = list(range(n))
    rng.shuffle(ids)
    pages = ints(ids[:b * cols]).view(b, cols)
    for k in range(holes):
        pages[rng.randrange(b), rng.randrange(cols)] = [-1, n, -2147483648, 2147483647][k % 4]
    q = (torch.randn(b, hq, d, generator=g) * sharp).to(dt)
    k, v = randn(g, n, page, hk, d, dtype=dt), randn(g, n, page, hk, dv, dtype=dt)
    used = torch.zeros(n, page, dtype=torch.bool)
    for r in range(b):
        for x in range(max(0, lens[r] - window) if window else 0, min(lens[r], cols * page)):
            at = int(pages[r, x // page])
            if 0 <= at < n:
                used[at, x % page] = True
    k[~used], v[~used] = math.nan, math.nan
    return q, k, v, pages, ints(lens)


def check_attention(q, k, v, pages, lens, scale=None, window=0, gpu=None, what=""):
    b, hq, d = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    want, lse, eo, el = O.attention(q, k, v, pages, lens, scale, window)
    out = torch.full((b, hq, v.shape[-1]), math.nan, dtype=q.dtype, device="cuda")
    ls = torch.full((b, hq), math.nan, device="cuda")
    kg, vg = gpu or (k.cuda(), v.cuda())
    args = (q.cuda(), kg, vg, pages.cuda(), lens.cuda())
    E.paged_attention(*args, out, lse=ls, scale=scale, window=window)
    within(out, want, eo, ("out", what))
    within(ls, lse, el, ("lse", what))
    again = torch.empty_like(out)
    E.paged_attention(*args, again, scale=scale, window=window)      # no lse; the same bits
    assert torch.equal(again, out), what
    return out


HEADS = [  # hq, hk, d, dv
    (1, 1, 1, 1), (3, 3, 64, 64), (8, 2, 128, 128), (12, 4, 96, 64), (16, 1, 80, 80), (17, 1, 33, 41), (40, 1, 64, 128),
    (6, 2, 192, 128), (4, 1, 256, 256), (2, 2, 200, 7), (8, 8, 81, 96), (4, 2, 128, 64), (4, 2, 7, 200), (32, 8, 96, 96),
    (5, 5, 192, 192), (2, 1, 130, 130), (2, 1, 64, 60),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "-".join(map(str, h)))
def test_attention_heads(dtype, heads):
    hq, hk, d, dv = heads
    lens = [0, 1, 2, 15, 16, 17, 33, 130, 300]
    check_attention(*attention_case(hq + d, DT[dtype], len(lens), hq, hk, d, dv, 16, lens), what=heads)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("page", [1, 2, 16, 17, 64, 100])
def test_attention_pages_and_holes(dtype, page):
    lens = [257, 0, 31, 32, 1000, -7, 64, 2]
    check_attention(*attention_case(page, DT[dtype], 8, 4, 2, 64, 64, page, lens, holes=9), what=page)
    check_attention(*attention_case(page, DT[dtype], 8, 4, 2, 64, 64, page, [x + 500 for x in lens], cols=3), what="past the table")


@pytest.mark.parametrize("dtype", list(DT))
def test_attention_windows(dtype):
    lens = [257, 0, 1, 100, 1500, 640]
    for window in (1, 2, 33, 100, 128, 1000, 2147483647):
        case = attention_case(window % 997, DT[dtype], 6, 6, 3, 80, 64, 17, lens, window=window, holes=3)
        check_attention(*case, window=window, what=window)
    # longer than its table, the window past it: nothing to attend to
    case = attention_case(3, DT[dtype], 2, 2, 1, 64, 64, 16, [5000, 40], window=64, cols=3)
    out = check_attention(*case, window=64, what="past")
    assert bool((out[0] == 0).all())


@pytest.mark.parametrize("dtype", list(DT))
def test_attention_long_and_split(dtype):
    check_attention(*attention_case(1, DT[dtype], 1, 4, 2, 64, 64, 64, [40001]), what="one long row")
    check_attention(*attention_case(2, DT[dtype], 3, 2, 1, 128, 128, 16, [9000, 0, 131]), what="ragged")
    check_attention(*attention_case(3, DT[dtype], 2, 2, 2, 32, 32, 16, [129, 5], cols=8192), what="a wide table, short rows")


@pytest.mark.parametrize("dtype", list(DT))
def test_attention_sharp_and_scaled(dtype):
    case = attention_case(4, DT[dtype], 3, 4, 2, 64, 64, 16, [700, 65, 3], sharp=8.0)
    check_attention(*case, what="sharp")
    for scale in (0.0, -0.3, 1.0):
        check_attention(*case, scale=scale, what=scale)


def test_attention_strides():
    dt = torch.bfloat16
    q, k, v, pages, lens = attention_case(6, dt, 4, 8, 2, 128, 64, 16, [100, 33, 0, 257], holes=2)
    n = k.shape[0]
    # [N, kv heads, page, d]; keys and values side by side; a table and lengths with strides
    kg = k.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    vg = torch.full((n, 16, 2, 2, 64), math.nan, dtype=dt, device="cuda")
    vg[:, :, 1] = v.cuda()
    check_attention(q, k, v, pages, lens, gpu=(kg, vg[:, :, 1]))
    want, lse, eo, el = O.attention(q, k, v, pages, lens, 128 ** -0.5)
    out = torch.full((8, 5, 70), 3.0, dtype=dt, device="cuda")
    view = out.transpose(0, 1)[:4, :, 2:66]
    ls = torch.zeros(8, 4, device="cuda").t()
    wide = torch.stack([pages, pages + 1], 2).cuda()[:, :, 0]
    E.paged_attention(torch.cat([q, q], 2).cuda()[..., 128:], k.cuda(), v.cuda(), wide, torch.stack([lens, lens], 1).cuda()[:, 0],
                      view, lse=ls)
    within(view, want, eo)
    within(ls, lse, el)
    assert bool((out[:, 4] == 3).all() and (out[..., :2] == 3).all() and (out[..., 66:] == 3).all())
    # rows that share one table, as a prompt's tokens do
    same = pages[:1].expand(4, -1)
    k[:], v[:] = randn(gen(1), *k.shape, dtype=dt), randn(gen(2), *v.shape, dtype=dt)
    check_attention(q, k, v, same, lens)


def test_attention_special_values():
    q, k, v, pages, lens = attention_case(7, torch.float32, 3, 2, 1, 64, 64, 16, [40, 40, 200])
    at = int(pages[0, 1])
    k[at, 3] = -math.inf * q[0, 0].sign()                          # a key of weight 0 for head 0
    v[int(pages[1, 0]), 2, 0, 5] = math.nan                        # a NaN that is attended to stays in its column
    v[int(pages[2, 0]), 2, 0, 6] = math.inf
    out = torch.empty(3, 2, 64, device="cuda")
    E.paged_attention(q.cuda(), k.cuda(), v.cuda(), pages.cuda(), lens.cuda(), out)
    out = out.cpu()
    assert bool(torch.isfinite(out[0, 0]).all())
    keep = torch.arange(64) != 5
    assert bool(torch.isnan(out[1, :, 5]).all() and torch.isfinite(out[1][:, keep]).all())
    assert bool((out[2, :, 6] == math.inf).all() and torch.isfinite(out[2][:, torch.arange(64) != 6]).all())


@pytest.mark.parametrize("dtype", list(DT))
def test_attention_infinite_values(dtype):
    """An infinity in a value that is attended to gives an infinity in its column, a NaN or two
    infinities of both signs a NaN, whatever the weight; the other columns are as without them."""
    d, dv = 64, 72
    for seed, lens in enumerate(([1, 2, 40, 300], [900, 64, 31, 33])):
        q, k, v, pages, lens = attention_case(70 + seed, DT[dtype], 4, 4, 2, d, dv, 16, lens, sharp=2.0)
        at = lambda r, x: (int(pages[r, x // 16]), x % 16)
        last = [int(x) - 1 for x in lens]
        clean = v.clone()
        for r in range(4):
            for c in (1, 7, 8, 70):
                v[at(r, last[r] // 2)][0, c] = math.inf
            v[at(r, last[r])][1, 3] = -math.inf
            v[at(r, 0)][0, 5] = math.nan
            v[at(r, 0)][1, 6], v[at(r, last[r])][1, 6] = math.inf, -math.inf     # of a row of one position: -inf
        out = torch.empty(4, 4, dv, dtype=DT[dtype], device="cuda")
        E.paged_attention(q.cuda(), k.cuda(), v.cuda(), pages.cuda(), lens.cuda(), out)
        out = out.cpu()
        want, _, eo, _ = O.attention(q, k, clean, pages, lens, d ** -0.5)
        for r in range(4):
            for h in range(4):
                special = {1: math.inf, 7: math.inf, 8: math.inf, 70: math.inf, 5: math.nan} if h < 2 else {
                    3: -math.inf, 6: math.nan if last[r] else -math.inf}
                for c, x in special.items():
                    got = float(out[r, h, c])
                    assert got == x or (math.isnan(x) and math.isnan(got)), (seed, r, h, c, got)
                keep = torch.tensor([c not in special for c in range(dv)])
                within(out[r, h][keep], want[r, h][keep], eo[r, h][keep], (seed, r, h))


def test_attention_infinite_value_of_small_weight():
    """The same far below the largest weight, down to 2^-100 of it."""
    for dtype in DT.values():
        for bits in (20, 37, 45, 100):
            k = torch.zeros(2, 16, 1, 64, dtype=dtype)
            v = torch.zeros(2, 16, 1, 64, dtype=dtype)
            k[..., 0] = -bits * math.log(2.0)
            k[0, 5, 0, 0] = 0.0
            v[0, 9, 0, 3], v[1, 9, 0, 4] = math.inf, -math.inf
            q = torch.zeros(1, 1, 64, dtype=dtype)
            q[..., 0] = 1.0
            out = torch.empty(1, 1, 64, dtype=dtype, device="cuda")
            E.paged_attention(q.cuda(), k.cuda(), v.cuda(), ints([[0, 1]]).cuda(), ints([30]).cuda(), out, scale=1.0)
            assert out[0, 0].tolist() == [0.0] * 3 + [math.inf, -math.inf] + [0.0] * 59, (dtype, bits)


def fine_bounds(q, k, v, pages, lens, scale):
    """want, and the bound on the error of a kernel that holds weights in 22 bits or more, of the
    row's largest weight not below 2^-47, whatever the type: the oracle's bound for binary32 inputs of
    these values, the weights' share of the values' size, and the output's rounding."""
    dt = q.dtype
    want, _, eo, _ = O.attention(q.float(), k.float(), v.float(), pages, lens, scale)
    size, _, _, _ = O.attention(q.float(), k.float(), v.float().abs(), pages, lens, scale)
    floor = 2.0 ** -47 * float(v.float().abs().max()) * int(max(lens))
    return want, eo + size * 2.0 ** -22 + floor + want.abs() * O.half_step(dt) + O.tiny(dt)


@pytest.mark.parametrize("dtype", list(DT))
def test_attention_many_small_weights(dtype):
    """One key in 32 with nearly all of the weight and value 0; the others, far below, make the output."""
    dt, n, d = DT[dtype], 2048, 64
    pages = torch.arange(n // 16, dtype=I32).view(1, -1)
    for bits, size in ((18, 1.0), (22, 500.0), (26, 6000.0), (30, 60000.0), (34, 60000.0)):
        g = gen(bits)
        k, v = torch.zeros(n // 16, 16, 1, d), torch.rand(n // 16, 16, 1, d, generator=g) * 0.5 + 0.5
        k[..., 0] = -bits * math.log(2.0) + torch.rand(n // 16, 16, 1, generator=g) * 0.4
        k[::2, 7, 0, 0], v[::2, 7] = 0.0, 0.0
        q = torch.zeros(1, 2, d)
        q[:, 0, 0], q[:, 1, 0] = 1.0, 0.75
        q, k, v = q.to(dt), k.to(dt), (v * size).to(dt)
        want, bound = fine_bounds(q, k, v, pages, [n], 1.0)
        out = torch.empty(1, 2, d, dtype=dt, device="cuda")
        E.paged_attention(q.cuda(), k.cuda(), v.cuda(), pages.cuda(), ints([n]).cuda(), out, scale=1.0)
        within(out, want, bound, (bits, size))


@pytest.mark.parametrize("dtype", list(DT))
def test_attention_values_that_cancel(dtype):
    """Two keys of nearly one weight, values 1 and -1: what is left, tanh(s / 2), shows the weights' error."""
    dt, b = DT[dtype], 16
    s = (torch.arange(1, b + 1) * 1.1e-4 * torch.tensor([1.0, -1.0]).repeat(b // 2)).to(dt)
    k, v = torch.zeros(b, 16, 1, 64, dtype=dt), torch.zeros(b, 16, 1, 64, dtype=dt)
    k[:, 0, 0, 5], v[:, 0], v[:, 1] = s, 1.0, -1.0
    q = torch.zeros(b, 1, 64, dtype=dt)
    q[..., 5] = 1.0
    out = torch.empty(b, 1, 64, dtype=dt, device="cuda")
    E.paged_attention(q.cuda(), k.cuda(), v.cuda(), torch.arange(b, dtype=I32).view(b, 1).cuda(), ints([2] * b).cuda(), out, scale=1.0)
    want = torch.tanh(s.double() / 2).view(b, 1, 1).expand(b, 1, 64)
    # each weight: a score of three roundings and a difference, exp2 within 2^-22, held to 2^-22; the
    # difference of two weights over their sum, three roundings; the output's
    u = 2.0 ** -24
    bound = s.double().abs().view(b, 1, 1) * 4 * u + 2.0 ** -21 + want.abs() * (4 * u + O.half_step(dt)) + O.tiny(dt)
    within(out, want, bound)


def test_attention_nothing_to_read():
    for n, cols in ((0, 3), (4, 0), (0, 0)):
        out = torch.full((2, 4, 8), 5.0, device="cuda")
        lse = torch.zeros(2, 4, device="cuda")
        E.paged_attention(torch.ones(2, 4, 8, device="cuda"), torch.zeros(n, 16, 2, 8, device="cuda"),
                          torch.zeros(n, 16, 2, 8, device="cuda"), torch.zeros(2, cols, dtype=I32, device="cuda"),
                          ints([7, 9]).cuda(), out, lse=lse)
        assert bool((out == 0).all() and (lse == -math.inf).all())
    E.paged_attention(torch.ones(0, 4, 8, device="cuda"), torch.zeros(3, 16, 2, 8, device="cuda"),
                      torch.zeros(3, 16, 2, 8, device="cuda"), torch.zeros(0, 2, dtype=I32, device="cuda"),
                      torch.zeros(0, dtype=I32, device="cuda"), torch.zeros(0, 4, 8, device="cuda"))


def test_offsets_past_32_bits():
    """Pages more than 2^32 bytes into the cache: append, attend, copy."""
    page, hk, d = 64, 8, 128
    n = (1 << 33) // (page * hk * d * 2) + 40
    kc, vc = (torch.empty(n, page, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = [n - 1, 3, n // 2 + 9, n - 2]
    g = gen(9)
    k, v = randn(g, 4 * page, hk, d, dtype=torch.bfloat16), randn(g, 4 * page, hk, d, dtype=torch.bfloat16)
    q = randn(g, 1, 16, d, dtype=torch.bfloat16)
    pages, pos = ints([ids]), torch.arange(4 * page, dtype=I32)
    E.rope_append(torch.zeros(4 * page, 1, d, dtype=torch.bfloat16, device="cuda"), k.cuda(), v.cuda(), pos.cuda(),
                  torch.zeros(4 * page, dtype=I32, device="cuda"), pages.cuda(), torch.zeros(0, dtype=torch.float64, device="cuda"),
                  torch.zeros(4 * page, 1, d, dtype=torch.bfloat16, device="cuda"), kc, vc)
    small = (k.view(4, page, hk, d), v.view(4, page, hk, d), ints([[0, 1, 2, 3]]))
    want, _, eo, _ = O.attention(q, *small, [4 * page - 1], d ** -0.5)
    out = torch.empty(1, 16, d, dtype=torch.bfloat16, device="cuda")
    E.paged_attention(q.cuda(), kc, vc, pages.cuda(), ints([4 * page - 1]).cuda(), out)
    within(out, want, eo)
    E.page_copy([kc, vc], ints(ids).cuda(), ints([5, n - 7, 6, n // 2]).cuda())
    E.paged_attention(q.cuda(), kc, vc, ints([[5, n - 7, 6, n // 2]]).cuda(), ints([4 * page - 1]).cuda(), out)
    within(out, want, eo)


# ---------------------------------------------------------------------------
# Pages.

def tables(seed, rows, cols, page, n, live):
    """Page tables with shared pages, holes and counts that match them."""
    rng = random.Random(seed)
    ids = rng.sample(range(n), min(live, n))
    lens = [rng.choice([0, 1, page, cols * page, rng.randint(0, cols * page)]) for _ in range(rows)]
    pages = torch.full((rows, cols), -1, dtype=I32)
    refs = [0] * n
    for r in range(rows):
        for j in range(-(-lens[r] // page)):
            if ids and rng.random() < 0.95:
                pages[r, j] = rng.choice(ids)
                refs[int(pages[r, j])] += 1
    return rng, pages, lens, refs


ASSIGN = [(1, 1, 1, 1), (3, 4, 16, 9), (8, 33, 4, 700), (300, 7, 8, 5000), (5, 600, 1, 70000), (2, 3, 5, 0), (0, 3, 4, 40),
          (70, 3, 100, 20), (1, 1500, 1, 1048577 + 64)]


@pytest.mark.parametrize("size", ASSIGN, ids=str)
def test_page_assign(size):
    rows, cols, page, n = size
    for seed in range(3):
        rng, pages, lens, refs = tables(seed, rows, cols, page, n, n // 3)
        parent = [rng.choice([r, r, rng.randrange(rows), -1, rows, 2147483647]) for r in range(rows)]
        add = [rng.choice([0, 1, 1, -3, page, 2147483647, rng.randint(0, cols * page)]) for _ in range(rows)]
        if rows:
            lens[rng.randrange(rows)] = [-5, 2147483647, cols * page + 1][seed]
        want = O.assign(pages.tolist(), lens, refs, parent, add, page)
        pg, rg = pages.cuda(), ints(refs).cuda()
        new = lambda *s: torch.full(s, 77, dtype=I32, device="cuda")
        outs = [new(rows, cols), new(rows), new(n), new(rows), new(rows), new(2)]
        ins = [pg, ints(lens).cuda(), rg, ints(parent).cuda(), ints(add).cuda()]
        E.page_assign(*ins, page, *outs)
        for name, got, w in zip("pages lens refs src dst stats".split(), outs, want):
            w = torch.tensor(w, dtype=torch.int64).reshape(got.shape)
            assert bool((got.cpu().long() == w).all()), (name, seed)
        wide = new(rows, 2 * cols + 1)                                # counts in place, a strided table
        strided = wide[:, 1::2][:, :cols]
        E.page_assign(*ins, page, strided, outs[1], rg, outs[3], outs[4], outs[5])
        assert torch.equal(strided, outs[0]) and torch.equal(rg, outs[2])
        assert bool((wide[:, 0::2] == 77).all())


COMPACT = [(1, 1, 1), (3, 4, 9), (8, 40, 509), (64, 33, 5000), (5, 600, 70001), (2, 3, 0), (0, 3, 40), (1, 3, 1048577 + 64),
           (4, 16, 64), (4, 16, 128)]


@pytest.mark.parametrize("size", COMPACT, ids=str)
def test_page_compact(size):
    rows, cols, n = size
    for seed, share in enumerate((0, 3, 2, 1)):
        rng, pages, _, refs = tables(seed, rows, cols, 1, n, n // share if share else 0)
        for k in range(min(6, rows * cols)):
            pages[rng.randrange(rows), rng.randrange(cols)] = [-1, n, -2147483648, 2147483647, 0, max(0, n - 1)][k]
        for k in range(min(4, n)):
            refs[rng.randrange(n)] = [-3, 5, 2147483647, 0][k]
        capacity = n // 2 + seed * 300
        want = O.compact(pages.tolist(), refs, capacity)
        new = lambda *s: torch.full(s, 77, dtype=I32, device="cuda")
        outs = [new(rows, cols), new(n), new(capacity), new(capacity), new(2)]
        pg, rg = pages.cuda(), ints(refs).cuda()
        E.page_compact(pg, rg, *outs)
        for name, got, w in zip("pages refs src dst stats".split(), outs, want):
            w = torch.tensor(w, dtype=torch.int64).reshape(got.shape)
            assert bool((got.cpu().long() == w).all()), (name, seed)
        E.page_compact(pg, rg, pg, *outs[1:])
        assert torch.equal(pg, outs[0])


@pytest.mark.parametrize("shape,dtype", [((9, 1, 1, 1), torch.float16), ((9, 3, 1, 5), torch.bfloat16), ((40, 16, 2, 64), torch.bfloat16),
                                         ((30, 16, 4, 128), torch.bfloat16), ((12, 17, 3, 33), torch.float32),
                                         ((9, 100, 8, 128), torch.float32), ((50, 1, 1, 2), I32)])
def test_page_copy(shape, dtype):
    n = shape[0]
    rng = random.Random(n)
    ids = rng.sample(range(n), n)
    half = n // 2
    src, dst = ids[:half] + [-1, 3, n, 2147483647], ids[half:2 * half] + [2, -1, 0, 1]
    g = gen(n)
    base = [torch.randint(-9, 9, shape, generator=g).to(dtype), torch.randint(-9, 9, (n, 2) + shape[1:], generator=g).to(dtype),
            torch.randint(-9, 9, shape[:2] + (shape[2], 2) + shape[3:], generator=g).to(dtype),
            torch.randint(-9, 9, (n, shape[2], shape[1], shape[3]), generator=g).to(dtype)]
    gpu = [b.cuda() for b in base]
    view = lambda b: [b[0], b[1][:, 1], b[2][:, :, :, 1], b[3].transpose(1, 2)]
    other = torch.randint(-9, 9, (n, 2, 1, 3), generator=g).to(dtype)       # another pool, other pages
    og = other.cuda()
    E.page_copy(view(gpu) + [og], ints(src).cuda(), ints(dst).cuda())
    pools = view(base) + [other]
    for p in pools:
        old = p.clone()
        for a, b in zip(src, dst):
            if 0 <= a < p.shape[0] and 0 <= b < p.shape[0]:
                p[b] = old[a]
    for got, w in zip(gpu + [og], base + [other]):
        assert torch.equal(got.cpu(), w)


def test_page_copy_many_pools():
    pools = [torch.randn(6, 4, 2, 8, device="cuda") for _ in range(61)]
    want = [p[2].clone() for p in pools]
    E.page_copy(pools, ints([2, -1]).cuda(), ints([5, -1]).cuda())
    assert all(torch.equal(p[5], w) and torch.equal(p[2], w) for p, w in zip(pools, want))
    E.page_copy([], ints([2]).cuda(), ints([5]).cuda())
    E.page_copy(pools[:1], ints([]).cuda(), ints([]).cuda())


# ---------------------------------------------------------------------------
# Streams, graphs, workspaces.

def step_state(seed=11):
    q, k, v, pages, lens = attention_case(seed, torch.bfloat16, 4, 8, 2, 64, 64, 16, [900, 17, 0, 300])
    out = torch.empty(4, 8, 64, dtype=torch.bfloat16, device="cuda")
    return [x.cuda() for x in (q, k, v, pages, lens)], out


def test_streams_and_workspace():
    args, out = step_state()
    E.paged_attention(*args, out)
    need = E.paged_attention_workspace(*args, out)
    assert need > 0
    for how in ("stream", "handle", "own workspace"):
        other = torch.empty_like(out)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        kw = dict(workspace=torch.empty(need, dtype=torch.uint8, device="cuda")) if how == "own workspace" else {}
        E.paged_attention(*args, other, stream=s.cuda_stream if how == "handle" else s, **kw)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(other, out), how
    with pytest.raises(E.Error):
        E.paged_attention(*args, out, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(E.Error):
        E.paged_attention(args[0].cpu(), *args[1:], out)


def test_default_stream_by_its_handle(monkeypatch):
    """stream=0: the scratch memory is of the default stream too, and the results are the same."""
    import types

    from elementwise_tensor_commands_amd import serving as S
    args, out = step_state()
    E.paged_attention(*args, out)
    allocated_on = []

    def scratch(size, device):
        allocated_on.append(torch.cuda.current_stream().cuda_stream)
        return binding.scratch(size, device)

    binding = S._binding
    monkeypatch.setattr(S, "_binding", types.SimpleNamespace(**{**vars(binding), "scratch": scratch}))
    rng, pages, lens, refs = tables(3, 300, 7, 8, 5000, 1000)
    new = lambda *s: torch.full(s, 77, dtype=I32, device="cuda")
    ins = [pages.cuda(), ints(lens).cuda(), ints(refs).cuda(), torch.arange(300, dtype=I32).cuda(), torch.ones(300, dtype=I32).cuda()]
    want, got = ([new(300, 7), new(300), new(5000), new(300), new(300), new(2)] for _ in range(2))
    E.page_assign(*ins, 8, *want)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        other = torch.empty_like(out)
        E.paged_attention(*args, other, stream=0)
        E.page_assign(*ins, 8, *got, stream=0)
    torch.cuda.synchronize()
    assert len(allocated_on) == 3 and allocated_on[1:] == [0, 0]
    assert torch.equal(other, out) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_step():
    """A whole decode step in one graph, replayed with other lengths and inputs."""
    def build():
        g = gen(21)
        rows, cols, page, hq, hk, d, n = 6, 8, 16, 8, 2, 64, 64
        s = dict(pages=torch.full((rows, cols), -1, dtype=I32), lens=ints([0] * rows), refs=ints([0] * n),
                 parent=ints(list(range(rows))), add=ints([40, 17, 1, 0, 90, 16]), pages2=torch.zeros(rows, cols, dtype=I32),
                 lens2=ints([0] * rows), refs2=ints([0] * n), src=ints([0] * rows), dst=ints([0] * rows), stats=ints([0, 0]),
                 row=torch.arange(rows, dtype=I32), q=randn(g, rows, hq, d, dtype=torch.bfloat16),
                 kv=randn(g, rows, 2 * hk, d, dtype=torch.bfloat16), q2=torch.zeros(rows, hq, d, dtype=torch.bfloat16),
                 kc=randn(g, n, page, hk, d, dtype=torch.bfloat16), vc=randn(g, n, page, hk, d, dtype=torch.bfloat16),
                 freq=E.rope_frequencies(d), out=torch.zeros(rows, hq, d, dtype=torch.bfloat16))
        return {k: v.cuda() for k, v in s.items()}

    def step(s):
        E.page_assign(s["pages"], s["lens"], s["refs"], s["parent"], s["add"], 16, s["pages2"], s["lens2"], s["refs2"],
                      s["src"], s["dst"], s["stats"])
        E.page_copy([s["kc"], s["vc"]], s["src"], s["dst"])
        pos = s["lens2"] - 1
        E.rope_append(s["q"], s["kv"][:, :2], s["kv"][:, 2:], pos, s["row"], s["pages2"], s["freq"], s["q2"], s["kc"], s["vc"])
        E.paged_attention(s["q2"], s["kc"], s["vc"], s["pages2"], s["lens2"], s["out"])
        for a, b in (("pages", "pages2"), ("lens", "lens2"), ("refs", "refs2")):
            s[a].copy_(s[b])

    eager, captured = build(), build()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(captured)
    plans = [([0, 1, 2, 3, 4, 5], [40, 17, 1, 0, 90, 16]), ([0, 0, 2, 1, 4, 4], [1] * 6), ([0, 1, 2, 3, 4, 5], [1] * 6),
             ([-1, 1, 0, 3, 4, 5], [7, 1, 1, 0, 1, 1]), ([0, 1, 2, 3, 4, 5], [1] * 6)]
    g = gen(5)
    for i, (parent, add) in enumerate(plans):
        q, kv = randn(g, 6, 8, 64, dtype=torch.bfloat16).cuda(), randn(g, 6, 4, 64, dtype=torch.bfloat16).cuda()
        for s in (eager, captured):
            s["parent"].copy_(ints(parent)), s["add"].copy_(ints(add)), s["q"].copy_(q), s["kv"].copy_(kv)
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for key in eager:
            assert torch.equal(eager[key], captured[key]), (i, key)


@pytest.mark.parametrize("b", [64, 65, 100, 300])
def test_attention_many_rows(b):
    """Row prefixes of one wave, of a work-group, and over several turns; few and many runs to a row."""
    rng = random.Random(b)
    lens = [rng.choice([0, 0, 1, 40, 200, 700]) for _ in range(b)]
    check_attention(*attention_case(b, torch.float16, b, 2, 1, 32, 32, 16, lens), what=b)
    lens = [0] * (b - 1) + [3000]
    check_attention(*attention_case(b, torch.bfloat16, b, 4, 4, 64, 64, 16, lens), what=("last", b))
    assert not bool(check_attention(*attention_case(b, torch.float32, b, 2, 2, 32, 32, 16, [0] * b, cols=20)).any())


def test_attention_more_rows_than_prefixes():
    b = 2100
    lens = [(i * 37) % 90 for i in range(b)]
    check_attention(*attention_case(1, torch.bfloat16, b, 2, 1, 32, 32, 16, lens), what=b)


@pytest.mark.parametrize("entries", [3200, 3201])
def test_pages_at_the_limit_of_one_launch(entries):
    """The largest tables of one launch and the smallest of two, with the most pages of one."""
    for rows, cols, n in ((64, 50, 4096), (1, 3200, 4095), (800, 4, 4096)) if entries == 3200 else (
            (33, 97, 4096), (1, 3201, 4095), (1067, 3, 4096)):
        rng, pages, lens, refs = tables(entries + rows, rows, cols, 4, n, n // 3)
        parent = [rng.choice([r, rng.randrange(rows), -1]) for r in range(rows)]
        add = [rng.choice([0, 1, 5, cols * 4]) for _ in range(rows)]
        want = O.assign(pages.tolist(), lens, refs, parent, add, 4)
        new = lambda *s: torch.full(s, 77, dtype=I32, device="cuda")
        outs = [new(rows, cols), new(rows), new(n), new(rows), new(rows), new(2)]
        ins = [pages.cuda(), ints(lens).cuda(), ints(refs).cuda(), ints(parent).cuda(), ints(add).cuda()]
        assert (E.page_assign_workspace(*ins, 4, *outs) == 0) == (rows * cols <= 3200)
        E.page_assign(*ins, 4, *outs)
        for got, w in zip(outs, want):
            assert got.cpu().tolist() == w
        want = O.compact(pages.tolist(), refs, n // 2)
        outs = [new(rows, cols), new(n), new(n // 2), new(n // 2), new(2)]
        assert (E.page_compact_workspace(ins[0], ins[2], *outs) == 0) == (rows * cols <= 3200)
        E.page_compact(ins[0], ins[2], *outs)
        for got, w in zip(outs, want):
            assert got.cpu().tolist() == w
