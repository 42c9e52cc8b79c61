"""The operators on trees of drafted tokens and on pages worth reading or keeping, on
the GPU against their definitions in 64 bits (cache_oracle.py), within bounds counted
from the roundings that include/ecmd_serving.h lists; whole numbers are equal."""
import math
import random

import pytest
import torch

import cache_oracle as C
import elementwise_tensor_commands_amd as E
import serving_oracle as O
from test_gpu_serving import DT, I32, gen, ints, randn, within

pytestmark = pytest.mark.gpu


def cache(g, n, page, heads, d, dtype, extra=0):
    """[n, page, heads, d] with `extra` elements after every slot, on the GPU and the CPU."""
    x = randn(g, n, page, heads, d, dtype=dtype)
    base = torch.full((n, page, heads * d + extra), math.nan, dtype=dtype, device="cuda")
    view = base[..., :heads * d].unflatten(2, (heads, d))
    view.copy_(x)
    return view, x


def table(rng, n, rows, cols, holes=0.1):
    """Pages of rows: no page twice while there are enough, some holes of either kind."""
    ids = [i % n for i in range(rows * cols)]
    rng.shuffle(ids)
    return ints([[rng.choice([-1, n, -7, 2 ** 31 - 1]) if rng.random() < holes else ids[r * cols + c] for c in range(cols)]
                 for r in range(rows)])


def parents(rng, t, bad=0.1):
    out = []
    for i in range(t):
        kind = rng.random()
        out.append(rng.choice([-2, i, i + 3, -2 ** 31, 2 ** 31 - 1]) if kind < bad else
                   -1 if i == 0 or kind < bad + 0.1 else i - 1 if kind < 0.6 else rng.randrange(i))
    return out


# ---------------------------------------------------------------------------
# Attention for trees.

TREES = [  # b, t, hq, hk, d, dv, page, cols, window
    (1, 1, 1, 1, 8, 8, 4, 1, 0), (1, 1, 4, 2, 64, 64, 16, 5, 0), (2, 8, 8, 2, 128, 128, 16, 9, 0), (3, 5, 6, 6, 80, 64, 17, 7, 30),
    (2, 16, 4, 4, 64, 64, 8, 20, 0), (2, 17, 4, 4, 64, 64, 8, 20, 9), (1, 33, 8, 2, 96, 128, 32, 4, 0), (4, 3, 5, 1, 33, 40, 3, 30, 0),
    (1, 64, 16, 2, 128, 128, 16, 20, 40), (1, 65, 3, 1, 128, 96, 16, 14, 3), (1, 200, 2, 1, 64, 128, 100, 4, 0), (1, 256, 1, 1, 128, 64, 16, 40, 0),
    (5, 7, 16, 1, 192, 128, 16, 8, 0), (2, 9, 6, 2, 256, 256, 16, 6, 0), (2, 30, 34, 2, 200, 136, 5, 20, 33), (3, 4, 2, 2, 1, 1, 4, 6, 0),
    (2, 20, 4, 2, 3, 70, 4, 30, 0), (2, 20, 4, 2, 70, 2, 1, 90, 0), (6, 12, 8, 4, 128, 128, 64, 24, 0), (3, 2, 40, 2, 128, 128, 16, 100, 0),
]


def tree_state(case, dtype, seed, reach=1.0):
    b, t, hq, hk, d, dv, page, cols, window = case
    g, rng = gen(seed), random.Random(seed)
    n = b * cols + 1
    kg, kc = cache(g, n, page, hk, d, DT[dtype], extra=(0, 8, 5)[seed % 3])
    vg, vc = cache(g, n, page, hk, dv, DT[dtype], extra=(0, 16)[seed % 2])
    q = randn(g, b, t, hq, d, dtype=DT[dtype])
    pages = table(rng, n, b, cols)
    lens = [rng.choice([int(cols * page * reach) - t, rng.randint(0, cols * page)]) for _ in range(b)]
    lens = ints([max(0, x) for x in lens])
    for i, special in enumerate([0, -3, cols * page + 5]):
        if b > i + 1:
            lens[i + 1] = special
    parent = ints([parents(rng, t) for _ in range(b)])
    return q, (kg, vg), (kc, vc), pages, lens, parent, window


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree_attention(case, dtype):
    q, (kg, vg), (kc, vc), pages, lens, parent, window = tree_state(TREES[case], dtype, case)
    b, t, hq, d = q.shape
    dv = vc.shape[3]
    scale = [1.0 / math.sqrt(d), -0.2, 0.7 / math.sqrt(d)][case % 3]
    want, want_lse, eo, el = C.tree(q, kc, vc, pages, lens, parent, scale, window)
    base = torch.full((t, b, hq, dv + 3), 7.0, dtype=DT[dtype], device="cuda")
    out = base.transpose(0, 1)[..., 1:dv + 1]
    lse = torch.full((b, hq, t), 7.0, device="cuda").transpose(1, 2)
    packed = torch.empty(b, t, hq + 2, d, dtype=DT[dtype], device="cuda")
    packed[:, :, 1:-1] = q.cuda()
    E.tree_attention(packed[:, :, 1:-1], kg, vg, pages.cuda(), lens.cuda(), parent.cuda(), out, lse=lse, scale=scale, window=window)
    within(out, want, eo, TREES[case])
    within(lse, want_lse, el, TREES[case])
    assert bool((base[..., 0] == 7).all() and (base[..., dv + 1:] == 7).all())
    again = torch.empty(b, t, hq, dv, dtype=DT[dtype], device="cuda")
    E.tree_attention(packed[:, :, 1:-1], kg, vg, pages.cuda(), lens.cuda(), parent.cuda(), again, scale=scale, window=window)
    assert torch.equal(again, out)


MANY = [  # of many query vectors, rows of the caches at multiples of 16 bytes
    (2, 12, 8, 2, 64, 64, 16, 20, 0), (1, 40, 8, 2, 56, 48, 16, 30, 70), (2, 20, 2, 1, 96, 128, 16, 30, 0), (1, 100, 2, 1, 72, 104, 8, 60, 0),
    (2, 11, 4, 1, 128, 128, 16, 40, 0), (3, 33, 8, 2, 128, 64, 16, 25, 100), (1, 256, 4, 2, 120, 128, 64, 16, 0), (2, 50, 1, 1, 192, 128, 16, 20, 0),
    (1, 20, 6, 2, 160, 96, 32, 12, 0), (2, 18, 2, 1, 192, 192, 16, 18, 40), (1, 34, 4, 4, 256, 256, 16, 18, 0), (1, 40, 1, 1, 8, 8, 16, 30, 0),
    (1, 70, 2, 2, 200, 136, 5, 60, 0), (9, 10, 16, 4, 128, 128, 16, 8, 0),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_tree_attention_of_many_query_vectors(case, dtype):
    q, (kg, vg), (kc, vc), pages, lens, parent, window = tree_state(MANY[case], dtype, 6 * case + 100)
    want, want_lse, eo, el = C.tree(q, kc, vc, pages, lens, parent, 1.0 / math.sqrt(q.shape[3]), window)
    out, lse = torch.full(want.shape, 7.0, dtype=DT[dtype], device="cuda"), torch.full(want_lse.shape, 7.0, device="cuda")
    E.tree_attention(q.cuda(), kg, vg, pages.cuda(), lens.cuda(), parent.cuda(), out, lse=lse, window=window)
    within(out, want, eo, MANY[case])
    within(lse, want_lse, el, MANY[case])


@pytest.mark.parametrize("dtype", list(DT))
def test_tree_attention_of_a_long_context(dtype):
    """Rows cut into segments, whole rows, many query vectors: the second launch."""
    for seed, case in enumerate([(1, 9, 4, 1, 64, 64, 16, 700, 0), (3, 40, 8, 1, 64, 64, 16, 300, 0), (2, 11, 2, 2, 128, 128, 64, 60, 2000),
                                 (40, 6, 8, 4, 32, 32, 16, 60, 0)]):
        q, (kg, vg), (kc, vc), pages, lens, parent, window = tree_state(case, dtype, seed + 50)
        want, want_lse, eo, el = C.tree(q, kc, vc, pages, lens, parent, 1.0 / math.sqrt(q.shape[3]), window)
        out, lse = torch.empty(want.shape, dtype=DT[dtype], device="cuda"), torch.empty(want_lse.shape, device="cuda")
        args = [q.cuda(), kg, vg, pages.cuda(), lens.cuda(), parent.cuda(), out]
        size = E.tree_attention_workspace(*args, window=window)
        assert size > 0
        work = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        E.tree_attention(*args, lse=lse, window=window, workspace=work)
        within(out, want, eo, case)
        within(lse, want_lse, el, case)


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("dtype", list(DT))
def test_tree_attention_leaves_out_what_it_does_not_attend_to(dtype, hq):
    """Infinities and NaN in slots that some tokens see and others do not."""
    dt = DT[dtype]
    g = gen(5)
    b, t, hk, d, page, cols = 1, 6, 2, 64, 8, 6
    q, k, v = randn(g, b, t, hq, d, dtype=dt), randn(g, cols, page, hk, d, dtype=dt), randn(g, cols, page, hk, d, dtype=dt)
    parent, length = [[-1, 0, 0, 1, -2, 2]], 21          # token 4 is padding
    slot = lambda i: divmod(length + i, page)
    pages = ints([list(range(cols))])
    k[slot(4)], v[slot(4)] = math.nan, math.nan                       # padding's slot: of no account to anybody
    k[slot(6)], v[slot(6)] = math.nan, math.nan                       # past the tree
    for i, column, value in ((1, 3, math.inf), (2, 5, -math.inf), (3, 7, math.nan)):
        v[slot(i)][:, column] = value
    want, want_lse, eo, el = C.tree(q, k, torch.nan_to_num(v, 0.0, 0.0, 0.0), pages, ints([length]), ints(parent), 0.125)
    out, lse = torch.empty(b, t, hq, d, dtype=dt, device="cuda"), torch.empty(b, t, hq, device="cuda")
    E.tree_attention(q.cuda(), k.cuda(), v.cuda(), pages.cuda(), ints([length]).cuda(), ints(parent).cuda(), out, lse=lse)
    got = out.cpu()
    sees = {0: [], 1: [(3, math.inf)], 2: [(5, -math.inf)], 3: [(3, math.inf), (7, math.nan)], 4: [], 5: [(5, -math.inf)]}
    for i, marks in sees.items():
        for column, value in marks:
            x = got[0, i, :, column].double()
            assert bool(x.isnan().all() if math.isnan(value) else (x == value).all()), (i, column, x)
            want[0, i, :, column], eo[0, i, :, column] = 0.0, math.inf
            got[0, i, :, column] = 0.0
    within(got, want, eo)
    within(lse, want_lse, el)
    # a NaN key is its own followers' matter only
    k2 = k.clone()
    k2[slot(1)] = math.nan
    E.tree_attention(q.cuda(), k2.cuda(), torch.nan_to_num(v, 0.0, 0.0, 0.0).cuda(), pages.cuda(), ints([length]).cuda(), ints(parent).cuda(), out, lse=lse)
    bad = out.isnan().flatten(2).all(-1)[0].tolist()
    assert bad == [i in (1, 3) for i in range(t)] and lse.isnan().all(-1)[0].tolist() == bad


def test_a_chain_is_attention_of_one_token_after_the_other():
    """A tree that is a chain against cmd_paged_attention of each of its tokens."""
    g = gen(8)
    b, t, hq, hk, d, page, cols = 2, 20, 8, 2, 128, 16, 12
    q = randn(g, b, t, hq, d, dtype=torch.float32).cuda()
    k, v = (randn(g, b * cols, page, hk, d, dtype=torch.float32).cuda() for _ in range(2))
    pages = ints([list(range(r * cols, (r + 1) * cols)) for r in range(b)]).cuda()
    lens = ints([100, 37])
    parent = ints([[i - 1 for i in range(t)]] * b).cuda()
    out, one = torch.empty(b, t, hq, d, device="cuda"), torch.empty(b, hq, d, device="cuda")
    for window in (0, 25):
        E.tree_attention(q, k, v, pages, lens.cuda(), parent, out, window=window)
        for i in range(t):
            E.paged_attention(q[:, i], k, v, pages, (lens + i + 1).cuda(), one, window=window)
            # each is within this of the exact result: scores of a few units, 120 keys
            assert float((out[:, i] - one).abs().max()) < 2 * 4.0 * (2 * 30 * 130 * 2 * C.U + 400 * C.U)


def test_tree_attention_without_anything():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=I32, device="cuda")
    out = torch.full((2, 3, 4, 8), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 3, 4), 5.0, device="cuda")
    for n, page, cols in ((0, 4, 3), (3, 0, 3), (3, 4, 0)):                     # no pages, no slots, no columns
        out.fill_(5)
        E.tree_attention(z(2, 3, 4, 8), z(n, page, 2, 8), z(n, page, 2, 8), i(2, cols), i(2) + 9, i(2, 3) - 1, out, lse=lse)
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    E.tree_attention(z(0, 3, 4, 8), z(3, 4, 2, 8), z(3, 4, 2, 8), i(0, 3), i(0), i(0, 3), z(0, 3, 4, 8))
    E.tree_attention(z(2, 0, 4, 8), z(3, 4, 2, 8), z(3, 4, 2, 8), i(2, 3), i(2), i(2, 0), z(2, 0, 4, 8))


# ---------------------------------------------------------------------------
# The accepted path and the move of its slots.

def test_tree_accept():
    rng = random.Random(2)
    for rows, t, words in [(1, 1, 2), (3, 5, 2), (40, 64, 2), (7, 65, 3), (9, 256, 2), (5, 200, 1), (1, 0, 2), (0, 4, 2)]:
        tokens, follow = (torch.tensor([[rng.randrange(words) for _ in range(t)] for _ in range(rows)], dtype=I32).view(rows, t) for _ in range(2))
        parent = torch.tensor([parents(rng, t, 0.05) for _ in range(rows)], dtype=I32).view(rows, t)
        if t:
            parent[:, 0] = torch.tensor([-1 if rng.random() < 0.8 else rng.choice([0, -2, 5]) for _ in range(rows)], dtype=I32)
        lens = torch.tensor([rng.choice([0, 17, -1, 2 ** 31 - 2, 1000]) for _ in range(rows)], dtype=I32)
        want = C.accept(tokens, parent, follow, lens)
        path = torch.full((t, rows), 99, dtype=I32, device="cuda").t()
        lens_out, last = torch.full((rows,), 99, dtype=I32, device="cuda"), torch.full((rows,), 99, dtype=I32, device="cuda")
        E.tree_accept(tokens.cuda(), parent.cuda(), follow.cuda(), lens.cuda(), path, lens_out, last)
        assert path.tolist() == want[0] and lens_out.tolist() == want[1] and last.tolist() == want[2], (rows, t)
        same = lens.cuda()
        E.tree_accept(tokens.cuda(), parent.cuda(), follow.cuda(), same, path, same, last)
        assert same.tolist() == want[1]


@pytest.mark.parametrize("dtype", ["bf16", "f32", "i32"])
def test_slot_move(dtype):
    dt = {**DT, "i32": I32}[dtype]
    rng = random.Random(4)
    for case, (rows, t, page, cols, heads, d, npools) in enumerate([(1, 5, 4, 6, 2, 8, 1), (3, 20, 16, 5, 2, 64, 2), (2, 256, 7, 60, 1, 3, 5),
                                                                    (5, 40, 5, 20, 3, 40, 30), (2, 9, 16, 4, 8, 128, 2), (1, 3, 2, 4, 5, 1, 1)]):
        g = gen(case)
        n = rows * cols + 2
        pools = []
        for i in range(npools):
            shape = (n, page, heads, d) if i % 3 != 1 else (n, page, 1, 2 * d)
            pools.append(torch.randint(-1000, 1000, shape, generator=g).to(dt))
        pages = table(rng, n, rows, cols, holes=0.1 if case % 2 else 0.0)
        lens = [rng.randint(0, cols * page - 1) for _ in range(rows)]
        path = []
        for r in range(rows):
            p = sorted(rng.sample(range(t), rng.randint(0, t)))
            if p and rng.random() < 0.5:
                p[0] = 0
            path.append(p + [-1] * (t - len(p)))
        if rows > 2:
            lens[1], lens[2] = -4, 2 ** 31 - 1
        lens, path = ints(lens), torch.tensor(path, dtype=I32).view(rows, t)
        want = C.move(pools, pages, lens, path)
        got = []
        for i, p in enumerate(pools):
            if i % 2:                                               # slots apart, off 16 bytes
                base = torch.zeros(n, page, p.shape[2] * p.shape[3] + 1, dtype=dt, device="cuda")
                view = base[..., 1:].unflatten(2, p.shape[2:])
            else:                                                   # heads before slots
                view = torch.zeros(n, p.shape[2], page, p.shape[3], dtype=dt, device="cuda").transpose(1, 2)
            view.copy_(p)
            got.append(view)
        E.slot_move(got, pages.cuda(), lens.cuda(), path.cuda())
        for a, b in zip(got, want):
            assert torch.equal(a.cpu(), b), case
    E.slot_move([], pages.cuda(), lens.cuda(), path.cuda())
    E.slot_move([torch.zeros(0, page, 2, 2, device="cuda")], pages.cuda(), lens.cuda(), path.cuda())


# ---------------------------------------------------------------------------
# Bounds, selection, attention over tables of heads.

@pytest.mark.parametrize("dtype", list(DT))
def test_page_bounds(dtype):
    dt = DT[dtype]
    for case, (rows, cols, page, hk, d) in enumerate([(1, 3, 4, 1, 8), (3, 6, 16, 2, 128), (2, 40, 1, 3, 7), (4, 5, 33, 8, 80), (1, 2, 300, 40, 64),
                                                      (2, 3, 5, 2, 1), (3, 9, 16, 4, 200), (1, 4, 8, 2, 3)]):
        g, rng = gen(case), random.Random(case)
        n = rows * cols + 1
        kg, kc = cache(g, n, page, hk, d, dt, extra=case % 3)
        kc[torch.rand(kc.shape, generator=g) < 0.02] = math.nan
        kc[torch.rand(kc.shape, generator=g) < 0.01] = math.inf
        kg.copy_(kc)
        pages = table(rng, n, rows, cols)
        lens = ints([rng.choice([cols * page, cols * page + 9, rng.randint(0, cols * page), -2]) for _ in range(rows)])
        since = ints([rng.choice([0, -5, max(0, int(x) - 1), rng.randint(0, cols * page)]) for x in lens])
        old = torch.sort(randn(g, n, hk, 2, d, dtype=dt), dim=2).values
        bg = torch.full((n, hk, 2, d + 1), 3.0, dtype=dt, device="cuda")
        bg[..., :d] = old.cuda()
        E.page_bounds(kg, pages.cuda(), lens.cuda(), since.cuda(), bg[..., :d])
        assert torch.equal(bg[..., :d].cpu(), C.bounds(kc, pages, lens, since, old)), case
        assert bool((bg[..., d] == 3).all())


SELECTS = [  # b, hq, hk, d, page, cols, take, first, last
    (1, 1, 1, 8, 4, 6, 3, 1, 1), (2, 8, 2, 128, 16, 40, 10, 1, 2), (3, 6, 6, 80, 17, 30, 5, 0, 0), (2, 16, 1, 64, 8, 300, 64, 2, 3),
    (1, 9, 3, 33, 16, 700, 100, 1, 2), (1, 20, 1, 192, 1, 1000, 17, 0, 1), (2, 4, 2, 256, 16, 20, 30, 1, 2), (1, 3, 1, 1, 16, 50, 9, 9, 0),
    (130, 4, 2, 64, 16, 24, 8, 1, 2), (1, 2, 1, 16, 1, 5000, 1200, 0, 5), (2, 4, 4, 5, 3, 9, 1, 0, 0),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", range(len(SELECTS)))
def test_page_select(case, dtype):
    b, hq, hk, d, page, cols, take, first, last = SELECTS[case]
    dt = DT[dtype]
    g, rng = gen(case), random.Random(case)
    n = b * cols // 2 + 1                                              # pages in several places: ties
    bounds = torch.sort(randn(g, n, hk, 2, d, dtype=dt), dim=2).values
    if case % 2:
        bounds[torch.rand(n, generator=g) < 0.05] = math.nan
        bounds[torch.rand(n, generator=g) < 0.05] = math.inf
    q = randn(g, b, hq, d, dtype=dt)
    pages = table(rng, n, b, cols, holes=0.2)
    lens = [cols * page + 3, 0, -1, page] if b > 3 else [cols * page - 1]
    lens = ints(lens + [rng.randint(0, cols * page) for _ in range(b - len(lens))])
    want, want_lens = C.select(q, bounds, pages, lens, page, take, first, last)
    base = torch.full((take, b, hk), 77, dtype=I32, device="cuda")
    out, out_lens = base.permute(1, 2, 0), torch.full((b, hk), 77, dtype=I32, device="cuda")
    args = [q.cuda(), bounds.cuda(), pages.cuda(), lens.cuda(), page, out, out_lens]
    size = E.page_select_workspace(*args, first=first, last=last)
    work = torch.full((max(16, size),), 255, dtype=torch.uint8, device="cuda")
    E.page_select(*args, first=first, last=last, workspace=work)
    assert torch.equal(out.cpu(), want) and torch.equal(out_lens.cpu(), want_lens)


@pytest.mark.parametrize("dtype", list(DT))
def test_attention_over_tables_of_heads(dtype):
    dt = DT[dtype]
    for case, (b, hq, hk, d, dv, page, cols, window) in enumerate([(1, 4, 2, 64, 64, 16, 5, 0), (3, 6, 3, 80, 64, 17, 20, 50), (2, 40, 2, 128, 128, 16, 90, 0),
                                                                   (70, 8, 4, 64, 64, 8, 9, 0), (1, 8, 8, 192, 128, 16, 160, 0), (9, 5, 5, 40, 33, 5, 300, 0)]):
        g, rng = gen(case), random.Random(case)
        n = 50
        kg, kc = cache(g, n, page, hk, d, dt, extra=case)
        vg, vc = cache(g, n, page, hk, dv, dt)
        q = randn(g, b, hq, d, dtype=dt)
        pages = table(rng, n, b * hk, cols).view(b, hk, cols)
        lens = ints([rng.choice([0, -1, cols * page + 2, rng.randint(1, cols * page), cols * page]) for _ in range(b * hk)]).view(b, hk)
        group, scale = hq // hk, 1.0 / math.sqrt(d)
        out, lse = torch.full((b, hq, dv), 7.0, dtype=dt, device="cuda"), torch.full((hq, b), 7.0, device="cuda").t()
        E.paged_attention(q.cuda(), kg, vg, pages.cuda(), lens.cuda(), out, lse=lse, window=window)
        for h in range(hk):
            heads = slice(h * group, (h + 1) * group)
            want, want_lse, eo, el = O.attention(q[:, heads], kc[:, :, h:h + 1], vc[:, :, h:h + 1], pages[:, h], lens[:, h], scale, window)
            within(out[:, heads], want, eo, (case, h))
            within(lse[:, heads], want_lse, el, (case, h))


# ---------------------------------------------------------------------------
# Mass and eviction.

MASSES = [  # b, hq, hk, d, page, cols, window
    (1, 1, 1, 8, 4, 1, 0), (2, 8, 2, 128, 16, 20, 0), (3, 12, 12, 80, 17, 9, 60), (1, 4, 1, 64, 300, 3, 0), (2, 20, 1, 96, 1, 400, 100),
    (2, 6, 3, 192, 100, 4, 0), (1, 40, 2, 256, 32, 10, 0), (4, 3, 3, 2, 16, 5, 0), (2, 10, 5, 33, 257, 2, 0), (3, 4, 4, 128, 64, 6, 1),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", range(len(MASSES)))
def test_page_mass(case, dtype):
    b, hq, hk, d, page, cols, window = MASSES[case]
    dt = DT[dtype]
    g, rng = gen(case), random.Random(case)
    n = b * cols + 1
    kg, kc = cache(g, n, page, hk, d, dt, extra=case % 3)
    q = randn(g, b, hq, d, dtype=dt)
    pages = table(rng, n, b, cols)
    lens = ints([cols * page - case % 2] + [rng.choice([0, -2, cols * page + 4, rng.randint(1, cols * page)]) for _ in range(b - 1)])
    scale = [1.0 / math.sqrt(d), -0.15][case % 2]
    _, lse, _, _ = O.attention(q, kc, kc, pages, lens.clamp(min=0), scale, window)
    lse = lse.float()
    lse[0, 0] = -math.inf                                              # such a head adds nothing
    for r in range(b):                                                 # unused slots may hold anything
        x = int(lens[r])
        if 0 < x < cols * page and x % page and 0 <= int(pages[r, x // page]) < n:
            kg[int(pages[r, x // page]), x % page:] = math.nan
    was = torch.rand(b, cols, generator=g)
    want, bound = C.mass(q, kc, pages, lens, lse, was, scale, 0.75, window)
    mg = was.cuda()
    out = torch.full((cols, b), 7.0, device="cuda").t()
    E.page_mass(q.cuda(), kg, pages.cuda(), lens.cuda(), lse.cuda(), mg, out, scale=scale, decay=0.75, window=window)
    within(out, want, bound, MASSES[case])
    E.page_mass(q.cuda(), kg, pages.cuda(), lens.cuda(), lse.cuda(), mg, mg, scale=scale, decay=0.75, window=window)
    assert torch.equal(mg, out)


@pytest.mark.parametrize("rows,cols,n,first,last", [(1, 1, 4, 0, 0), (3, 20, 80, 1, 2), (5, 300, 900, 0, 0), (2, 5000, 4000, 2, 3), (40, 64, 700, 1, 1),
                                                    (0, 5, 9, 0, 0), (3, 0, 9, 0, 0), (2, 7, 0, 0, 0), (4, 30, 60, 20, 20)])
def test_page_evict(rows, cols, n, first, last):
    g, rng = gen(rows * cols), random.Random(rows + cols)
    page = 4
    pages = table(rng, max(n, 1), rows, cols, holes=0.1).view(rows, cols)
    lens = torch.tensor([rng.choice([cols * page, rng.randint(0, cols * page), cols * page + 7, -1]) for _ in range(rows)], dtype=I32)
    mass = torch.rand(rows, cols, generator=g)
    mass = torch.where(mass < 0.3, (mass * 10).floor() / 10, mass)       # ties
    for value in (0.0, -0.0, -1.0, math.inf, -math.inf, math.nan):
        mass[torch.rand(mass.shape, generator=g) < 0.03] = value
    refs = torch.tensor([rng.randint(3, 90) for _ in range(n)], dtype=I32)
    budget = torch.tensor([rng.choice([0, -3, cols, rng.randint(0, max(1, cols))]) for _ in range(rows)], dtype=I32)
    want = C.evict(pages, lens, refs, mass, budget, page, first, last)
    out, refs_out, count = (torch.full(s, 77, dtype=I32, device="cuda") for s in ((cols, rows), (n,), (rows,)))
    E.page_evict(pages.cuda(), lens.cuda(), refs.cuda(), mass.cuda(), budget.cuda(), page, out.t(), refs_out, count, first=first, last=last)
    assert out.t().tolist() == want[0] and refs_out.tolist() == want[1] and count.tolist() == want[2]
    pg, rg = pages.cuda(), refs.cuda()
    E.page_evict(pg, lens.cuda(), rg, mass.cuda(), budget.cuda(), page, pg, rg, count, first=first, last=last)
    assert pg.tolist() == want[0] and rg.tolist() == want[1] and count.tolist() == want[2]
