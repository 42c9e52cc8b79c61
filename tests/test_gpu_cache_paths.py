"""The operators on trees and pages where the library takes another way than on the
sizes of test_gpu_cache_ops.py: tables whose keys no work-group holds, caches past
32-bit offsets; and how they are called: streams, workspaces, graphs, two at once."""
import math
import random

import pytest
import torch

import cache_oracle as C
import elementwise_tensor_commands_amd as E
from test_gpu_cache_ops import parents, table, tree_state
from test_gpu_serving import DT, I32, gen, ints, randn, within

pytestmark = pytest.mark.gpu


def new(*shape, dtype=I32, fill=77):
    return torch.full(shape, fill, dtype=dtype, device="cuda")


# ---------------------------------------------------------------------------
# Long tables: up to 1024 and 8192 columns stay in a work-group's registers.

@pytest.mark.parametrize("cols,take", [(1024, 100), (1025, 100), (8192, 3000), (8193, 8000), (20000, 77), (9000, 9000)])
def test_page_select_of_long_tables(cols, take):
    g, rng = gen(cols), random.Random(cols)
    n, hq, hk, d = 600, 4, 2, 8                                        # every page in many places: ties
    bounds = torch.sort(randn(g, n, hk, 2, d, dtype=torch.float16), dim=2).values
    q = randn(g, 2, hq, d, dtype=torch.float16)
    pages = torch.tensor([[rng.randrange(n) if rng.random() < 0.9 else -1 for _ in range(cols)] for _ in range(2)], dtype=I32)
    lens = ints([cols * 4 - 1, rng.randint(0, cols * 4)])
    want, want_lens = C.select(q, bounds, pages, lens, 4, take, 1, 2)
    out, out_lens = new(2, hk, take), new(2, hk)
    E.page_select(q.cuda(), bounds.cuda(), pages.cuda(), lens.cuda(), 4, out, out_lens)
    assert torch.equal(out.cpu(), want) and torch.equal(out_lens.cpu(), want_lens)


@pytest.mark.parametrize("cols", [5, 300, 1500, 9000])
def test_page_select_of_equal_scores(cols):
    """One page in every column, and pages that differ in the last bit alone: the lower columns win."""
    for step in (0.0, 2.0 ** -10):
        bounds = torch.ones(2, 1, 2, 4, dtype=torch.float16)
        bounds[1] += step
        pages = torch.zeros(1, cols, dtype=I32)
        pages[0, cols // 2:] = 1
        take = max(3, cols // 3)
        q, lens = torch.ones(1, 1, 4, dtype=torch.float16), ints([cols])
        want, want_lens = C.select(q, bounds, pages, lens, 1, take, 1, 1)
        out, out_lens = new(1, 1, take), new(1, 1)
        E.page_select(q.cuda(), bounds.cuda(), pages.cuda(), lens.cuda(), 1, out, out_lens, first=1, last=1)
        assert torch.equal(out.cpu(), want) and torch.equal(out_lens.cpu(), want_lens)


@pytest.mark.parametrize("cols", [1024, 1025, 8192, 8193, 20000])
def test_page_evict_of_long_tables(cols):
    g, rng = gen(cols), random.Random(cols)
    n, rows, page = 500, 3, 2
    pages = table(rng, n, rows, cols, holes=0.1)
    lens = ints([cols * page, rng.randint(0, cols * page), cols])
    mass = torch.rand(rows, cols, generator=g)
    mass = torch.where(mass < 0.5, (mass * 20).floor() / 20, mass)
    refs = torch.full((n,), 1000, dtype=I32)
    budget = ints([cols // 2, cols // 7, 3])
    want = C.evict(pages, lens, refs, mass, budget, page, 1, 2)
    out, refs_out, count = new(rows, cols), new(n), new(rows)
    E.page_evict(pages.cuda(), lens.cuda(), refs.cuda(), mass.cuda(), budget.cuda(), page, out, refs_out, count, first=1, last=2)
    assert out.tolist() == want[0] and refs_out.tolist() == want[1] and count.tolist() == want[2]


# ---------------------------------------------------------------------------
# Up to 64 query vectors under wide tables: the library goes by the tables' size, so the same rows
# with columns of holes behind them take the kernel that stages tiles.

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", [
    (2, 20, 2, 1, 96, 128, 16, 30, 0), (2, 11, 4, 1, 128, 128, 16, 40, 0), (2, 50, 1, 1, 192, 128, 16, 20, 0), (1, 20, 6, 2, 160, 96, 32, 12, 0),
    (2, 18, 2, 1, 192, 192, 16, 18, 40), (1, 34, 4, 4, 256, 256, 16, 18, 0), (1, 40, 1, 1, 8, 8, 16, 30, 0), (9, 10, 16, 4, 128, 128, 16, 8, 0),
    (3, 17, 2, 2, 64, 64, 16, 30, 0), (2, 8, 8, 2, 128, 128, 16, 33, 50), (4, 32, 1, 1, 48, 64, 5, 70, 0), (2, 9, 7, 1, 72, 40, 17, 20, 9),
])
def test_tree_attention_under_wide_tables(case, dtype):
    q, (kg, vg), (kc, vc), pages, lens, parent, window = tree_state(case, dtype, 6 * sum(case))     # slots at multiples of 16 bytes
    b, t, hq, hk, d, dv, page, cols, _ = case
    assert 16 < t * hq // hk <= 64
    wide = torch.cat([pages, torch.full((b, 257 * 128 // page + 1), -1, dtype=I32)], 1)
    want, want_lse, eo, el = C.tree(q, kc, vc, pages, lens, parent, 1.0 / math.sqrt(d), window)
    out, lse = new(*want.shape, dtype=q.dtype), new(*want_lse.shape, dtype=torch.float32)
    E.tree_attention(q.cuda(), kg, vg, wide.cuda(), lens.cuda(), parent.cuda(), out, lse=lse, window=window)
    # a length past the shorter table: its window ends elsewhere
    same = [r for r in range(b) if int(lens[r]) <= cols * page]
    within(out[same], want[same], eo[same], case)
    within(lse[same], want_lse[same], el[same], case)


# Widths between those of test_gpu_cache_ops.py: an instance to each range of them.

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", [
    (2, 6, 2, 1, 192, 192, 16, 9, 0), (1, 9, 3, 3, 150, 160, 8, 12, 20), (2, 5, 2, 2, 80, 48, 16, 8, 0), (1, 7, 4, 4, 72, 60, 7, 20, 0),
    (2, 4, 4, 1, 88, 100, 16, 9, 0), (1, 11, 2, 1, 192, 64, 16, 10, 0), (1, 3, 2, 2, 137, 128, 16, 10, 9), (1, 6, 2, 1, 130, 200, 16, 7, 0),
    (1, 5, 2, 2, 100, 193, 16, 7, 0), (2, 3, 3, 1, 80, 80, 16, 9, 0),
])
def test_tree_attention_of_other_widths(case, dtype):
    q, (kg, vg), (kc, vc), pages, lens, parent, window = tree_state(case, dtype, sum(case))
    want, want_lse, eo, el = C.tree(q, kc, vc, pages, lens, parent, 1.0 / math.sqrt(q.shape[3]), window)
    out, lse = new(*want.shape, dtype=q.dtype), new(*want_lse.shape, dtype=torch.float32)
    E.tree_attention(q.cuda(), kg, vg, pages.cuda(), lens.cuda(), parent.cuda(), out, lse=lse, window=window)
    within(out, want, eo, case)
    within(lse, want_lse, el, case)


@pytest.mark.parametrize("dtype", list(DT))
def test_page_select_of_other_widths(dtype):
    for d, hq in ((3, 1), (4, 4), (7, 2), (48, 2), (64, 3), (80, 4), (96, 2), (97, 6), (128, 1), (150, 4), (192, 8), (200, 2), (256, 3)):
        g, rng = gen(d), random.Random(d)
        bounds = torch.sort(randn(g, 60, 1, 2, d, dtype=DT[dtype]), dim=2).values
        bounds[5], bounds[6, :, 1] = math.nan, math.inf
        q = randn(g, 2, hq, d, dtype=DT[dtype])
        q[0, 0, 0] = 0.0                                               # 0 times infinity
        pages, lens = table(rng, 60, 2, 50), ints([200, 151])
        want, want_lens = C.select(q, bounds, pages, lens, 4, 9, 1, 2)
        out, out_lens = new(2, 1, 9), new(2, 1)
        E.page_select(q.cuda(), bounds.cuda(), pages.cuda(), lens.cuda(), 4, out, out_lens)
        assert torch.equal(out.cpu(), want) and torch.equal(out_lens.cpu(), want_lens), d


# ---------------------------------------------------------------------------
# Caches past 32-bit offsets: pages 2^31 elements apart, and a bit.

@pytest.mark.parametrize("dtype,t,hq", [("bf16", 7, 2), ("bf16", 40, 8), ("f32", 9, 2)])
def test_caches_past_32_bits(dtype, t, hq):
    dt, g = DT[dtype], gen(3)
    n, page, hk, d, b, cols = 3, 16, 2, 64, 1, 3
    stride = (1 << 31) + 64
    def far(x):
        base = torch.empty(2 * stride + page * hk * d, dtype=dt, device="cuda")
        view = base.as_strided((n, page, hk, d), (stride, hk * d, d, 1))
        view.copy_(x)
        return view
    kc, vc = randn(g, n, page, hk, d, dtype=dt), randn(g, n, page, hk, d, dtype=dt)
    kg, vg = far(kc), far(vc)
    pages, lens = ints([[2, 0, 1]]), ints([page * cols - t - 1 if t < 30 else 5])
    q = randn(g, b, t, hq, d, dtype=dt)
    parent = ints([[i - 1 for i in range(t)]])
    scale = 1.0 / math.sqrt(d)
    want, want_lse, eo, el = C.tree(q, kc, vc, pages, lens, parent, scale)
    out, lse = new(b, t, hq, d, dtype=dt), new(b, t, hq, dtype=torch.float32)
    E.tree_attention(q.cuda(), kg, vg, pages.cuda(), lens.cuda(), parent.cuda(), out, lse=lse)
    within(out, want, eo)
    within(lse, want_lse, el)
    bounds, since = new(n, hk, 2, d, dtype=dt, fill=1), ints([0])
    E.page_bounds(kg, pages.cuda(), lens.cuda(), since.cuda(), bounds)
    assert torch.equal(bounds.cpu(), C.bounds(kc, pages, lens, since, torch.ones(n, hk, 2, d, dtype=dt)))
    mass, none = new(b, cols, dtype=torch.float32), torch.zeros(b, cols)
    first = q[:, 0]
    ls = torch.zeros(b, hq)
    want, bound = C.mass(first, kc, pages, lens, ls, none, scale, 1.0)
    E.page_mass(first.cuda(), kg, pages.cuda(), lens.cuda(), ls.cuda(), none.cuda(), mass)
    within(mass, want, bound)
    path = ints([[0, 2] + [-1] * (t - 2)])
    moved = C.move([kc, vc], pages, lens, path)
    E.slot_move([kg, vg], pages.cuda(), lens.cuda(), path.cuda())
    assert torch.equal(kg.cpu(), moved[0]) and torch.equal(vg.cpu(), moved[1])


# ---------------------------------------------------------------------------
# Streams, workspaces, graphs.

def tree_call(seed, case=(3, 12, 8, 2, 64, 64, 16, 100, 0), dtype="bf16"):
    q, caches, _, pages, lens, parent, window = tree_state(case, dtype, seed)
    args = [q.cuda(), *caches, pages.cuda(), lens.cuda(), parent.cuda()]
    return args, torch.empty(*q.shape[:3], caches[1].shape[3], dtype=q.dtype, device="cuda")


def select_call(seed):
    g, rng = gen(seed), random.Random(seed)
    bounds = torch.sort(randn(g, 90, 2, 2, 64, dtype=torch.bfloat16), dim=2).values
    return [randn(g, 3, 8, 64, dtype=torch.bfloat16).cuda(), bounds.cuda(), table(rng, 90, 3, 60).cuda(),
            ints([rng.randint(400, 960) for _ in range(3)]).cuda(), 16], (new(3, 2, 9), new(3, 2))


def test_streams_and_workspaces():
    args, out = tree_call(6)
    E.tree_attention(*args, out)
    sel, picked = select_call(1)
    E.page_select(*sel, *picked)
    need, need_sel = E.tree_attention_workspace(*args, out), E.page_select_workspace(*sel, *picked)
    assert need > 0 and need_sel > 0
    for how in ("stream", "handle", "own workspace"):
        other, other_picked = torch.empty_like(out), (new(3, 2, 9), new(3, 2))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        stream = s.cuda_stream if how == "handle" else s
        own = lambda size: dict(workspace=torch.empty(size, dtype=torch.uint8, device="cuda")) if how == "own workspace" else {}
        E.tree_attention(*args, other, stream=stream, **own(need))
        E.page_select(*sel, *other_picked, stream=stream, **own(need_sel))
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(other, out) and all(torch.equal(a, b) for a, b in zip(other_picked, picked)), how
    with pytest.raises(E.Error):
        E.tree_attention(*args, out, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(E.Error):
        E.page_select(*sel, *picked, workspace=torch.empty(need_sel - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(E.Error):
        E.tree_attention(args[0].cpu(), *args[1:], out)


def test_default_stream_by_its_handle(monkeypatch):
    """stream=0: the scratch memory is of the default stream too."""
    import types

    from elementwise_tensor_commands_amd import serving as S
    args, out = tree_call(6)
    sel, picked = select_call(1)
    E.tree_attention(*args, out)
    E.page_select(*sel, *picked)
    allocated_on = []

    def scratch(size, device):
        allocated_on.append(torch.cuda.current_stream().cuda_stream)
        return binding.scratch(size, device)

    binding = S._binding
    monkeypatch.setattr(S, "_binding", types.SimpleNamespace(**{**vars(binding), "scratch": scratch}))
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        other, other_picked = torch.empty_like(out), (new(3, 2, 9), new(3, 2))
        torch.cuda.synchronize()
        E.tree_attention(*args, other, stream=0)
        E.page_select(*sel, *other_picked, stream=0)
    torch.cuda.synchronize()
    assert allocated_on == [0, 0]
    assert torch.equal(other, out) and all(torch.equal(a, b) for a, b in zip(other_picked, picked))


def test_two_calls_at_once():
    """Calls on two streams, each with scratch memory of its own."""
    calls = [tree_call(s, case) for s, case in ((6, (3, 12, 8, 2, 64, 64, 16, 100, 0)), (7, (2, 40, 16, 2, 64, 64, 16, 200, 0)))]
    want = []
    for args, out in calls:
        E.tree_attention(*args, out)
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        for (args, out), s in zip(calls, streams):
            with torch.cuda.stream(s):
                E.tree_attention(*args, out)
    torch.cuda.synchronize()
    for (_, out), w in zip(calls, want):
        assert torch.equal(out, w)


def test_version_counters_advance():
    args, out = tree_call(6)
    lse = new(*out.shape[:3], dtype=torch.float32)
    before = [x._version for x in (out, lse, *args)]
    E.tree_attention(*args, out, lse=lse)
    assert [x._version for x in (out, lse, *args)] == [before[0] + 1, before[1] + 1] + before[2:]
    sel, picked = select_call(1)
    E.page_select(*sel, *picked)
    assert all(x._version == 1 for x in picked)
    pool = torch.zeros(4, 4, 1, 8, device="cuda")
    E.slot_move([pool], new(1, 2, fill=0), new(1, fill=0), new(1, 2, fill=-1))
    assert pool._version == 1


def test_captured_calls():
    """All of them in a graph, replayed with other inputs and eager work between."""
    def build():
        g, rng = gen(9), random.Random(9)
        n, page, hk, d, rows, cols, t = 64, 16, 2, 64, 3, 20, 6
        s = dict(k=randn(g, n, page, hk, d, dtype=torch.bfloat16), v=randn(g, n, page, hk, d, dtype=torch.bfloat16),
                 pages=table(rng, n, rows, cols, holes=0.0), lens=ints([200, 17, 90]), refs=torch.ones(n, dtype=I32),
                 q=randn(g, rows, t, 8, d, dtype=torch.bfloat16), parent=ints([[-1, 0, 0, 1, 3, -2]] * rows),
                 tokens=ints([[1, 2, 3, 4, 5, 6]] * rows), follow=ints([[3, 4, 9, 9, 9, 9], [2, 4, 9, 5, 9, 9], [7, 9, 9, 9, 9, 9]]),
                 out=torch.zeros(rows, t, 8, d, dtype=torch.bfloat16), path=torch.zeros(rows, t, dtype=I32), lens2=ints([0] * rows),
                 last=ints([0] * rows), bounds=torch.zeros(n, hk, 2, d, dtype=torch.bfloat16), since=ints([0] * rows),
                 picked=torch.zeros(rows, hk, 4, dtype=I32), picked_lens=torch.zeros(rows, hk, dtype=I32),
                 one=torch.zeros(rows, 8, d, dtype=torch.bfloat16), some=torch.zeros(rows, 8, d, dtype=torch.bfloat16),
                 lse=torch.zeros(rows, 8), mass=torch.zeros(rows, cols), budget=ints([9, 99, 4]), pages2=torch.zeros(rows, cols, dtype=I32),
                 refs2=torch.zeros(n, dtype=I32), count=ints([0] * rows))
        return {k: v.cuda() for k, v in s.items()}

    def step(s):
        E.tree_attention(s["q"], s["k"], s["v"], s["pages"], s["lens"], s["parent"], s["out"])
        E.tree_accept(s["tokens"], s["parent"], s["follow"], s["lens"], s["path"], s["lens2"], s["last"])
        E.slot_move([s["k"], s["v"]], s["pages"], s["lens"], s["path"])
        E.page_bounds(s["k"], s["pages"], s["lens2"], s["since"], s["bounds"])
        one = s["q"][:, 0]
        E.page_select(one, s["bounds"], s["pages"], s["lens2"], 16, s["picked"], s["picked_lens"], first=1, last=1)
        E.paged_attention(one, s["k"], s["v"], s["picked"], s["picked_lens"], s["some"])
        E.paged_attention(one, s["k"], s["v"], s["pages"], s["lens2"], s["one"], lse=s["lse"])
        E.page_mass(one, s["k"], s["pages"], s["lens2"], s["lse"], s["mass"], s["mass"], decay=0.5)
        E.page_evict(s["pages"], s["lens2"], s["refs"], s["mass"], s["budget"], 16, s["pages2"], s["refs2"], s["count"])

    eager, captured = build(), build()
    step(eager), step(captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    g = gen(4)
    for i, lens in enumerate([[200, 17, 90], [0, 300, 1], [160, 161, 314], [32, 31, 33]]):
        q, follow = randn(g, 3, 6, 8, 64, dtype=torch.bfloat16).cuda(), torch.randint(2, 7, (3, 6), generator=g).to(I32).cuda()
        for s in (eager, captured):
            s["lens"].copy_(ints(lens)), s["q"].copy_(q), s["follow"].copy_(follow)
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for key in eager:
            assert torch.equal(eager[key], captured[key]), (i, key)
