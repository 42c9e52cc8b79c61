"""The operators on trees of drafted tokens and on pages worth reading or keeping, on the
host: argument checks (every refusal comes before any HIP call, so CPU tensors do),
workspace sizes, what one launch holds, and their oracle against hand-worked cases."""
import math
import os
import re

import pytest
import torch

import cache_oracle as C
import elementwise_tensor_commands_amd as E
from test_serving_host import I32, ROOT, _refused, build_module, check_only, i32, made_up

INF = math.inf


def accepted(fn, *args, **kw):
    """All checks pass: what is left to refuse is that no GPU holds the tensors."""
    assert "GPU" in _refused("CMD_E_ARG", fn, *args, **kw)


def test_library_exports_every_new_function():
    for name in ("paged_attention_heads", "paged_attention_heads_workspace", "tree_attention", "tree_attention_workspace", "tree_accept",
                 "slot_move", "page_bounds", "page_select", "page_select_workspace", "page_mass", "page_evict"):
        assert hasattr(E.lib, "cmd_" + name), name


# ---------------------------------------------------------------------------
# Attention for trees.

def tree_args(**kw):
    a = dict(q=torch.zeros(3, 5, 4, 8), k=torch.zeros(7, 16, 2, 8), v=torch.zeros(7, 16, 2, 6), pages=i32(3, 2), lens=i32(3),
             parent=i32(3, 5), out=torch.zeros(3, 5, 4, 6))
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("name,kw", [
    ("CMD_E_DTYPE", dict(q=torch.zeros(3, 5, 4, 8, dtype=torch.float64))),
    ("CMD_E_DTYPE", dict(k=torch.zeros(7, 16, 2, 8, dtype=torch.float16))),
    ("CMD_E_DTYPE", dict(parent=torch.zeros(3, 5, dtype=torch.int64))),
    ("CMD_E_DTYPE", dict(out=torch.zeros(3, 5, 4, 6, dtype=torch.bfloat16))),
    ("CMD_E_SHAPE", dict(q=torch.zeros(3, 4, 8))),
    ("CMD_E_SHAPE", dict(q=torch.zeros(3, 5, 4, 9))),
    ("CMD_E_SHAPE", dict(q=torch.zeros(3, 5, 3, 8), out=torch.zeros(3, 5, 3, 6))),
    ("CMD_E_SHAPE", dict(v=torch.zeros(7, 15, 2, 6))),
    ("CMD_E_SHAPE", dict(pages=i32(2, 2))),
    ("CMD_E_SHAPE", dict(lens=i32(4))),
    ("CMD_E_SHAPE", dict(parent=i32(3, 4))),
    ("CMD_E_SHAPE", dict(out=torch.zeros(3, 5, 4, 8))),
    ("CMD_E_SHAPE", dict(q=torch.zeros(3, 5, 4, 0), k=torch.zeros(7, 16, 2, 0))),
    ("CMD_E_LIMIT", dict(q=torch.zeros(3, 257, 4, 8), parent=i32(3, 257), out=torch.zeros(3, 257, 4, 6))),
    ("CMD_E_LIMIT", dict(q=torch.zeros(3, 5, 4, 257), k=torch.zeros(7, 16, 2, 257))),
    ("CMD_E_LIMIT", dict(pages=torch.zeros(3, 1, dtype=I32).expand(3, 1 << 27))),
    ("CMD_E_STRIDE", dict(q=torch.zeros(3, 5, 8, 4).transpose(2, 3))),
    ("CMD_E_STRIDE", dict(out=torch.zeros(3, 1, 4, 6).expand(3, 5, 4, 6))),
    ("CMD_E_STRIDE", dict(out=torch.zeros(3, 5, 4, 12)[..., ::2])),
])
def test_tree_refusals(name, kw):
    _refused(name, E.tree_attention, *tree_args(**kw))
    _refused(name, E.tree_attention_workspace, *tree_args(**kw))


def test_tree_options_and_aliases():
    accepted(E.tree_attention, *tree_args())
    accepted(E.tree_attention, *tree_args(), lse=torch.zeros(3, 5, 4), window=1)
    accepted(E.tree_attention, *tree_args(out=torch.zeros(5, 3, 4, 9)[..., 2:8].transpose(0, 1)), lse=torch.zeros(4, 5, 6).permute(2, 1, 0)[::2])
    _refused("CMD_E_ARG", E.tree_attention, *tree_args(), window=-1)
    _refused("CMD_E_ARG", E.tree_attention, *tree_args(), scale=math.nan)
    _refused("CMD_E_ARG", E.tree_attention, *tree_args(), scale=3e38)
    _refused("CMD_E_SHAPE", E.tree_attention, *tree_args(), lse=torch.zeros(3, 4, 5))
    _refused("CMD_E_DTYPE", E.tree_attention, *tree_args(), lse=torch.zeros(3, 5, 4, dtype=torch.float64))
    a = tree_args(v=torch.zeros(7, 16, 2, 8))
    a[6] = a[0]
    _refused("CMD_E_ALIAS", E.tree_attention, *a)
    buf = torch.zeros(2000)
    _refused("CMD_E_ALIAS", E.tree_attention, *tree_args(out=buf[:360].view(3, 5, 4, 6)), lse=buf[300:360].view(3, 5, 4))


def test_tree_workspace():
    from elementwise_tensor_commands_amd import serving as S
    assert E.tree_attention_workspace(*tree_args()) == 0                              # too few keys to cut
    a = tree_args(pages=i32(3, 4096))
    need = E.tree_attention_workspace(*a)
    assert need > 0 and E.tree_attention_workspace(*a, window=100) == 0
    args = S._pack(S._TREE, *a, None)[0]
    buf = torch.zeros(need, dtype=torch.uint8)
    call = E.lib.cmd_tree_attention
    assert call(args, 1.0, 0, None, 0, 0, None) == -1
    assert call(args, 1.0, 0, buf.data_ptr(), need - 1, 0, None) == -1 and b"workspace" in E.lib.cmd_last_error(None)
    assert call(None, 1.0, 0, None, 0, 0, None) == -1 and call(args, 1.0, 0, None, 0, 2, None) == -1
    assert call(args, 1.0, 0, None, 0, S.CHECK_ONLY, None) == 0
    # nothing to do needs nothing
    for kw in (dict(q=torch.zeros(3, 0, 4, 8), parent=i32(3, 0), out=torch.zeros(3, 0, 4, 6)),
               dict(q=torch.zeros(0, 5, 4, 8), pages=i32(0, 2), lens=i32(0), parent=i32(0, 5), out=torch.zeros(0, 5, 4, 6))):
        assert E.tree_attention_workspace(*tree_args(**kw)) == 0


# ---------------------------------------------------------------------------
# The accepted path.

def accept_args(**kw):
    a = dict(tokens=i32(3, 5), parent=i32(3, 5), next=i32(3, 5), lens=i32(3), path=i32(3, 5), lens_out=i32(3), last=i32(3))
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("name,kw", [
    ("CMD_E_DTYPE", dict(tokens=torch.zeros(3, 5, dtype=torch.int64))),
    ("CMD_E_DTYPE", dict(last=torch.zeros(3))),
    ("CMD_E_SHAPE", dict(tokens=i32(15))),
    ("CMD_E_SHAPE", dict(parent=i32(3, 4))),
    ("CMD_E_SHAPE", dict(next=i32(4, 5))),
    ("CMD_E_SHAPE", dict(path=i32(3, 6))),
    ("CMD_E_SHAPE", dict(lens_out=i32(5))),
    ("CMD_E_LIMIT", {k: i32(3, 257) for k in ("tokens", "parent", "next", "path")}),
    ("CMD_E_STRIDE", dict(path=i32(3, 1).expand(3, 5))),
])
def test_accept_refusals(name, kw):
    _refused(name, E.tree_accept, *accept_args(**kw))


def test_accept_aliases():
    a = accept_args()
    a[5] = a[3]
    accepted(E.tree_accept, *a)                                      # the lengths may be updated in place
    for out, of in ((4, 0), (4, 1), (4, 2), (6, 3), (6, 5)):
        a = accept_args()
        a[out] = a[of]
        _refused("CMD_E_ALIAS", E.tree_accept, *a)
    both = i32(4)
    _refused("CMD_E_ALIAS", E.tree_accept, *accept_args(lens=both[:3], lens_out=both[1:]))


def test_move_refusals():
    pool, pages, lens, path = torch.zeros(7, 16, 2, 8), i32(3, 2), i32(3), i32(3, 5)
    accepted(E.slot_move, [pool, torch.zeros(9, 16, 3, 5, dtype=torch.float16), i32(7, 16, 1, 1)], pages, lens, path)
    accepted(E.slot_move, [pool.transpose(1, 2).contiguous().transpose(1, 2)], pages, lens, path)
    _refused("CMD_E_SHAPE", E.slot_move, [pool, torch.zeros(7, 8, 2, 8)], pages, lens, path)
    _refused("CMD_E_SHAPE", E.slot_move, [pool[0]], pages, lens, path)
    _refused("CMD_E_SHAPE", E.slot_move, [pool], pages, i32(4), path)
    _refused("CMD_E_SHAPE", E.slot_move, [pool], pages, lens, i32(2, 5))
    _refused("CMD_E_DTYPE", E.slot_move, [pool.to(torch.int8)], pages, lens, path)
    _refused("CMD_E_DTYPE", E.slot_move, [pool], pages.long(), lens, path)
    _refused("CMD_E_STRIDE", E.slot_move, [pool[..., ::2]], pages, lens, path)
    _refused("CMD_E_STRIDE", E.slot_move, [pool[:1].expand(7, 16, 2, 8)], pages, lens, path)
    _refused("CMD_E_ALIAS", E.slot_move, [pool, pool[1:]], pages, lens, path)
    _refused("CMD_E_ALIAS", E.slot_move, [pages.view(1, 3, 2, 1)], pages, lens, path)
    _refused("CMD_E_LIMIT", E.slot_move, [pool], pages, lens, i32(3, 257))
    _refused("CMD_E_LIMIT", E.slot_move, [pool], i32(3, 1).expand(3, 1 << 27), lens, path)
    # the second pool's fault is found before the first one's launch
    from elementwise_tensor_commands_amd import serving as S
    bad = S._pack(b"\2\1\2\4\4", pages, lens, path, pool, torch.zeros(7, 16, 2, 8)[..., ::2])[0]
    assert E.lib.cmd_slot_move(bad[3 * S._SIZE:], 2, bad[:3 * S._SIZE], 0, None) != 0
    assert E.lib.cmd_slot_move(None, 1, bad[:3 * S._SIZE], 0, None) == -1
    assert E.lib.cmd_slot_move(bad[3 * S._SIZE:], -1, bad[:3 * S._SIZE], 0, None) == -1


# ---------------------------------------------------------------------------
# Pages worth reading.

def bounds_args(**kw):
    a = dict(k=torch.zeros(7, 16, 2, 8), pages=i32(3, 2), lens=i32(3), since=i32(3), bounds=torch.zeros(7, 2, 2, 8))
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("name,kw", [
    ("CMD_E_DTYPE", dict(bounds=torch.zeros(7, 2, 2, 8, dtype=torch.float16))),
    ("CMD_E_DTYPE", dict(k=torch.zeros(7, 16, 2, 8, dtype=I32))),
    ("CMD_E_SHAPE", dict(bounds=torch.zeros(7, 2, 3, 8))),
    ("CMD_E_SHAPE", dict(bounds=torch.zeros(6, 2, 2, 8))),
    ("CMD_E_SHAPE", dict(since=i32(2))),
    ("CMD_E_STRIDE", dict(bounds=torch.zeros(1, 2, 2, 8).expand(7, 2, 2, 8))),
    ("CMD_E_STRIDE", dict(k=torch.zeros(7, 16, 2, 16)[..., ::2])),
    ("CMD_E_LIMIT", dict(pages=i32(3, 1).expand(3, 1 << 27))),
])
def test_bounds_refusals(name, kw):
    _refused(name, E.page_bounds, *bounds_args(**kw))


def test_bounds_aliases():
    accepted(E.page_bounds, *bounds_args())
    both = torch.zeros(7, 20, 2, 8)                                   # bounds beside the slots of their page
    accepted(E.page_bounds, *bounds_args(k=both[:, :16], bounds=both[:, 16:18]))
    _refused("CMD_E_ALIAS", E.page_bounds, *bounds_args(k=both[:, :16], bounds=both[:, 14:16]))


def select_args(**kw):
    a = dict(q=torch.zeros(3, 4, 8), bounds=torch.zeros(7, 2, 2, 8), pages=i32(3, 9), lens=i32(3), page=16, pages_out=i32(3, 2, 4),
             lens_out=i32(3, 2))
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("name,kw", [
    ("CMD_E_DTYPE", dict(q=torch.zeros(3, 4, 8, dtype=torch.bfloat16))),
    ("CMD_E_DTYPE", dict(pages_out=torch.zeros(3, 2, 4))),
    ("CMD_E_SHAPE", dict(q=torch.zeros(3, 5, 8))),
    ("CMD_E_SHAPE", dict(bounds=torch.zeros(7, 2, 1, 8))),
    ("CMD_E_SHAPE", dict(pages_out=i32(3, 3, 4))),
    ("CMD_E_SHAPE", dict(lens_out=i32(3, 4))),
    ("CMD_E_ARG", dict(page=0)),
    ("CMD_E_ARG", dict(pages_out=i32(3, 2, 2))),                      # 1 first and 2 last of 2
    ("CMD_E_ARG", dict(pages_out=i32(3, 2, 0))),
    ("CMD_E_LIMIT", dict(q=torch.zeros(3, 4, 257), bounds=torch.zeros(7, 2, 2, 257))),
    ("CMD_E_LIMIT", dict(pages=i32(3, 1).expand(3, (1 << 20) + 1))),
    ("CMD_E_STRIDE", dict(pages_out=i32(3, 1, 4).expand(3, 2, 4))),
])
def test_select_refusals(name, kw):
    _refused(name, E.page_select, *select_args(**kw))
    _refused(name, E.page_select_workspace, *select_args(**kw))


def test_select_options_and_workspace():
    from elementwise_tensor_commands_amd import serving as S
    accepted(E.page_select, *select_args())
    accepted(E.page_select, *select_args(), first=0, last=0)
    accepted(E.page_select, *select_args(), first=3, last=1)
    for kw in (dict(first=-1), dict(last=-1), dict(first=3, last=2)):
        _refused("CMD_E_ARG", E.page_select, *select_args(), **kw)
    a = select_args()
    a[5] = a[2][:, :8].view(3, 2, 4)
    _refused("CMD_E_ALIAS", E.page_select, *a)
    need = E.page_select_workspace(*select_args())
    assert need == 3 * 2 * 9 * 8                                      # a score each
    assert E.page_select_workspace(*select_args(pages=i32(3, 0))) == 0
    assert E.page_select_workspace(*select_args(q=torch.zeros(0, 4, 8), pages=i32(0, 9), lens=i32(0), pages_out=i32(0, 2, 4),
                                                lens_out=i32(0, 2))) == 0
    a = select_args()
    args = S._pack(S._SELECT, a[0], a[1], a[2], a[3], a[5], a[6])[0]
    buf = torch.zeros(need, dtype=torch.uint8)
    call = E.lib.cmd_page_select
    assert call(args, 16, 1, 2, buf.data_ptr(), need - 1, 0, None) == -1 and b"workspace" in E.lib.cmd_last_error(None)
    assert call(args, 16, 1, 2, None, 0, 0, None) == -1 and call(None, 16, 1, 2, None, 0, 0, None) == -1
    assert call(args, 16, 1, 2, None, 0, S.CHECK_ONLY, None) == 0


def test_tables_of_heads():
    """paged_attention takes a table for every kv head; the lengths then too."""
    q, k, v, out = torch.zeros(3, 4, 8), torch.zeros(7, 16, 2, 8), torch.zeros(7, 16, 2, 6), torch.zeros(3, 4, 6)
    accepted(E.paged_attention, q, k, v, i32(3, 2, 5), i32(3, 2), out)
    assert E.paged_attention_workspace(q, k, v, i32(3, 2, 4096), i32(3, 2), out) > 0
    _refused("CMD_E_SHAPE", E.paged_attention, q, k, v, i32(3, 2, 5), i32(3), out)
    _refused("CMD_E_SHAPE", E.paged_attention, q, k, v, i32(3, 3, 5), i32(3, 3), out)
    _refused("CMD_E_SHAPE", E.paged_attention, q, k, v, i32(3, 2, 5), i32(3, 3), out)
    _refused("CMD_E_SHAPE", E.paged_attention, q, k, v, i32(3, 5), i32(3, 2), out)


# ---------------------------------------------------------------------------
# Pages worth keeping.

def mass_args(**kw):
    a = dict(q=torch.zeros(3, 4, 8), k=torch.zeros(7, 16, 2, 8), pages=i32(3, 2), lens=i32(3), lse=torch.zeros(3, 4),
             mass=torch.zeros(3, 2), out=torch.zeros(3, 2))
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("name,kw", [
    ("CMD_E_DTYPE", dict(k=torch.zeros(7, 16, 2, 8, dtype=torch.float16))),
    ("CMD_E_DTYPE", dict(mass=torch.zeros(3, 2, dtype=torch.float64))),
    ("CMD_E_SHAPE", dict(lse=torch.zeros(3, 2))),
    ("CMD_E_SHAPE", dict(mass=torch.zeros(3, 3))),
    ("CMD_E_SHAPE", dict(out=torch.zeros(2, 2))),
    ("CMD_E_SHAPE", dict(q=torch.zeros(3, 5, 8), lse=torch.zeros(3, 5))),
    ("CMD_E_LIMIT", dict(q=torch.zeros(3, 4, 257), k=torch.zeros(7, 16, 2, 257))),
    ("CMD_E_LIMIT", dict(pages=i32(3, 1).expand(3, 1 << 27), mass=torch.zeros(3, 1).expand(3, 1 << 27), out=torch.zeros(1))),
    ("CMD_E_STRIDE", dict(out=torch.zeros(3, 1).expand(3, 2))),
    ("CMD_E_STRIDE", dict(q=torch.zeros(3, 8, 4).transpose(1, 2))),
])
def test_mass_refusals(name, kw):
    if name == "CMD_E_LIMIT" and "out" in kw:                          # nothing of that size is made
        args = [made_up("f32", (3, 4, 8), 1), made_up("f32", (7, 16, 2, 8), 2), made_up("i32", (3, 1 << 27), 3, (0, 0)),
                made_up("i32", (3,), 4), made_up("f32", (3, 4), 5), made_up("f32", (3, 1 << 27), 6), made_up("f32", (3, 1 << 27), 7)]
        assert E.Error(check_only("cmd_page_mass", args, 1.0, 1.0, 0), "").name == name
        return
    _refused(name, E.page_mass, *mass_args(**kw))


def test_mass_options_and_aliases():
    accepted(E.page_mass, *mass_args())
    a = mass_args()
    a[6] = a[5]
    accepted(E.page_mass, *a, decay=0.5, window=3)                     # added up in place
    for kw in (dict(window=-1), dict(scale=INF), dict(decay=INF), dict(decay=math.nan)):
        _refused("CMD_E_ARG", E.page_mass, *mass_args(), **kw)
    both = torch.zeros(3, 3)
    _refused("CMD_E_ALIAS", E.page_mass, *mass_args(mass=both[:, :2], out=both[:, 1:]))


def evict_args(**kw):
    a = dict(pages=i32(3, 4), lens=i32(3), refs=i32(9), mass=torch.zeros(3, 4), budget=i32(3), page=16, pages_out=i32(3, 4),
             refs_out=i32(9), count=i32(3))
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("name,kw", [
    ("CMD_E_DTYPE", dict(mass=i32(3, 4))),
    ("CMD_E_DTYPE", dict(budget=torch.zeros(3))),
    ("CMD_E_SHAPE", dict(mass=torch.zeros(4, 3))),
    ("CMD_E_SHAPE", dict(pages_out=i32(3, 5))),
    ("CMD_E_SHAPE", dict(refs_out=i32(8))),
    ("CMD_E_SHAPE", dict(count=i32(4))),
    ("CMD_E_ARG", dict(page=0)),
    ("CMD_E_LIMIT", dict(page=1 << 29)),
    ("CMD_E_STRIDE", dict(refs_out=i32(1).expand(9))),
])
def test_evict_refusals(name, kw):
    _refused(name, E.page_evict, *evict_args(**kw))


def test_evict_options_and_aliases():
    a = evict_args()
    a[6], a[7] = a[0], a[2]
    accepted(E.page_evict, *a)                                         # in place
    accepted(E.page_evict, *evict_args(), first=9, last=9)
    for kw in (dict(first=-1), dict(last=-1)):
        _refused("CMD_E_ARG", E.page_evict, *evict_args(), **kw)
    a = evict_args()
    a[8] = a[4]
    _refused("CMD_E_ALIAS", E.page_evict, *a)
    both = i32(10)
    _refused("CMD_E_ALIAS", E.page_evict, *evict_args(refs=both[:9], refs_out=both[1:]))


# ---------------------------------------------------------------------------
# What one launch holds: 2^24 - 1 work-groups.

def test_calls_larger_than_a_launch():
    def name(rc):
        return "ok" if rc == 0 else E.Error(rc, "").name

    def tree(b, t, hk, group, cols):
        q, none = made_up("f16", (b, t, hk * group, 8), 1), E.cmd_arg()
        cache = [made_up("f16", (4, 16, hk, 8), 2 + i) for i in range(2)]
        return name(check_only("cmd_tree_attention", [q, *cache, made_up("i32", (b, cols), 4, (0, 0)), made_up("i32", (b,), 5),
                                                      made_up("i32", (b, t), 6, (0, 0)), made_up("f16", (b, t, hk * group, 8), 7), none],
                               1.0, 0, None, 0))

    assert tree(131000, 1, 128, 1, 8) == "ok"
    assert tree(131072, 1, 128, 1, 8) == "CMD_E_LIMIT"
    assert tree(65000, 256, 4, 1, 4) == "ok"
    assert tree(65600, 256, 4, 1, 4) == "CMD_E_LIMIT"                  # the second launch, a vector to a wave

    def select(b, hk, cols):
        return name(check_only("cmd_page_select", [made_up("f16", (b, hk, 8), 1), made_up("f16", (4, hk, 2, 8), 2),
                                                   made_up("i32", (b, cols), 3, (0, 0)), made_up("i32", (b,), 4),
                                                   made_up("i32", (b, hk, 4), 5), made_up("i32", (b, hk), 6)], 16, 1, 2, None, 0))

    assert select((1 << 17) - 1, 128, 9) == "ok"
    assert select(1 << 17, 128, 9) == "CMD_E_LIMIT"

    def mass(b, cols, page):
        return name(check_only("cmd_page_mass", [made_up("f16", (b, 2, 8), 1), made_up("f16", (4, page, 2, 8), 2),
                                                 made_up("i32", (b, cols), 3, (0, 0)), made_up("i32", (b,), 4), made_up("f32", (b, 2), 5),
                                                 made_up("f32", (b, cols), 6), made_up("f32", (b, cols), 7)], 1.0, 1.0, 0))

    assert mass((1 << 23) - 1, 2, 64) == "ok"
    assert mass(1 << 23, 2, 64) == "CMD_E_LIMIT"

    def rows(fn, n):
        i = lambda at, *shape: made_up("i32", shape, at)
        if fn == "accept":
            return name(check_only("cmd_tree_accept", [i(1, n, 2), i(2, n, 2), i(3, n, 2), i(4, n), i(5, n, 2), i(6, n), i(7, n)]))
        if fn == "bounds":
            return name(check_only("cmd_page_bounds", [made_up("f16", (4, 16, 2, 8), 1), i(2, n, 2), i(3, n), i(4, n),
                                                       made_up("f16", (4, 2, 2, 8), 5)]))
        if fn == "evict":
            return name(check_only("cmd_page_evict", [i(1, n, 2), i(2, n), i(3, 9), made_up("f32", (n, 2), 4), i(5, n), i(6, n, 2), i(7, 9),
                                                      i(8, n)], 16, 0, 1))
        return name(E.lib.cmd_slot_move(bytes(made_up("f16", (4, 16, 2, 8), 1)), 1, b"".join(map(bytes, (i(2, n, 2), i(3, n), i(4, n, 2)))),
                                        1, None))

    for fn in ("accept", "bounds", "evict", "move"):
        assert rows(fn, (1 << 24) - 1) == "ok", fn
        assert rows(fn, 1 << 24) == "CMD_E_LIMIT", fn


# ---------------------------------------------------------------------------
# The oracle.

def test_oracle_of_trees_by_hand():
    # 0 -> 1 -> 3, 0 -> 2, 4 after the context, 5 and 6 below it are padding
    assert C.above([-1, 0, 0, 1, -1, 5, 5]) == [[0], [1, 0], [2, 0], [3, 1, 0], [4], None, None]
    q = torch.ones(1, 3, 1, 1)
    k = torch.zeros(3, 2, 1, 1)
    v = torch.tensor([1.0, 2.0, 4.0, 8.0, 16.0, 32.0]).view(3, 2, 1, 1)
    pages, lens, parent = torch.tensor([[2, 0, 1]]), [2], torch.tensor([[-1, 0, 0]])
    # positions hold 16, 32 (the context), then 1, 2, 4 of the tokens
    out, lse, _, _ = C.tree(q, k, v, pages, lens, parent, 1.0)
    assert torch.allclose(out.view(3), torch.tensor([49 / 3, 51 / 4, 53 / 4], dtype=torch.float64))
    assert torch.allclose(lse.view(3), torch.tensor([3.0, 4.0, 4.0], dtype=torch.float64).log())
    out, _, _, _ = C.tree(q, k, v, pages, lens, parent, 1.0, window=2)   # itself and the one above
    assert torch.allclose(out.view(3), torch.tensor([33 / 2, 3 / 2, 5 / 2], dtype=torch.float64))
    out, lse, _, _ = C.tree(q, k, v, pages, lens, torch.tensor([[-2, 0, -1]]), 1.0)
    assert out.view(3).tolist()[:2] == [0.0, 0.0] and lse.view(3).tolist()[:2] == [-INF, -INF]
    out, _, _, _ = C.tree(q, k, v, torch.tensor([[2, -1, 1]]), [2], parent, 1.0)   # tokens 0 and 1 in a hole
    assert torch.allclose(out.view(3), torch.tensor([24.0, 24.0, 52 / 3], dtype=torch.float64))


def test_oracle_of_paths_by_hand():
    tokens, parent = torch.tensor([[9, 4, 5, 6, 5, 7]]), torch.tensor([[-1, 0, 0, 2, 0, 3]])
    follow = torch.tensor([[5, 0, 6, 8, 1, 2]])
    path, lens, last = C.accept(tokens, parent, follow, torch.tensor([10]))
    assert path == [[0, 2, 3, -1, -1, -1]] and lens == [13] and last == [8]
    path, lens, last = C.accept(tokens, torch.tensor([[0, 0, 0, 2, 0, 3]]), follow, torch.tensor([10]))
    assert path == [[-1] * 6] and lens == [10] and last == [-1]


def test_oracle_of_pages_by_hand():
    k = torch.tensor([[1.0, 5.0], [3.0, -2.0]]).view(2, 2, 1, 1)        # page 0 holds 1, 5; page 1 holds 3, -2
    was = torch.full((2, 1, 2, 1), 7.0)
    got = C.bounds(k, torch.tensor([[1, 0]]), [3], [1], was)
    assert got[1].flatten().tolist() == [-2.0, 7.0] and got[0].flatten().tolist() == [1.0, 1.0]   # widened; made anew
    bounds = torch.tensor([[-1.0, 1.0], [0.0, 3.0], [-5.0, 0.0], [2.0, 2.0]]).view(4, 1, 2, 1)
    table = torch.tensor([[0, 1, 2, 3]])
    pick = lambda q, **kw: C.select(torch.tensor([[[q]]]), bounds, table, [7], 2, kw.get("take", 2), kw.get("first", 0), kw.get("last", 0))
    pages, lens = pick(1.0)
    assert pages.tolist() == [[[1, 3]]] and lens.tolist() == [[3]]       # the last page holds one position
    pages, lens = pick(-1.0)
    assert pages.tolist() == [[[0, 2]]] and lens.tolist() == [[4]]
    pages, _ = pick(1.0, first=1, last=1)
    assert pages.tolist() == [[[0, 3]]]
    pages, refs, count = C.evict(torch.tensor([[3, 1, -1, 0]]), [7], torch.tensor([1, 1, 0, 2]), torch.tensor([[0.5, 0.25, 0.0, 0.1]]), [1], 2, 0, 1)
    assert pages == [[-1, -1, -1, 0]] and refs == [1, 0, 0, 1] and count == [2]
    q, key = torch.ones(1, 1, 1), torch.zeros(2, 2, 1, 1)
    m = C.mass(q, key, torch.tensor([[1, 0]]), [3], torch.tensor([[math.log(3.0)]]), torch.tensor([[2.0, 4.0]]), 1.0, 0.5)[0]
    assert torch.allclose(m, torch.tensor([[1 + 2 / 3, 2 + 1 / 3]], dtype=torch.float64))


# ---------------------------------------------------------------------------
# The kernels' own assembly.

@pytest.mark.parametrize("name", ["kernels_tree_f16", "kernels_tree_bf16", "kernels_tree_f32", "kernels_tree_join", "kernels_accept",
                                  "kernels_select", "kernels_mass_f16", "kernels_mass_bf16", "kernels_mass_f32"])
def test_own_assembly(name):
    """No packed binary32 arithmetic, products on matrix instructions, no scratch memory: but for a few
    registers' worth in attention for trees."""
    import subprocess
    B = build_module()
    src, path = "serving/%s.hip" % name, os.path.join(B.BUILD, name + ".s")
    folder = os.path.join(B.CSRC, "serving")
    newest = max(os.path.getmtime(os.path.join(folder, f)) for f in os.listdir(folder))
    if not os.path.exists(path) or os.path.getmtime(path) < newest:
        os.makedirs(B.BUILD, exist_ok=True)
        subprocess.run([B.HIPCC, *B.FLAGS, *B.FILE_FLAGS.get(src, []), "-x", "hip", "--offload-device-only", "-S",
                        os.path.join(B.CSRC, src), "-o", path], check=True, capture_output=True)
    text = open(path).read()
    sizes = [int(s) for s in re.findall(r"\.private_segment_fixed_size:\s+(\d+)", text)]
    assert sizes and max(sizes) <= (96 if name in ("kernels_tree_f16", "kernels_tree_bf16", "kernels_tree_f32") else 0)
    assert not re.search(r"v_pk_(add|mul|fma)_f32", text)
    kind = {"f16": "16x16x32_f16", "bf16": "16x16x32_bf16", "f32": "16x16x4_f32"}.get(name.rsplit("_", 1)[1])
    if kind:
        assert text.count("v_mfma_f32_" + kind) > 50
