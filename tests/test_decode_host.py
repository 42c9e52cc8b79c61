"""The parts of decode.py that need no GPU."""
import random

import pytest
import torch

from elementwise_tensor_commands_amd.decode import Decoder, merge_alike, tree_depths

I32 = torch.int32


def plain(parents):
    """(parents, depths) by walking up from every token; depths of padding: None."""
    out, depths = [], []
    for i, p in enumerate(parents):
        if p == -1 or (0 <= p < i and depths[p] is not None):
            out.append(p)
            depths.append(0 if p == -1 else depths[p] + 1)
        else:
            out.append(-2)
            depths.append(None)
    return out, depths


def test_depths_of_a_tree_by_hand():
    parent, depth = tree_depths(torch.tensor([[-1, 0, 0, 1, 3, 4, -2, 6, 6]], dtype=I32))
    assert parent.tolist() == [[-1, 0, 0, 1, 3, 4, -2, -2, -2]] and parent.dtype == I32
    assert depth[0, :6].tolist() == [0, 1, 1, 2, 3, 4] and depth.dtype == I32


@pytest.mark.parametrize("bad", [0, 1, 4, 2 ** 31 - 1, -2, -3, -2 ** 31])
def test_a_parent_that_is_no_token_before_it_is_padding(bad):
    """Of token i: i + 0, i + 1, ..., past the tree, or negative; and what is below it."""
    for i in range(5):
        row = [-1, 0, 1, 0, 3]
        row[i] = min(i + bad, 2 ** 31 - 1) if bad >= 0 else bad
        want, depths = plain(row)
        parent, depth = tree_depths(torch.tensor([[-1, 0, 1, 0, 3], row], dtype=I32))
        assert parent.tolist() == [[-1, 0, 1, 0, 3], want]
        assert [d for d, x in zip(depth[1].tolist(), depths) if x is not None] == [x for x in depths if x is not None]


@pytest.mark.parametrize("t", [1, 2, 3, 8, 65, 256])
def test_depths_of_any_trees(t):
    rng = random.Random(t)
    rows = [[i - 1 for i in range(t)]]                              # a chain
    for _ in range(40):
        rows.append([rng.choice([-1, i - 1, i - 1, i - 1, rng.randrange(max(1, i)), rng.choice([i, i + 3, t, 2 ** 31 - 1, -2, -7])])
                     if i else -1 for i in range(t)])
    parent, depth = tree_depths(torch.tensor(rows, dtype=I32))
    for r, row in enumerate(rows):
        want, depths = plain(row)
        assert parent[r].tolist() == want
        assert all(x is None or int(depth[r, i]) == x for i, x in enumerate(depths))


def test_guesses_that_begin_alike_are_merged_by_hand():
    # 0 -> 1 -> 2 and 0 -> 3 -> 4, tokens 1 and 3 the same: 4 follows 1
    tokens = torch.tensor([[9, 5, 6, 5, 7], [9, 5, 6, 5, 6], [9, 5, 6, 4, 6]], dtype=I32)
    parent = torch.tensor([[-1, 0, 1, 0, 3]] * 3, dtype=I32)
    got = merge_alike(tokens, parent)
    assert got.tolist() == [[-1, 0, 1, -2, 1], [-1, 0, 1, -2, -2], [-1, 0, 1, 0, 3]] and got.dtype == I32


@pytest.mark.parametrize("t", [1, 2, 5, 17, 64, 200])
def test_merged_guesses(t):
    """Against the paths themselves: each once, by the first token that ends it, its parent the path one shorter."""
    rng = random.Random(t)
    for words in (1, 2, 5):
        rows = [[i - 1 for i in range(t)]] + [[rng.choice([i - 1, rng.randrange(max(1, i)), rng.randrange(max(1, i)), -1, -2 if rng.random() < 0.3 else 0])
                                               if i else -1 for i in range(t)] for _ in range(15)]
        parent, _ = tree_depths(torch.tensor(rows, dtype=I32))
        tokens = torch.tensor([[rng.randrange(words) for _ in range(t)] for _ in rows], dtype=I32)
        got = merge_alike(tokens, parent)
        for r in range(len(rows)):
            paths, ends = [], {}
            for i, p in enumerate(parent[r].tolist()):
                path = None if p == -2 else ((paths[p] if p >= 0 else ()) + (int(tokens[r, i]),))
                paths.append(path)
                first = ends.setdefault(path, i)
                want = -2 if path is None or first != i else ends[path[:-1]] if p >= 0 else -1
                assert int(got[r, i]) == want, (r, i)


def test_no_trees():
    for shape in ((0, 5), (3, 0)):
        parent, depth = tree_depths(torch.zeros(shape, dtype=I32))
        assert parent.shape == depth.shape == shape
        assert merge_alike(torch.zeros(shape, dtype=I32), parent).shape == shape


def test_refused_kinds_of_steps():
    """Before anything is launched: pages that are not read get no weight, and what a decoder does not keep up."""
    args = [torch.zeros(3, dtype=torch.int64), torch.arange(3, dtype=I32), torch.ones(3, dtype=I32)]
    budget = torch.full((3,), 2, dtype=I32)
    for select in (False, True):
        for weigh in (False, True):
            m = Decoder(rows=3, n=8, cols=4, device="cpu", select=select, weigh=weigh)
            for how, fine in ((dict(take=2, budget=budget), False), (dict(take=2), select), (dict(budget=budget), weigh)):
                if not fine:
                    with pytest.raises(ValueError):
                        m.decode(*args, **how)
            assert m.cache.lens.tolist() == [0, 0, 0]
        with pytest.raises(ValueError):
            m.decode(*args, take=-1)


def test_refused_trees():
    """Before the tables change: trees that the operators refuse."""
    m = Decoder(rows=3, n=8, cols=4, device="cpu")
    for shape, like in (((3, 257), None), ((2, 4), None), ((4, 4), None), ((3, 4), (3, 5)), ((3, 4), (2, 4))):
        with pytest.raises((ValueError, RuntimeError)):
            m.verify(torch.zeros(shape, dtype=I32), torch.zeros(like or shape, dtype=I32) - 1, torch.ones(3, dtype=I32))
    assert m.cache.lens.tolist() == [0, 0, 0] and bool((m.cache.pages == -1).all())
