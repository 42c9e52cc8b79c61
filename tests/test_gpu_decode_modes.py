"""Decoders whose steps are of different kinds: all pages read or some, checked trees, budgets."""
import math

import pytest
import torch

import cache_oracle as C
from elementwise_tensor_commands_amd.decode import Decoder, PagedCache
from test_gpu_decode_cache import CLOSE, KW, PROMPTS, ints, refs_are_the_table_s

pytestmark = pytest.mark.gpu

I32 = torch.int32


def bounds_are_the_keys_s(c, what):
    for layer in range(len(c.k)):
        for r in range(c.rows):
            for j in range(-(-int(c.lens[r]) // c.page)):
                p, n = int(c.pages[r, j]), min(c.page, int(c.lens[r]) - c.page * j)
                if p < 0:
                    continue
                keys = c.k[layer][p, :n]
                assert torch.equal(c.bounds[layer][p, :, 0], keys.amin(0)), (what, layer, r, j)
                assert torch.equal(c.bounds[layer][p, :, 1], keys.amax(0)), (what, layer, r, j)


@pytest.mark.parametrize("weigh", [False, True])
def test_bounds_hold_whatever_the_steps_were(weigh):
    """Steps that read all pages, some, or check a tree, forks, ended rows and packed pages between: a
    page's bounds are those of the keys that it holds."""
    m, plain = (Decoder(n=90, select=x, weigh=weigh, **KW) for x in (True, False))
    for x in (m, plain):
        x.prefill(PROMPTS)
    bounds_are_the_keys_s(m.cache, "prompts")
    g = torch.Generator().manual_seed(3)
    own = [0, 1, 2, 3, 4]
    kinds = ["all", "every", "tree", "every", "fork", "all", "tree", "every", "end", "some", "budget", "tree", "all", "some", "every"]
    for i, kind in enumerate(kinds):
        plan = {"fork": [0, 0, 2, 1, 1], "end": [0, -1, 2, 3, 4]}.get(kind, own)
        alive = ints([int(p >= 0) for p in plan])
        if kind == "tree":
            tokens = torch.randint(0, 61, (5, 6), generator=g).to(I32)
            tokens[:, 1] = 9
            for x in (m, plain):
                x.verify(tokens.cuda(), ints([[-1, 0, 1, 1, 3, 0]] * 5), alive)
        else:
            tokens = torch.randint(0, 61, (5,), generator=g).cuda()
            how = dict(take={"some": 3, "every": 16}.get(kind, 0))
            if kind == "budget" and weigh:
                how = dict(budget=ints([99] * 5))
            a = m.decode(tokens, ints(plan), alive, **how)
            b = plain.decode(tokens, ints(plan), alive)
            if kind != "some" and "some" not in kinds[:i]:
                assert float((a - b).abs().max()) <= CLOSE * float(b.abs().max())
        bounds_are_the_keys_s(m.cache, (i, kind))
        if i == 6:
            m.cache.compact()
            bounds_are_the_keys_s(m.cache, "packed")
        refs_are_the_table_s(m.cache, 90)


def test_pages_are_chosen_by_the_keys_they_hold():
    """After steps that read all pages, the pages taken are those of the definition."""
    m = Decoder(n=90, select=True, **KW)
    m.prefill(PROMPTS)
    g = torch.Generator().manual_seed(8)
    own, ones = ints([0, 1, 2, 3, 4]), torch.ones(5, dtype=I32).cuda()
    step = lambda **how: m.decode(torch.randint(0, 61, (5,), generator=g).cuda(), own, ones, **how)
    for _ in range(17):
        step()
    m.verify(torch.randint(0, 61, (5, 4), generator=g).to(I32).cuda(), ints([[-1, 0, 1, 2]] * 5), ones)
    seen = []
    attend = m.cache.attend_some

    def noted(layer, q, out, since, take):
        attend(layer, q, out, since, take)
        seen.append((layer, q.clone(), out.clone()))

    m.cache.attend_some = noted
    step(take=3)
    c = m.cache
    for layer, q, out in seen:
        k, v = c.k[layer].cpu(), c.v[layer].cpu()
        bounds = torch.zeros(90, 2, 2, 32)
        for r in range(5):
            for j in range(-(-int(c.lens[r]) // 4)):
                keys = k[int(c.pages[r, j]), :min(4, int(c.lens[r]) - 4 * j)]
                bounds[int(c.pages[r, j])] = torch.stack([keys.amin(0), keys.amax(0)], 1)
        pages, lens = C.select(q.cpu(), bounds, c.pages.cpu(), c.lens.cpu(), 4, 3, 1, 1)
        for r in range(5):
            for h in range(2):
                at = [(int(pages[r, h, x // 4]), x % 4) for x in range(int(lens[r, h]))]
                kk, vv = (torch.stack([z[p, s, h] for p, s in at]).double() for z in (k, v))
                want = torch.softmax(q[r, 2 * h:2 * h + 2].cpu().double() @ kk.t() / math.sqrt(32), -1) @ vv
                assert float((out[r, 2 * h:2 * h + 2].cpu() - want).abs().max()) <= CLOSE * float(vv.abs().max()), (layer, r, h)


def test_weights_follow_their_rows():
    """A step's rows take their parents' weights; rows whose parent is none start with none, whatever was there."""
    c = PagedCache(1, 20, 4, 2, 8, 5, 6, weigh=True)
    c.step(ints([-1] * 5), ints([5, 1, 9, 0, 3]))
    c.mass.copy_(torch.arange(30.0).view(5, 6))
    c.mass[4, 2], c.mass[3, 0] = math.inf, math.nan
    was = c.mass.clone()
    c.step(ints([2, -1, 2 ** 31 - 1, 5, 1]), ints([1, 0, 2, 0, -1]))
    assert torch.equal(c.mass, torch.stack([was[2], was[0] * 0, was[0] * 0, was[0] * 0, was[1]]))
    assert c.lens.tolist() == [10, 0, 2, 0, 1]
    refs_are_the_table_s(c, 20)
    c.step(ints([0, 4, -2 ** 31, -7, 4]), ints([0] * 5))
    assert torch.equal(c.mass, torch.stack([was[2], was[1], was[0] * 0, was[0] * 0, was[1]]))
