"""Decoder.verify with trees, caches and decoders that test_gpu_decode_cache.py does not have."""
import pytest
import torch

from elementwise_tensor_commands_amd.decode import Decoder
from test_gpu_decode_cache import KW, PROMPTS, ints, refs_are_the_table_s

pytestmark = pytest.mark.gpu

I32 = torch.int32


def held(c, r):
    """Keys and values of row r's positions, every layer's."""
    n = int(c.lens[r])
    at = [(int(c.pages[r, i // c.page]), i % c.page) for i in range(n)]
    assert all(p >= 0 for p, _ in at)
    return [torch.stack([z[p, s] for p, s in at]) for z in c.k + c.v] if n else []


def test_any_parent_that_is_no_token_before_it_is_padding():
    """Parents past the tree, of the token itself or far below 0, and tokens below such: as -2."""
    models = [Decoder(n=90, **KW) for _ in range(2)]
    tree = [-1, 0, 0, 1, 2, 3, 4, 5]
    bad = [[7, 8], [2 ** 31 - 1, 6], [3, -2 ** 31], [5, 2 ** 31 - 1], [9, 4]]
    got = []
    for m, odd in zip(models, (True, False)):
        m.prefill(PROMPTS)
        parent = []
        for r in range(5):
            row = list(tree)
            row[3], row[6] = bad[r] if odd else (-2, -2)            # token 5 is below token 3, 7 below 5
            parent.append(row)
        tokens = ints([[11 + r, 3, 5, 7, 9, 11, 13, 15] for r in range(5)])
        got.append(m.verify(tokens, ints(parent), torch.ones(5, dtype=I32).cuda()))
        refs_are_the_table_s(m.cache, 90)
    for a, b in zip(*got):
        assert torch.equal(a, b)
    for r in range(5):
        for a, b in zip(held(models[0].cache, r), held(models[1].cache, r)):
            assert torch.equal(a, b)
