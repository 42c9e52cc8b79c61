"""Attention for trees of more rows than one wave deals out, of more than the dealing holds, and of
heads of every width's instance."""
import math
import random

import pytest
import torch

import cache_oracle as C
import elementwise_tensor_commands_amd as E
from test_gpu_cache_ops import tree_state
from test_gpu_serving import DT, ints, within

pytestmark = pytest.mark.gpu


def check(case, dtype, seed, lens=None):
    q, (kg, vg), (kc, vc), pages, own, parent, window = tree_state(case, dtype, seed)
    lens = own if lens is None else lens
    want, want_lse, eo, el = C.tree(q, kc, vc, pages, lens, parent, 1.0 / math.sqrt(q.shape[3]), window)
    out, lse = torch.full(want.shape, 7.0, dtype=DT[dtype], device="cuda"), torch.full(want_lse.shape, 7.0, device="cuda")
    args = [q.cuda(), kg, vg, pages.cuda(), lens.cuda(), parent.cuda(), out]
    size = E.tree_attention_workspace(*args, window=window)
    work = torch.full((max(size, 16),), 255, dtype=torch.uint8, device="cuda")
    E.tree_attention(*args, lse=lse, window=window, workspace=work)
    within(out, want, eo, case)
    within(lse, want_lse, el, case)
    return size


@pytest.mark.parametrize("case", [
    (2, 7, 2, 2, 96, 64, 16, 9, 0), (2, 7, 2, 1, 96, 32, 16, 9, 20), (1, 9, 3, 1, 90, 64, 16, 12, 0), (2, 6, 2, 2, 128, 64, 16, 9, 0),
    (2, 6, 4, 2, 128, 7, 16, 9, 0), (1, 12, 2, 2, 112, 50, 7, 20, 33), (2, 5, 2, 1, 64, 128, 16, 9, 0), (1, 8, 2, 2, 50, 100, 16, 12, 0),
    (2, 7, 4, 4, 80, 128, 16, 9, 0), (3, 4, 2, 1, 75, 65, 16, 9, 9), (1, 70, 1, 1, 65, 64, 16, 12, 0), (1, 70, 1, 1, 97, 64, 16, 12, 0),
])
def test_heads_of_other_widths(case):
    check(case, "f32", sum(case))


def spread(rng, b, cols, page, t):
    """Mostly short rows, some empty, some of no length, a few long, a few past the table."""
    held = cols * page
    return ints([rng.choice([0, -1, rng.randint(0, 40), rng.randint(0, 40), rng.randint(0, held)] + [held - t, held, held + 3] * (r % 16 == 3))
                 for r in range(b)])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", [
    # past 64 rows the work-group deals them together; past 256 in several turns
    (65, 3, 4, 2, 32, 32, 16, 60, 0), (100, 3, 2, 1, 64, 64, 16, 60, 50), (130, 5, 1, 1, 40, 24, 16, 60, 0), (300, 2, 2, 1, 16, 16, 16, 60, 0),
    (100, 20, 1, 1, 64, 64, 16, 60, 0), (70, 18, 4, 2, 64, 32, 16, 60, 100), (257, 20, 1, 1, 16, 16, 8, 110, 0),
    (90, 3, 2, 1, 64, 64, 16, 60, 300), (80, 18, 4, 2, 64, 32, 16, 60, 310),
    # as many as are dealt, and more: each row a work-group's
    (1024, 1, 2, 1, 16, 8, 16, 60, 0), (1025, 1, 2, 1, 16, 8, 16, 60, 0), (1030, 17, 1, 1, 8, 8, 16, 52, 20),
])
def test_many_rows(case, dtype):
    b, t, hq, hk, d, dv, page, cols, window = case
    size = check(case, dtype, 6 * sum(case), spread(random.Random(sum(case)), b, cols, page, t))
    if window == 0:                                                 # (a short window goes without dealing)
        assert (size > 0) == (b <= 1024)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", [(65, 2, 2, 1, 16, 16, 16, 60, 0), (140, 2, 1, 1, 16, 16, 16, 60, 0), (300, 1, 1, 1, 16, 16, 16, 60, 0),
                                  (140, 20, 1, 1, 16, 16, 16, 60, 0)])
def test_many_rows_of_nearly_one_length(case, dtype):
    """Runs that are whole rows."""
    b, t, page, cols = case[0], case[1], case[6], case[7]
    rng = random.Random(b)
    check(case, dtype, 6 * sum(case), ints([cols * page - t - rng.randint(0, 60) for _ in range(b)]))
