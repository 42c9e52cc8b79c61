"""Attention for trees of heads of every width's instance."""
import math

import pytest
import torch

import cache_oracle as C
import elementwise_tensor_commands_amd as E
from test_gpu_cache_ops import tree_state
from test_gpu_serving import DT, within

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
