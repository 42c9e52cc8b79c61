"""page_select on the bounds that page_bounds makes of keys with NaN and infinities: the pages
by the definition in include/ecmd_serving.h, written out."""
import math

import pytest
import torch

import elementwise_tensor_commands_amd as E
from test_gpu_serving import DT, I32, gen, ints, randn

pytestmark = pytest.mark.gpu


def score(q, least, largest):
    """Of query heads q [g, d]; None: no number in every head."""
    best = None
    for row in q.tolist():
        total = 0.0
        for x, lo, hi in zip(row, least.tolist(), largest.tolist()):
            total += x * (lo if x < 0 else hi)
        if not math.isnan(total):
            best = total if best is None else max(best, total)
    return best


@pytest.mark.parametrize("group,d", [(1, 8), (4, 64), (3, 80), (5, 7)])
@pytest.mark.parametrize("dtype", list(DT))
def test_pages_of_no_numbers_come_last(dtype, group, d):
    dt, g = DT[dtype], gen(d + group)
    n, page, hk, take = 24, 4, 2, 15
    k = randn(g, n, page, hk, d, dtype=dt)
    for i in range(0, 6):
        k[i, :, i % 2, i % d] = math.nan                               # in every key: least +inf, largest -inf
    k[6, 1:, 0, 3], k[7, :2] = math.nan, math.nan                      # in some: of no account
    k[8, 2, 1, 2], k[9, :, 0, 1], k[10, 0, :, 4] = math.inf, -math.inf, math.inf
    q = randn(g, 1, group * hk, d, dtype=dt)
    q[0, 0, 0] = q[0, group, 4] = 0.0                                  # of the first head of each: 0 times an infinity
    pages, lens = torch.arange(n, dtype=I32).flip(0).view(1, n), ints([n * page])
    bounds = torch.zeros(n, hk, 2, d, dtype=dt, device="cuda")
    E.page_bounds(k.cuda(), pages.cuda(), lens.cuda(), ints([0]).cuda(), bounds)
    b = bounds.cpu().double()
    assert bool((b[0, 0, 0, 0] == math.inf) & (b[0, 0, 1, 0] == -math.inf)) and not bool(b.isnan().any())
    out, out_lens = torch.empty(1, hk, take, dtype=I32, device="cuda"), torch.empty(1, hk, dtype=I32, device="cuda")
    E.page_select(q.cuda(), bounds, pages.cuda(), lens.cuda(), page, out, out_lens, first=0, last=0)
    for h in range(hk):
        s = [score(q[0, h * group:(h + 1) * group].double(), *b[int(pages[0, c]), h]) for c in range(n)]
        order = sorted(range(n), key=lambda c: (s[c] is None, -(s[c] or 0.0), c))
        assert out[0, h].tolist() == [int(pages[0, c]) for c in sorted(order[:take])], h
        worst = [c for c in range(n) if s[c] is None or s[c] == -math.inf]
        assert len(worst) >= 2 and (len(worst) > n - take or not set(worst) & set(order[:take]))
