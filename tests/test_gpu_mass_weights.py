"""page_mass where scores and log-sums are large and their differences small: a weight is off by what
the difference is rounded by, not by what the two numbers are."""
import pytest
import torch

import elementwise_tensor_commands_amd as E
from test_gpu_serving import DT, I32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hk,d,page", [(1, 1, 8, 4), (12, 12, 80, 17), (8, 2, 128, 16), (20, 1, 64, 300)])
@pytest.mark.parametrize("dtype", list(DT))
def test_weights_of_scores_near_their_log_sum(dtype, hq, hk, d, page):
    """Every score is a whole number near 200 or -200, every log-sum such a number too: where they are the same a
    weight is 1, and 1 below that it is exp(-1) to within a few of its last places."""
    dt, b, cols = DT[dtype], 2, 3
    n = b * cols
    for big in (200.0, -200.0):
        k = torch.zeros(n, page, hk, d, dtype=dt)
        k[..., 0], k[..., 1] = big, -1.0
        k[:, ::2, :, 1] = 0.0                                       # every other slot: the larger score
        q = torch.zeros(b, hq, d, dtype=dt)
        q[..., :2] = 1.0
        lse = torch.full((b, hq), big)
        pages = torch.arange(n, dtype=I32).view(b, cols)
        mass = torch.zeros(b, cols, device="cuda")
        lens = torch.full((b,), cols * page, dtype=I32)
        E.page_mass(q.cuda(), k.cuda(), pages.cuda(), lens.cuda(), lse.cuda(), mass, mass, scale=1.0)
        ones, less = (page + 1) // 2, page // 2
        want = hq * (ones + less * torch.tensor(-1.0, dtype=torch.float64).exp())
        # exp(-1): its exponent in base 2 rounded once, exp2 within 2^-22; the sums of hq * page numbers
        off = hq * less * 0.37 * (2.0 ** -24 + 2.0 ** -22) + want * (hq * page + 8) * 2.0 ** -24
        assert float((mass.cpu().double() - want).abs().max()) <= off
        # of the larger scores alone nothing is rounded
        k[:, 1::2, :, 1] = -500.0 if big > 0 else -100.0            # (a weight below 2^-140)
        E.page_mass(q.cuda(), k.cuda(), pages.cuda(), lens.cuda(), lse.cuda(), mass, mass, scale=1.0, decay=0.0)
        assert bool((mass == hq * ones).all())
