"""How far attention for trees holds a weight from what it is: sums in which everything else
cancels, against the exact result within what include/ecmd_serving.h says."""
import math

import pytest
import torch

import elementwise_tensor_commands_amd as E
from test_gpu_serving import DT, I32

pytestmark = pytest.mark.gpu

# Of the weight: half a step of the rest's last place, and the 2^-23 by which it is made larger.
SPLIT = {"bf16": 1.01 * 2.0 ** -16, "f16": 2.0 ** -21, "f32": 0.0}


@pytest.mark.parametrize("t", [1, 80])                              # straight to registers, and staged
@pytest.mark.parametrize("dtype", list(DT))
def test_weights_are_held_to_half_a_step_of_their_rest(dtype, t):
    """Every token attends to three positions: one of weight w and value 1, itself, of weight 1 and
    value -1/2, and one of weight 1 whose value is w - 1/2 rounded to the type, negated.  What is left is
    far below the weight's last places.  w lies a little above 1/2, where those are the largest part
    of it, at as many places between as there are rows."""
    dt, b, d, page = DT[dtype], 200, 8, 4
    first = {"bf16": 2.0 ** -9, "f16": 2.0 ** -12, "f32": 2.0 ** -12}[dtype]     # the rest's largest: a step of the leading part
    want = 0.5 + first * (1 + torch.arange(b, dtype=torch.float64) / b)
    x = want.log()
    k, v = torch.zeros(b, page * 32, 1, d, dtype=dt), torch.zeros(b, page * 32, 1, d, dtype=dt)
    left = x
    for e in range(4):                                              # a score as the sum of a few elements
        k[:, 0, 0, e] = left.to(dt)
        left = left - k[:, 0, 0, e].double()
    w = k[:, 0, 0].double().sum(-1).exp()
    assert float((w - want).abs().max()) < 2.0 ** -20
    v[:, 0, 0, 0] = 1.0
    v[:, 1, 0, 0] = -(w - 0.5).to(dt)
    v[:, 2:, 0, 0] = -0.5                                           # all of the tokens
    exact = (w - 0.5 + v[:, 1, 0, 0].double()) / (2.0 + w)
    pages = torch.arange(b * 32, dtype=I32).view(b, 32)
    q = torch.zeros(b, t, 1, d, dtype=dt)
    q[..., :4] = 1.0
    out = torch.empty(b, t, 1, d, dtype=dt, device="cuda")
    paged = lambda c: c.view(b * 32, page, 1, d).cuda()
    E.tree_attention(q.cuda(), paged(k), paged(v), pages.cuda(), torch.full((b,), 2, dtype=I32, device="cuda"),
                     torch.full((b, t), -1, dtype=I32, device="cuda"), out, scale=1.0)
    got = out[..., 0, 0].cpu().double()
    # w: its score in base 2 (three roundings of a number near 1), exp2 within 2^-23, so within 2^-22; the other
    # two weights: 2^-23 and half as much; the sum of three products below 1: three roundings
    off = (w * (SPLIT[dtype] + 2.0 ** -22) + 1.5 * 2.0 ** -23 + 3 * 2.0 ** -24) / (2.0 + w)
    off = off + exact.abs() * torch.finfo(dt).eps + 2.0 ** -25
    worst = ((got - exact[:, None]).abs() / off[:, None]).max()
    assert float(worst) <= 1.0, float(worst)
    assert bool((out[..., 1:] == 0).all())


@pytest.mark.parametrize("length", [2, 100])                        # at the tree's end, and in a tile that all see all of
@pytest.mark.parametrize("dtype,t", [("bf16", 2), ("bf16", 20), ("bf16", 80), ("f16", 2), ("f16", 80), ("f32", 20)])
def test_an_infinite_value_with_a_weight_of_any_last_bits(dtype, t, length):
    """The parts of a weight are positive, whatever its last bits, down to 2^-90 of the row's largest: an
    infinity of either sign stays one."""
    dt, b, d, page, cols = DT[dtype], 64, 8, 4, 64
    k, v = torch.zeros(b, cols * page, 1, d, dtype=dt), torch.ones(b, cols * page, 1, d, dtype=dt)
    k[:, 0, 0, 0] = -torch.arange(b, dtype=torch.float32).to(dt) * (31 / 32)           # to exp(-61.03), 2^-88.05
    v[:, 0, 0, 1], v[:, 0, 0, 2] = math.inf, -math.inf
    q = torch.ones(b, t, 1, d, dtype=dt)
    out = torch.empty(b, t, 1, d, dtype=dt, device="cuda")
    paged = lambda c: c.view(b * cols, page, 1, d).cuda()
    E.tree_attention(q.cuda(), paged(k), paged(v), torch.arange(b * cols, dtype=I32).view(b, cols).cuda(),
                     torch.full((b,), length, dtype=I32, device="cuda"), torch.full((b, t), -1, dtype=I32, device="cuda"), out, scale=1.0)
    assert bool((out[..., 1] == math.inf).all() and (out[..., 2] == -math.inf).all())
    # all other values are 1: off by the weights' parts and the sums of 102 of them, below half a step of 16 bits
    assert float((out[..., [0, 3]].float() - 1).abs().max()) <= (2.0 ** -23 * 110 if dtype == "f32" else 0.0)
