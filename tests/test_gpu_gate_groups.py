"""moe_gate's groups on the GPU against the plain float64 form: sums whose errors differ from
group to group, and 16-bit logits."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_amd as moe
import layer_util as lu
from parity_util import say

pytestmark = pytest.mark.gpu


def choose(l, K, bias, sigmoid, groups, top_groups, group_top):
    """The library's choice, which has to be that of the plain form."""
    got = moe.moe_gate(l.cuda(), K, bias=None if bias is None else bias.cuda(),
                       score=moe.MOE_SCORE_SIGMOID if sigmoid else moe.MOE_SCORE_SOFTMAX, groups=groups,
                       top_groups=top_groups, group_top=group_top)[0].cpu().numpy()
    want = lu.gate(lu.f64(l), K, None if bias is None else lu.f64(bias), None, sigmoid, groups, top_groups, group_top,
                   True, 1.0)[0]
    assert np.array_equal(got, want), (groups, top_groups, group_top, np.nonzero((got != want).any(1))[0][:8])
    return got


def logit(s):
    s = torch.tensor(s, dtype=torch.float64)
    return torch.log(s / (1 - s)).float()


def test_a_cancelling_group_beside_ordinary_ones():
    # next to 2^20 float32 does not see group 0's scores: its sum, .09, is the largest, in float32 0
    say("gate: one group's biases cancel")
    l = logit([[.06, .03, .05, .03, .035, .025, .03, .02]])
    bias = torch.zeros(8)
    bias[0], bias[1] = 2.0 ** 20, -2.0 ** 20
    assert choose(l, 2, bias, True, 4, 2, 2).tolist() == [[0, 2]]
    # and a group that float32 puts too high: .035 - 2^20 is rounded to 1/16 - 2^20, so .04 counts as .0625
    l = logit([[.005, .035, .035, .025, .03, .02, .03, .015]])
    assert choose(l, 2, bias, True, 4, 2, 2).tolist() == [[2, 4]]


def test_a_cancelling_group_of_many():
    say("gate: one group of 20 and of 40 cancels")
    for groups in (20, 40):
        s = np.tile([.03, .02], groups) + np.arange(2 * groups) * 1e-4
        s[:2] = .06, .03
        bias = torch.zeros(2 * groups)
        bias[0], bias[1] = 2.0 ** 20, -2.0 ** 20
        got = choose(logit(s[None]), 3, bias, True, groups, 3, 2)
        assert got[0, 0] == 0


# (experts, groups): 1, 2, 4, 6, 8, 16 and up to 32 experts a lane, a group in 1 to 32 lanes, up to 16 groups and more
LAYOUTS = [(64, 16), (64, 2), (128, 32), (128, 4), (256, 16), (256, 64), (384, 16), (512, 8), (512, 64), (640, 16),
           (1000, 10), (1000, 40), (1023, 33), (1024, 2), (1024, 64)]


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [2, 3, 4])
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
def test_groups_that_cancel_by_different_amounts(layout, group_top, sigmoid):
    # of every second group the best are a bias of up to 2^20, its negative and experts without one: float32 has
    # a group's sum right to anything from 2^-24 to 1/8
    E, groups = layout
    size, T = E // groups, 24
    say(f"gate: {E} experts in {groups} groups of different magnitudes, {group_top} best")
    rng = np.random.default_rng(E + 31 * groups + group_top)
    l = torch.from_numpy(2 * rng.standard_normal((T, E))).float()
    b = np.zeros((groups, size))
    for g in range(0, groups, 2):
        m = 2.0 ** rng.integers(0, 21)
        b[g, group_top:] = -4 * m                              # not among the best
        at = rng.permutation(group_top)
        b[g, at[0]], b[g, at[1]] = m, -m
    bias = torch.from_numpy(b.reshape(-1)).float()
    for top_groups in (max(1, groups // 4), max(1, groups // 2)):
        choose(l, min(8, size * top_groups), bias, sigmoid, groups, top_groups, group_top)


def distinct(T, E, dtype, rng):
    """[T, E] logits of a 16-bit type, distinct within a token and none the negative of another (so that no two
    sums of sigmoids are equal by symmetry): every fourth value of the type from 2^-3 on, half of them negated."""
    first = torch.tensor([0.125], dtype=dtype).view(torch.int16).item()
    v = (first + 4 * torch.arange(E)).to(torch.int16).view(dtype) if dtype is torch.float16 else \
        (first + torch.arange(E)).to(torch.int16).view(dtype)
    assert v.float().unique().numel() == E and v.max() < 60
    sign = torch.from_numpy(rng.choice([-1.0, 1.0], E)).to(dtype)
    return torch.stack([(v * sign)[torch.from_numpy(rng.permutation(E))] for _ in range(T)])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", [(64, 8, 4, 2), (65, 13, 3, 5), (160, 8, 3, 3), (256, 8, 4, 2), (384, 64, 9, 2),
                                    (512, 4, 1, 100), (1000, 10, 5, 2), (1024, 64, 20, 16)], ids=str)
def test_16_bit_logits_whose_groups_are_sums(layout, dtype):
    E, groups, top_groups, group_top = layout
    say(f"gate: {dtype} logits, sums of {group_top}")
    rng = np.random.default_rng(E + groups)
    l = distinct(30, E, lu.DT[dtype], rng)
    bias = torch.from_numpy(0.3 * rng.standard_normal(E)).float()
    for sigmoid in (False, True):
        for b in (None, bias):
            choose(l, min(8, E // groups * top_groups), b, sigmoid, groups, top_groups, group_top)
