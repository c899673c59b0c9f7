"""moe_gate and moe_gate_bwd on the GPU against plain float64 forms: the choice
exactly, weights and gradients within the float32 roundings that the forms count."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_amd as moe
import layer_util as lu
import ops_util as ou
from parity_util import say

pytestmark = pytest.mark.gpu

INF = float("inf")
# tokens, experts, top_k, groups, top_groups, group_top
SHAPES = [
    (1, 1, 1, 1, 1, 1), (1, 384, 6, 1, 1, 1), (5, 2, 2, 1, 1, 1), (7, 63, 8, 1, 1, 1), (9, 64, 8, 8, 4, 2),
    (33, 65, 3, 5, 2, 1), (4, 65, 13, 13, 3, 5), (130, 256, 8, 8, 4, 2), (17, 257, 12, 1, 1, 1), (6, 300, 30, 60, 20, 3),
    (64, 384, 6, 64, 9, 2), (3, 512, 64, 4, 1, 100), (10, 1000, 10, 10, 5, 2), (5, 1024, 64, 64, 64, 16),
    (3, 1024, 8, 1, 1, 1), (12, 6, 6, 6, 6, 1), (8, 40, 4, 1, 1, 3), (1025, 16, 2, 4, 1, 1),
]


def draw(shape, dtype, seed=0, masked=True):
    T, E = shape[:2]
    rng = np.random.default_rng(100 * seed + T + 7 * E)
    l = torch.from_numpy(2 * rng.standard_normal((T, E))).to(dtype)
    if masked and T > 2 and E > 1:                            # experts out of the question, and a token with none
        off = rng.random((T, E)) < 0.3
        off[2] = True
        l[torch.from_numpy(off)] = -INF
    bias = torch.from_numpy(0.3 * rng.standard_normal(E)).float()
    mask = torch.from_numpy(rng.random(T) < 0.8)
    return l, bias, mask, rng


def check(l, got, K, bias, mask, sigmoid, groups, top_groups, group_top, renorm, scale):
    l64 = lu.f64(l)
    idx, w = lu.gate(l64, K, None if bias is None else lu.f64(bias), None if mask is None else mask.cpu().numpy(),
                     sigmoid, groups, top_groups, group_top, renorm, scale)
    assert got[0].dtype == torch.int32 and got[1].dtype == torch.float32
    assert np.array_equal(got[0].cpu().numpy(), idx), np.nonzero((got[0].cpu().numpy() != idx).any(1))
    # the score, the chosen ones' sum (6 levels) and quotient, the scale
    steps = lu.gate_steps(l64, l.shape[1]) * 2 + 10
    lu.within(got[1], w, steps * lu.U32 * abs(w) + 2.0 ** -126)


@pytest.mark.parametrize("dtype", list(lu.DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_choice_against_the_plain_form(shape, dtype):
    say(f"gate {shape} {dtype}")
    T, E, K, groups, top_groups, group_top = shape
    l, bias, mask, _ = draw(shape, lu.DT[dtype])
    if dtype != "f32" and group_top > 1:
        # (16-bit logits repeat, and sums of their scores tie in ways float64 does not decide)
        l = draw(shape, torch.float32)[0]
    for sigmoid in (False, True):
        for b in (None, bias):
            for m, renorm, scale in ((None, True, 1.0), (mask, False, 2.5)):
                got = moe.moe_gate(l.cuda(), K, bias=None if b is None else b.cuda(),
                                   mask=None if m is None else m.cuda(),
                                   score=moe.MOE_SCORE_SIGMOID if sigmoid else moe.MOE_SCORE_SOFTMAX,
                                   groups=groups, top_groups=top_groups, group_top=group_top, renorm=renorm, scale=scale)
                check(l, got, K, b, m, sigmoid, groups, top_groups, group_top, renorm, scale)


@pytest.mark.parametrize("run", [1, 2, 4, 6, 8, 16])
def test_groups_of_whole_lanes(run):
    # groups of 1 to 64 lanes' experts, few and many of them
    for lanes in (1, 2, 4, 8, 16, 32):
        groups, E = 64 // lanes, 64 * run
        say(f"gate {E} experts in {groups} groups")
        l, bias, mask, _ = draw((9, E), torch.float32, lanes)
        for group_top in (1, 2):
            top_groups = max(1, groups // 3)
            K = min(5, lanes * run * top_groups)
            if group_top > lanes * run:
                continue
            for sigmoid, b in ((False, bias), (True, bias), (True, None)):
                got = moe.moe_gate(l.cuda(), K, bias=None if b is None else b.cuda(),
                                   score=moe.MOE_SCORE_SIGMOID if sigmoid else moe.MOE_SCORE_SOFTMAX,
                                   groups=groups, top_groups=top_groups, group_top=group_top)
                check(l, got, K, b, None, sigmoid, groups, top_groups, group_top, True, 1.0)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [2, 3])
def test_groups_whose_biases_cancel(group_top, sigmoid):
    # sums of small scores and of biases of both signs, next to which float32 cannot see the scores
    T, E, size = 300, 64, group_top
    groups = E // size
    say(f"gate: {groups} groups of cancelling biases")
    l, _, _, rng = draw((T, groups * size), torch.float32, 7, masked=False)
    bias = torch.tensor([4096.0, -4096.0, 0.0][:size]).repeat(groups)
    got = moe.moe_gate(l.cuda(), 4, bias=bias.cuda(), score=moe.MOE_SCORE_SIGMOID if sigmoid else moe.MOE_SCORE_SOFTMAX,
                       groups=groups, top_groups=max(2, groups // 4), group_top=group_top)
    check(l, got, 4, bias, None, sigmoid, groups, max(2, groups // 4), group_top, True, 1.0)


@pytest.mark.parametrize("K", [2, 3, 4])
def test_near_neighbours_in_every_slot(K):
    # the slots' values but the last two well apart, and these too near for float32, the higher id ahead
    say(f"gate: near neighbours in the last of {K} slots")
    l = torch.full((1, 130), -3.0)
    bias = torch.zeros(130)
    for j in range(K - 2):
        bias[100 + j] = 8192.0 - j
    l[0, 40], l[0, 41] = 1.0, 1.0 + 2.0 ** -12                # scores 2^-14 apart, next to 4096
    bias[40:42] = 4096.0
    want = [100 + j for j in range(K - 2)] + [41, 40]
    for k in (K - 1, K, K + 1):
        idx, _ = moe.moe_gate(l.cuda(), k, bias=bias.cuda(), score=moe.MOE_SCORE_SIGMOID)
        assert idx[0, :K].tolist() == want[:k]


def test_ties_go_to_the_lower_id():
    say("ties")
    T, E = 40, 320
    rng = np.random.default_rng(1)
    l = torch.from_numpy(rng.integers(-2, 3, (T, E))).float()
    l[0] = 0.0
    l[1] = torch.tensor([0.0, -0.0] * (E // 2))               # equal zeros
    l[2] = torch.finfo(torch.float32).min                     # the lowest value is a value, not a mask
    bias = torch.from_numpy(rng.integers(-1, 2, E)).float()
    for sigmoid in (False, True):
        for b in (None, torch.zeros(E), bias):
            for groups, top_groups in ((1, 1), (10, 3)):
                score = moe.MOE_SCORE_SIGMOID if sigmoid else moe.MOE_SCORE_SOFTMAX
                got = moe.moe_gate(l.cuda(), 9, bias=None if b is None else b.cuda(), score=score, groups=groups,
                                   top_groups=top_groups)
                check(l, got, 9, b, None, sigmoid, groups, top_groups, 1, True, 1.0)
    h = l.clamp(min=-60000).half()
    got = moe.moe_gate(h.cuda(), 9)
    check(h, got, 9, None, None, False, 1, 1, 1, True, 1.0)


def test_neighbours_that_float32_scores_cannot_tell_apart():
    # sigmoids 2^-26 apart near 1, and saturated ones: the choice goes by the formula in 64 bits
    say("near neighbours")
    E = 128
    l = torch.linspace(17, 18, E)[torch.randperm(E, generator=torch.Generator().manual_seed(3))].view(1, E)
    l = torch.cat([l, l + 20, -l])
    for b in (None, torch.full((E,), 0.25)):
        got = moe.moe_gate(l.cuda(), 20, bias=None if b is None else b.cuda(), score=moe.MOE_SCORE_SIGMOID)
        idx = lu.gate(lu.f64(l[[0, 2]]), 20, None if b is None else lu.f64(b), None, True, 1, 1, 1, True, 1.0)[0]
        assert np.array_equal(got[0][[0, 2]].cpu().numpy(), idx)
    got = moe.moe_gate(l.cuda(), 20, score=moe.MOE_SCORE_SIGMOID)[0]  # without a bias the logits decide
    assert torch.equal(got[1].cpu(), torch.argsort(l[1], descending=True)[:20].int())


def test_masks_infinities_and_nan():
    say("masks, infinities, NaN")
    E, K, nan = 70, 4, float("nan")
    l = torch.randn(8, E, generator=torch.Generator().manual_seed(5))
    l[0] = -INF
    l[1, 3:] = -INF                                           # fewer experts than slots
    l[2, 50] = INF
    l[3, 60] = nan
    l[3, 4] = -INF
    l[4, 10] = -INF
    bias = torch.zeros(E)
    bias[20] = -INF
    for score in (0, 1):
        for b in (None, bias.cuda()):
            for renorm in (False, True):
                idx, w = (t.cpu() for t in moe.moe_gate(l.cuda(), K, bias=b, score=score, renorm=renorm))
                assert torch.all(idx[0] == -1) and torch.all(w[0] == 0)
                assert set(idx[1, :3].tolist()) == {0, 1, 2} and idx[1, 3] == -1 and w[1, 3] == 0
                assert torch.isfinite(w[[0, 1, 4, 5, 6, 7]]).all()
                assert not (idx[[4, 5, 6, 7]] == 10).all(1).any() and 10 not in idx[4].tolist()
                if b is not None:
                    assert not (idx == 20).any()
                if score == 1:
                    assert idx[2, 0] == 50 and idx[3, 0] == 60 and torch.isnan(w[3, 0])
                    assert torch.isfinite(w[2]).all()
                    assert torch.isnan(w[3]).all() if renorm else torch.isfinite(w[3, 1:]).all()
                else:
                    assert torch.isnan(w[[2, 3]]).all() and 4 not in idx[3].tolist()
                    if b is None:
                        assert idx[2, 0] == 50 and idx[3, 0] == 60
    # a token that is masked out is not read
    idx, w = moe.moe_gate(l.cuda(), K, mask=torch.tensor([1, 1, 0, 0, 1, 1, 1, 1], dtype=torch.uint8).cuda())
    assert torch.all(idx[2:4] == -1) and torch.all(w[2:4] == 0) and torch.isfinite(w).all()


@pytest.mark.parametrize("dtype", list(lu.DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradient_against_the_formula(shape, dtype):
    say(f"gate gradient {shape} {dtype}")
    T, E, K = shape[:3]
    dt = lu.DT[dtype]
    l, _, _, rng = draw(shape, dt)
    idx = torch.from_numpy(np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32))
    drop = torch.from_numpy(rng.random((T, K)) < 0.2)
    idx[drop] = torch.from_numpy(rng.choice([-1, -5, E, 2 ** 31 - 1], int(drop.sum())).astype(np.int32))
    if K > 1:
        idx[0, 1] = idx[0, 0] = E - 1                         # an expert named twice
    if T > 3:
        idx[3] = -1
        l[3] = float("nan")                                   # not read
    dw = torch.from_numpy(rng.standard_normal((T, K))).float()
    dw[(idx < 0) | (idx >= E)] = float("nan")
    if T > 2:                                                 # (a token without experts has no slots either)
        idx[2] = -1
    l64 = lu.f64(l)
    for sigmoid in (False, True):
        for renorm, scale in ((True, 1.0), (False, 1.5)):
            got = moe.moe_gate_bwd(l.cuda(), idx.cuda(), dw.cuda(), score=int(sigmoid), renorm=renorm, scale=scale)
            assert got.dtype == dt
            want, mag = lu.gate_grad(l64, idx.numpy(), lu.f64(dw), sigmoid, renorm, scale)
            # dp: the scores' roundings in its terms and twice in D, a run over the slots; the score; slots that meet
            steps = 4 * lu.gate_steps(l64, E) + 2 * K + 25
            lu.within(got, want, lu.rounded_bound(want, steps * lu.U32 * mag, dt))


def test_gradient_against_differences():
    say("gate gradient by differences")
    T, E, K = 6, 40, 5
    g = torch.Generator().manual_seed(8)
    l, v, dw = (torch.randn(T, n, generator=g) for n in (E, E, K))
    h = 2.0 ** -10
    for score in (0, 1):
        for renorm in (False, True):
            idx, _ = moe.moe_gate(l.cuda(), K, score=score, renorm=renorm)
            d = moe.moe_gate_bwd(l.cuda(), idx, dw.cuda(), score=score, renorm=renorm)
            at = idx.cpu().long()

            def loss(x):
                s = torch.from_numpy(lu.gate_scores(x.numpy(), score == 1)).gather(1, at)
                return ((s / (s.sum(1, keepdim=True) + 1e-20) if renorm else s) * dw.double()).sum().item()

            l2, v2 = l.double(), v.double()
            slope = (loss(l2 + h * v2) - loss(l2 - h * v2)) / (2 * h)
            # third derivatives of the weights are below 6 of the slope's size, h^2 = 2^-20
            size = (d.double().cpu().abs() * v2.abs()).sum().item()
            assert abs((d.double().cpu() * v2).sum().item() - slope) <= 2.0 ** -16 * size


def test_strides_outputs_and_views():
    say("gate strides")
    T, E, K = 37, 100, 7
    l, bias, mask, _ = draw((T, E), torch.bfloat16, 3)
    big = torch.full((T, E + 9), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:, 3:3 + E] = l.cuda()
    view = big[:, 3:3 + E]
    want = moe.moe_gate(l.cuda(), K, bias=bias.cuda())
    idx, w = torch.full((T, K), 77, dtype=torch.int32, device="cuda"), torch.zeros(T, K, device="cuda")
    got = moe.moe_gate(view, K, bias=bias.cuda(), topk_idx=idx, topk_w=w)
    assert got[0] is idx and got[1] is w
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    dw = torch.randn(T, K, device="cuda")
    out = torch.full((T, E + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_gate_bwd(view, idx, dw, out=out[:, 1:1 + E])
    assert torch.equal(out[:, 1:1 + E], moe.moe_gate_bwd(l.cuda(), idx, dw))
    assert torch.all(out[:, :1] == 9) and torch.all(out[:, 1 + E:] == 9)
    one = moe.moe_gate(big[5:6, 3:3 + E], K, bias=bias.cuda())
    assert torch.equal(one[0], want[0][5:6]) and torch.equal(one[1], want[1][5:6])


def test_no_tokens_and_many():
    say("no tokens, many tokens")
    e = torch.empty(0, 48, device="cuda")
    idx, w = moe.moe_gate(e, 4)
    assert idx.shape == (0, 4) and w.shape == (0, 4) and moe.moe_gate_bwd(e, idx, w).shape == (0, 48)
    # 2^32 bytes of logits and more: the last tokens as by themselves
    T, E = (1 << 24) + 5, 130
    l = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    l[-300:].normal_()
    idx, w = moe.moe_gate(l, 3)
    a, b = moe.moe_gate(l[-300:].clone(), 3)
    assert torch.equal(idx[-300:], a) and torch.equal(w[-300:], b)
    assert torch.all(idx[:1000] == torch.arange(3, device="cuda"))
    d = moe.moe_gate_bwd(l, idx, torch.ones_like(w), renorm=False)
    assert torch.equal(d[-300:], moe.moe_gate_bwd(l[-300:].clone(), a, torch.ones_like(b), renorm=False))
    del l, d
    torch.cuda.empty_cache()


def test_binding_refusals():
    l, i, w = torch.randn(6, 32, device="cuda"), torch.zeros(6, 2, dtype=torch.int32, device="cuda"), torch.ones(6, 2, device="cuda")
    leaf = l.clone().requires_grad_()
    bad = [lambda: moe.moe_gate(l.double(), 2), lambda: moe.moe_gate(l.t(), 2), lambda: moe.moe_gate(l[0], 2),
           lambda: moe.moe_gate(l, 2, bias=l[0].half()), lambda: moe.moe_gate(l, 2, bias=l[0, :31]),
           lambda: moe.moe_gate(l, 2, bias=l[0].cpu()), lambda: moe.moe_gate(l, 2, mask=w[:, 0]),
           lambda: moe.moe_gate(l, 2, mask=torch.ones(5, dtype=torch.bool, device="cuda")),
           lambda: moe.moe_gate(l, 2, topk_idx=i.long()), lambda: moe.moe_gate(l, 3, topk_w=w),
           lambda: moe.moe_gate(l, 1 << 32), lambda: moe.moe_gate(leaf, 2), lambda: moe.moe_gate_bwd(leaf, i, w),
           lambda: moe.moe_gate_bwd(l, i, w.clone().requires_grad_()), lambda: moe.moe_gate_bwd(l, i, w, out=leaf),
           lambda: moe.moe_gate_bwd(l, i[:, 0], w), lambda: moe.moe_gate_bwd(l, i, w[:, :1]),
           lambda: moe.moe_gate_bwd(l, i, w, out=l.half())]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: moe.moe_gate(l, 0), lambda: moe.moe_gate(l, -1), lambda: moe.moe_gate(l, 33), lambda: moe.moe_gate(l, 2, groups=5),
              lambda: moe.moe_gate(l, 2, group_top=33), lambda: moe.moe_gate(l, 2, top_groups=2),
              lambda: moe.moe_gate_bwd(l, i, w, out=l)):
        with pytest.raises(moe.MoEError):
            f()
    with torch.no_grad():
        moe.moe_gate(leaf, 2)
