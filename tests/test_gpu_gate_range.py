"""moe_gate and moe_gate_bwd on the GPU at the ends of their ranges: chosen scores whose sum
comes near the 1e-20 that is added to it, and more slots than 31 bits count."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_amd as moe
import layer_util as lu
from parity_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(lu.DT))
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_gradient_of_chosen_scores_next_to_nothing(sigmoid, dtype):
    # a router with a balance bias may choose experts whose own scores are e^-40 to e^-70
    say(f"gate gradient of tiny scores {dtype}")
    T, E, K = 32, 96, 4
    rng = np.random.default_rng(11)
    l = torch.from_numpy(rng.standard_normal((T, E)))
    idx = torch.from_numpy(np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32))
    far = torch.linspace(38, 70, T).double()[:, None].expand(T, K)
    l.scatter_(1, idx.long(), -far + 0.5 * torch.from_numpy(rng.standard_normal((T, K))))
    l = l.to(lu.DT[dtype])
    dw = torch.from_numpy(rng.standard_normal((T, K))).float()
    got = moe.moe_gate_bwd(l.cuda(), idx.cuda(), dw.cuda(), score=int(sigmoid), renorm=True)
    want, mag = lu.gate_grad(lu.f64(l), idx.numpy(), lu.f64(dw), sigmoid, True, 1.0)
    # as for ordinary scores: the scores' roundings in dp's terms and twice in D, a run over the slots, the score
    steps = 4 * lu.gate_steps(lu.f64(l), E) + 2 * K + 25
    lu.within(got, want, lu.rounded_bound(want, steps * lu.U32 * mag, lu.DT[dtype]))


def test_gradient_of_experts_far_below_the_best():
    # logits whose differences are exact, so that no rounding grows with them; beside the best expert the others'
    # terms are too small to count in the sum.  Roundings: exp 4 (2 the hardware's, 2 of its argument's repair), the sum's 3
    # levels of lanes and 3 of rows, its reciprocal 2, their product; the same but for exp, which is 1, of the best
    # expert's score; times dw, and the product
    say("gate gradient of far experts")
    T, E = 500, 64
    g = torch.Generator().manual_seed(2)
    l = -(20 + torch.randint(0, 60 * 64, (T, E), generator=g) / 64.0)
    l[:, 0] = 0
    dw = torch.rand(T, 1, generator=g) + 0.5
    idx = torch.zeros(T, 1, dtype=torch.int32)
    got = moe.moe_gate_bwd(l.cuda(), idx.cuda(), dw.cuda(), renorm=False)
    want, mag = lu.gate_grad(lu.f64(l), idx.numpy(), lu.f64(dw), False, False, 1.0)
    lu.within(got[:, 1:], want[:, 1:], (4 + (6 + 2 + 1) + (6 + 2 + 1) + 2) * lu.U32 * mag[:, 1:])


def test_more_slots_than_31_bits():
    say("gate: 2^31 slots and more")
    T, E, K, n = (1 << 27) + 77, 16, 16, 300
    l = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    l[-n:].normal_()
    idx, w = moe.moe_gate(l, K)
    a, b = moe.moe_gate(l[-n:].clone(), K)
    assert torch.equal(idx[-n:], a) and torch.equal(w[-n:], b)
    assert torch.equal(idx[:n], torch.arange(K, device="cuda", dtype=torch.int32).expand(n, K))
    w[:-n] = 1.0
    w[-n:].normal_()
    d = moe.moe_gate_bwd(l, idx, w, renorm=False)
    assert torch.equal(d[-n:], moe.moe_gate_bwd(l[-n:].clone(), a, w[-n:].clone(), renorm=False))
    del l, d, idx, w
    torch.cuda.empty_cache()


def test_more_slots_than_experts_are_refused_before_they_are_allocated():
    l = torch.zeros(1 << 20, 32, device="cuda")
    with pytest.raises(moe.MoEError):
        moe.moe_gate(l, 1 << 30)                              # (2^52 bytes)
