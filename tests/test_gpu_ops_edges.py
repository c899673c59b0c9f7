"""Corners of the row operators on the GPU: empty batches, the largest
launches, absent lists, tensors autograd knows."""
import pytest
import torch

import fp8_grouped_gemm_amd as moe
from parity_util import say

pytestmark = pytest.mark.gpu


def empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_a_training_step_on_an_empty_batch(dtype):
    # a rank that received no token, its pool empty (alignment 1) or all padding
    W, offsets = 40, ints(0, 0, 0)
    for R in (0, 6):
        say(f"empty batch, {R} pool rows, {dtype}")
        row_src, src_row = ints(*[-1] * R), ints()
        x, w = empty(0, W, dtype=dtype), empty(0, 2)
        xp = moe.moe_permute(x, row_src, src_row, offsets)
        y = moe.moe_unpermute(xp, src_row, 0, w)
        assert xp.shape == (R, W) and y.shape == (0, W)
        for need in ((True, True), (True, False), (False, True)):
            yp = xp if need[1] else None
            dyp, dw = moe.moe_unpermute_bwd(y, yp, row_src, src_row, offsets, w, need_dyp=need[0], need_dw=need[1])
            assert (dyp.shape == (R, W) and dyp.dtype is dtype) if need[0] else dyp is None
            assert dw.shape == w.shape if need[1] else dw is None
        assert moe.moe_permute_bwd(xp, src_row, 0).shape == (0, W)
        with pytest.raises(moe.MoEError):                     # nothing asked for
            moe.moe_unpermute_bwd(y, xp, row_src, src_row, offsets, w, need_dyp=False, need_dw=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_every_slot_masked_and_an_empty_pool(dtype):
    T, K, W = 5, 2, 24
    say(f"no routed slot, {dtype}")
    none, src_row = ints(), ints(*[-1] * (T * K))
    dy, pool = torch.randn(T, W, device="cuda").to(dtype), empty(0, W, dtype=dtype)
    offsets = ints(0, 0)
    dyp, dw = moe.moe_unpermute_bwd(dy, pool, none, src_row, offsets)
    assert dyp.shape == (0, W) and dw.shape == (T, K) and torch.all(dw == 0)
    dyp, dw = moe.moe_unpermute_bwd(dy, None, none, src_row, offsets, need_dw=False)
    assert dyp.shape == (0, W) and dw is None
    dyp, dw = moe.moe_unpermute_bwd(dy, pool, none, src_row, offsets, need_dyp=False)
    assert dyp is None and torch.all(dw == 0)
