"""Corners of the row operators' C ABI that need no GPU."""
import pytest

import fp8_grouped_gemm_amd as moe
from test_ops_abi import BF16, F32, GRAD, INV, OK, call


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_of_empty_batches_are_no_ops(dtype):
    # an empty output has no address: torch's empty tensors pass null
    base = {**GRAD, "dtype": dtype}
    none = dict(dy=0, yp=0, row_src=0, src_row=0, topk_w=0, dyp=0, dw=0)
    assert call("moe_unpermute_bwd", base, T=0, R=0, **none) == OK
    assert call("moe_unpermute_bwd", base, T=0, R=0, **{**none, "used": 0}) == OK
    assert call("moe_unpermute_bwd", base, T=0, dy=0, src_row=0, topk_w=0, dyp=0, dw=0) == OK
    assert call("moe_unpermute_bwd", base, R=0, yp=0, row_src=0, dyp=0, dw=0) == OK
    # outputs that have elements: one of them at least, as before
    assert call("moe_unpermute_bwd", base, dyp=0, dw=0) == INV
    # what else is wrong with an empty call is still refused
    for bad in (dict(T=0, R=-1), dict(T=-1, R=0), dict(T=0, R=0, width=0), dict(T=0, R=0, dy_ld=8),
                dict(T=0, R=0, dtype=7)):
        assert call("moe_unpermute_bwd", base, **{**none, **bad}) == INV, bad


def test_tiles_of_dense_calls_whose_weights_stream():
    # measured points: the best kernel, or within 10 % of it
    for rows, n, k, tile in ((1, 16384, 9216, (32, 64)), (32, 16384, 9216, (32, 64)), (96, 16384, 9216, (64, 128)),
                             (96, 12288, 16384, (64, 128)), (64, 32768, 8192, (64, 128)), (48, 20480, 14336, (64, 128)),
                             (1, 32768, 8192, (32, 128)), (1, 131072, 2048, (32, 128)), (16, 40960, 4096, (32, 128)),
                             (128, 32768, 8192, (128, 128)), (128, 151936, 4096, (128, 128))):
        assert tuple(moe.moe_gemm_mxfp4_info(rows, n, k).values()) == tile, (rows, n, k)
