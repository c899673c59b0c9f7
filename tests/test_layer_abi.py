"""The C ABI of the operators around the experts' products (moe_gate, moe_rms_norm,
moe_swiglu and their gradients, moe_gemm_wgrad): every invalid call is refused on the host (CPU
only: each call fails its checks before the device is queried, or is a no-op)."""
import ctypes

import pytest
import torch

import fp8_grouped_gemm_amd as moe
from fp8_grouped_gemm_amd import ops

X, Y, Z, V, W, U = (0x10000000 * i for i in range(1, 7))  # never dereferenced
P = ctypes.c_void_p
INV, SHAPE, SMALL, OK = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE, moe.MOE_ERR_WORKSPACE_TOO_SMALL,
                         moe.MOE_OK)
BF16, F16, F32, U8 = range(4)

GATE = dict(T=4, E=64, K=4, dtype=BF16, p_logits=X, ld=0, p_bias=Y, p_mask=Z, score=0, groups=8, top_groups=2,
            group_top=2, renorm=1, scale=1.0, p_idx=V, p_w=W, p_stream=0)
GATE_BWD = dict(T=4, E=64, K=4, dtype=BF16, p_logits=X, ld=0, p_idx=Y, p_dw=Z, score=1, renorm=1, scale=1.0,
                p_out=V, out_ld=0, p_stream=0)
NORM = dict(rows=4, width=256, dtype=BF16, p_x=X, x_ld=0, p_res=Y, res_ld=0, p_weight=Z, w_dtype=F32, eps=1e-6,
            p_z=V, z_ld=0, p_rstd=V + 8192, p_y=W, y_ld=0, p_codes=U, p_sf=U + 4096, fmt=0, p_stream=0)
NORM_BWD = dict(rows=4, width=256, dtype=BF16, p_dy=X, dy_ld=0, p_z=Y, z_ld=0, p_weight=Z, w_dtype=BF16, p_rstd=V,
                p_dz=V + 4096, dz_ld=0, p_dx=W, dx_ld=0, p_dw=W + 8192, p_ws=U, ws_bytes=256 * 4, p_stream=0)
SWIGLU = dict(R=4, inner=128, dtype=BF16, p_gu=X, gu_ld=0, clamp=0.0, p_row_src=Y, p_used=Y + 4096, p_h=Z, h_ld=0,
              p_hc=V, p_hsf=V + 4096, p_gc=W, p_gsf=W + 4096, fmt=0, p_stream=0)
SWIGLU_BWD = dict(R=4, inner=128, dtype=BF16, p_dh=X, dh_ld=0, p_gu=0, gu_ld=0, p_gc=Y, p_gsf=Y + 4096, fmt=0,
                  clamp=0.0, p_row_src=Z, p_used=Z + 4096, p_dgu=V, dgu_ld=0, p_stream=0)

WGRAD = dict(groups=2, rows=64, n=48, k=128, dtype=BF16, p_dy=X, dy_ld=0, p_x=Y, p_sf=Z, fmt=0, p_off=V, p_counts=V + 64,
             accumulate=0, p_dw=W, dw_dtype=F32, p_ws=U, ws_bytes=0, p_stream=0)


def call(name, base, **change):
    a = {**base, **change}
    return getattr(ops.ops_lib(), name)(*[(P(v) if v else None) if k.startswith("p_") else v for k, v in a.items()])


@pytest.mark.parametrize("name,base,changes", [
    ("moe_gate", GATE, [
        (dict(T=-1), INV), (dict(E=0), INV), (dict(K=0), INV), (dict(K=65, E=64), INV), (dict(dtype=U8), INV),
        (dict(dtype=-1), INV), (dict(score=2), INV), (dict(score=-1), INV), (dict(E=1032, groups=8), SHAPE),
        (dict(E=512, K=65), SHAPE), (dict(T=1 << 28), SHAPE), (dict(groups=0), INV), (dict(groups=7), INV),
        (dict(top_groups=0), INV), (dict(top_groups=9), INV), (dict(group_top=0), INV), (dict(group_top=9), INV),
        (dict(K=17), INV), (dict(groups=1, top_groups=2), INV), (dict(groups=1, top_groups=1, group_top=65), INV),
        (dict(E=130, groups=65, group_top=1), SHAPE), (dict(p_logits=0), INV), (dict(p_idx=0), INV),
        (dict(p_w=0), INV), (dict(p_logits=X + 1), INV), (dict(p_bias=Y + 2), INV), (dict(p_idx=V + 2), INV),
        (dict(p_w=W + 1), INV), (dict(ld=63), INV), (dict(ld=-1), INV), (dict(ld=(1 << 30) + 1), INV),
        (dict(p_idx=X), INV), (dict(p_w=X + 4 * 64 * 2 - 4), INV), (dict(p_w=Y), INV), (dict(p_idx=Z), INV),
        (dict(p_w=V), INV), (dict(p_w=V + 60), INV)]),
    ("moe_gate_bwd", GATE_BWD, [
        (dict(T=-1), INV), (dict(K=0), INV), (dict(dtype=U8), INV), (dict(score=2), INV),
        (dict(E=1025), SHAPE), (dict(E=512, K=65), SHAPE), (dict(p_logits=0), INV), (dict(p_idx=0), INV),
        (dict(p_dw=0), INV), (dict(p_out=0), INV), (dict(ld=63), INV), (dict(out_ld=63), INV),
        (dict(p_out=V + 1), INV), (dict(p_out=X), INV), (dict(p_out=Y), INV), (dict(p_out=Z), INV)]),
    ("moe_rms_norm", NORM, [
        (dict(rows=-1), INV), (dict(width=0), INV), (dict(dtype=U8), INV), (dict(w_dtype=F16), INV),
        (dict(w_dtype=9), INV), (dict(rows=1 << 28), SHAPE), (dict(width=1 << 24, p_codes=0, p_sf=0), SHAPE),
        (dict(width=192), SHAPE), (dict(width=144, fmt=1), SHAPE), (dict(fmt=2), INV), (dict(fmt=-1), INV),
        (dict(p_x=0), INV), (dict(p_y=0, p_codes=0, p_sf=0), INV), (dict(p_codes=0), INV), (dict(p_sf=0), INV),
        (dict(p_res=0), INV), (dict(x_ld=255), INV), (dict(res_ld=255), INV), (dict(z_ld=255), INV),
        (dict(y_ld=-3), INV), (dict(p_x=X + 1), INV), (dict(p_z=V + 1), INV), (dict(p_weight=Z + 2), INV),
        (dict(p_codes=U + 4), INV), (dict(p_sf=U + 4098), INV), (dict(p_rstd=V + 8193), INV),
        (dict(p_z=X + 2), INV), (dict(p_z=X, z_ld=257), INV), (dict(p_y=Y - 2), INV), (dict(p_y=X, p_z=X), INV),
        (dict(p_y=V), INV), (dict(p_rstd=Z), INV), (dict(p_codes=X), INV), (dict(p_sf=U + 1020), INV)]),
    ("moe_rms_norm_bwd", NORM_BWD, [
        (dict(rows=-1), INV), (dict(width=0), INV), (dict(dtype=U8), INV), (dict(w_dtype=F16), INV),
        (dict(rows=1 << 28), SHAPE), (dict(width=1 << 24), SHAPE), (dict(p_dx=0, p_dw=0), INV),
        (dict(p_dy=0), INV), (dict(p_z=0), INV), (dict(p_rstd=0), INV), (dict(p_ws=0), INV),
        (dict(ws_bytes=256 * 4 - 1), SMALL), (dict(p_ws=U + 8), INV), (dict(dy_ld=1), INV), (dict(z_ld=1), INV),
        (dict(dz_ld=1), INV), (dict(dx_ld=1), INV), (dict(p_dx=X, dx_ld=300), INV), (dict(p_dx=Y), INV),
        (dict(p_dx=X + 2), INV), (dict(p_dw=Z), INV), (dict(p_dw=W), INV), (dict(p_ws=X), INV), (dict(p_ws=W), INV),
        (dict(p_dw=W + 8194), INV)]),
    ("moe_swiglu", SWIGLU, [
        (dict(R=-1), INV), (dict(inner=0), INV), (dict(dtype=U8), INV), (dict(R=1 << 28), SHAPE),
        (dict(inner=1 << 23), SHAPE), (dict(inner=96), SHAPE), (dict(inner=48, fmt=1), SHAPE), (dict(fmt=2), INV),
        (dict(p_gu=0), INV), (dict(p_h=0, p_hc=0, p_hsf=0, p_gc=0, p_gsf=0), INV), (dict(p_hc=0), INV),
        (dict(p_hsf=0), INV), (dict(p_gc=0), INV), (dict(p_gsf=0), INV), (dict(gu_ld=255), INV),
        (dict(h_ld=127), INV), (dict(p_gu=X + 1), INV), (dict(p_h=Z + 1), INV), (dict(p_hc=V + 4), INV),
        (dict(p_gsf=W + 4098), INV), (dict(p_row_src=Y + 1), INV), (dict(p_used=Y + 2), INV), (dict(p_h=X), INV),
        (dict(p_hc=X + 8), INV), (dict(p_gc=Y), INV), (dict(p_h=Y + 4096), INV), (dict(p_hc=W), INV),
        (dict(p_gsf=V + 508), INV)]),
    ("moe_swiglu_bwd", SWIGLU_BWD, [
        (dict(R=-1), INV), (dict(inner=0), INV), (dict(dtype=U8), INV), (dict(inner=96), SHAPE), (dict(fmt=7), INV),
        (dict(p_dh=0), INV), (dict(p_dgu=0), INV), (dict(p_gc=0, p_gsf=0), INV), (dict(p_gsf=0), INV),
        (dict(p_gu=W), INV), (dict(dh_ld=127), INV), (dict(dgu_ld=255), INV),
        (dict(p_gu=W, p_gc=0, p_gsf=0, gu_ld=255), INV), (dict(p_gc=Y + 4), INV), (dict(p_dgu=V + 1), INV),
        (dict(p_dgu=X), INV), (dict(p_dgu=Y), INV), (dict(p_dgu=Z), INV),
        (dict(p_gu=V, gu_ld=300, p_gc=0, p_gsf=0), INV), (dict(p_gu=V + 2, p_gc=0, p_gsf=0), INV)]),
    ("moe_gemm_wgrad", WGRAD, [
        (dict(groups=0), INV), (dict(rows=-1), INV), (dict(n=-1), INV), (dict(k=0), INV), (dict(dtype=F32), INV),
        (dict(dtype=U8), INV), (dict(dw_dtype=U8), INV), (dict(dw_dtype=5), INV), (dict(fmt=2), INV),
        (dict(p_off=0), INV), (dict(p_off=0, groups=1), INV), (dict(k=96), SHAPE), (dict(k=48, fmt=1), SHAPE),
        (dict(k=(1 << 20) + 128), SHAPE), (dict(groups=1025), SHAPE), (dict(rows=1 << 28), SHAPE),
        (dict(n=1 << 20), SHAPE), (dict(p_dy=0), INV), (dict(p_x=0), INV), (dict(p_sf=0), INV), (dict(p_dw=0), INV),
        (dict(dy_ld=47), INV), (dict(dy_ld=(1 << 24) + 1), INV), (dict(p_dy=X + 1), INV), (dict(p_x=Y + 8), INV), (dict(p_sf=Z + 2), INV),
        (dict(p_dw=W + 2), INV), (dict(p_off=V + 1), INV), (dict(p_counts=V + 66), INV), (dict(p_ws=U + 8), INV),
        (dict(p_dw=X), INV), (dict(p_dw=Y), INV), (dict(p_dw=Z + 4 * 60), INV), (dict(p_dw=V), INV),
        (dict(p_dw=V + 64), INV),
        (dict(groups=1, p_off=0, p_counts=0, rows=8192, ws_bytes=0), SMALL),
        (dict(groups=1, p_off=0, p_counts=0, rows=8192, p_ws=0, ws_bytes=1 << 30), INV),
        (dict(groups=1, p_off=0, p_counts=0, rows=8192, p_ws=W, ws_bytes=1 << 30), INV)]),
])
def test_refusals(name, base, changes):
    for change, code in changes:
        assert call(name, base, **change) == code, (name, change)


def test_empty_calls_are_no_ops():
    assert call("moe_gate", GATE, T=0, p_logits=0, p_idx=0, p_w=0, p_mask=0) == OK
    assert call("moe_gate_bwd", GATE_BWD, T=0, p_logits=0, p_idx=0, p_dw=0, p_out=0) == OK
    assert call("moe_rms_norm", NORM, rows=0, p_x=0, p_y=0, p_codes=0, p_sf=0) == OK
    assert call("moe_rms_norm_bwd", NORM_BWD, rows=0, p_dw=0, p_dx=0, p_dy=0) == OK
    assert call("moe_rms_norm_bwd", NORM_BWD, rows=0, p_dw=0) == OK
    assert call("moe_swiglu", SWIGLU, R=0, p_gu=0, p_h=0) == OK
    assert call("moe_swiglu_bwd", SWIGLU_BWD, R=0, p_dh=0, p_dgu=0) == OK
    assert call("moe_gemm_wgrad", WGRAD, n=0, p_dw=0) == OK
    assert call("moe_gemm_wgrad", WGRAD, rows=0, accumulate=1, p_dw=0) == OK
    # what else is wrong with an empty call is still refused
    assert call("moe_gate", GATE, T=0, E=0) == INV
    assert call("moe_rms_norm", NORM, rows=0, width=200) == SHAPE
    assert call("moe_swiglu", SWIGLU, R=0, fmt=3) == INV


def test_workspace_query():
    q = moe.moe_rms_norm_bwd_workspace_bytes
    assert q(0, 4096) == 0 and q(1, 100) == 400
    sizes = [q(r, 4096) for r in (1, 2, 100, 1000, 100000, 1 << 27)]
    assert sizes == sorted(sizes) and sizes[-1] < 64 << 20       # bounded, whatever the rows
    for bad, code in (((-1, 4), INV), ((4, 0), INV), ((1 << 28, 4), SHAPE), ((4, 1 << 24), SHAPE)):
        with pytest.raises(moe.MoEError) as e:
            q(*bad)
        assert e.value.code == code
    with pytest.raises(ValueError, match="beyond 32 bits"):
        q((1 << 32) + 4, 4)
    assert ops.ops_lib().moe_rms_norm_bwd_workspace_bytes(4, 4, None) == INV
    # weight gradients: nothing where tiles fill the card, bounded where rows are split
    w = moe.moe_gemm_wgrad_workspace_bytes
    assert w(32, 12288, 4096, 4096) == 0 and w(1, 0, 64, 64) == 0 and w(1, 100000, 0, 64) == 0
    assert 0 < w(1, 1 << 20, 64, 64) <= 64 * 64 * 64 * 4 and w(1, 8192, 384, 7168) <= 16 * 384 * 7168 * 4
    for bad, code in (((0, 4, 4, 32), INV), ((1, 4, 4, 48), SHAPE), ((1025, 4, 4, 32), SHAPE)):
        with pytest.raises(moe.MoEError) as e:
            w(*bad)
        assert e.value.code == code


def test_binding_refuses_host_tensors():
    x, i = torch.zeros(2, 256), torch.zeros(2, 2, dtype=torch.int32)
    for f in (lambda: moe.moe_gate(x, 2), lambda: moe.moe_gate_bwd(x, i, x[:, :2]), lambda: moe.moe_rms_norm(x),
              lambda: moe.moe_rms_norm_bwd(x, x, x[:, 0]), lambda: moe.moe_swiglu(x),
              lambda: moe.moe_swiglu_bwd(x, gu=x),
              lambda: moe.moe_gemm_wgrad(x.half(), x.to(torch.uint8), x[:, :8].to(torch.uint8))):
        with pytest.raises(ValueError, match="expected a GPU"):
            f()
