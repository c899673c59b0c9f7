"""The row operators' C ABI: the library exports what include/moe_ops.h
declares, and every invalid call is refused on the host (CPU only: each call
fails its checks before the device is queried, or is a no-op)."""
import ctypes
import os
import re

import pytest
import torch

import fp8_grouped_gemm_amd as moe
from fp8_grouped_gemm_amd import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_ops.h")

X, Y, Z, V, W = (0x10000000 * i for i in range(1, 6))  # never dereferenced
P = ctypes.c_void_p
INV, SHAPE, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE, moe.MOE_OK
BF16, F16, F32, U8 = range(4)


def test_header_names_and_types():
    text = open(HEADER).read()
    names = re.findall(r"^(?:int)\s+(moe_\w+)\s*\(", text, re.M)
    assert sorted(names) == sorted(ops.EXPORTED_SYMBOLS)
    for n in names:
        assert hasattr(moe.lib(), n)
        assert getattr(moe, n) is getattr(ops, n)
        # the binding passes as many arguments as the header declares
        args = re.search(rf"^int\s+{n}\s*\((.*?)\);", text, re.M | re.S).group(1)
        assert len(getattr(ops.ops_lib(), n).argtypes) == args.count(",") + 1
    for n, v in (("BF16", 0), ("F16", 1), ("F32", 2), ("U8", 3)):
        assert getattr(moe, "MOE_DTYPE_" + n) == v
        assert re.search(rf"#define MOE_DTYPE_{n} {v}\b", text)


def call(name, base, **change):
    """The entry point's code for the valid call `base` with some arguments changed."""
    a = {**base, **change}
    return getattr(ops.ops_lib(), name)(*[P(v) if k in PTRS and v else (None if k in PTRS else v)
                                          for k, v in a.items()])


PTRS = {"x", "row_src", "src_row", "used", "xp", "stream", "dxp", "dx", "yp", "topk_w", "y", "dy",
        "dyp", "dw", "codes", "sf", "a", "a_sf", "b", "b_sf", "offsets", "counts"}
ROWS = dict(T=4, K=2, R=16, width=64, dtype=BF16)
PERMUTE = dict(**ROWS, x=X, x_ld=0, row_src=Y, src_row=Z, used=V, xp=W, xp_ld=0, stream=0)
SUMS = dict(**ROWS, yp=X, yp_ld=0, src_row=Y, topk_w=Z, y=W, y_ld=0, stream=0)
PBWD = {k: v for k, v in SUMS.items() if k != "topk_w"}
GRAD = dict(**ROWS, dy=X, dy_ld=0, yp=Y, yp_ld=0, row_src=Z, src_row=V, used=V + 4096,
            topk_w=V + 8192, dyp=W, dyp_ld=0, dw=W + (1 << 20), stream=0)
QUANT = dict(rows=4, cols=64, dtype=BF16, x=X, x_ld=0, codes=Y, sf=Z, stream=0)
DEQUANT = dict(rows=4, cols=64, dtype=BF16, codes=Y, sf=Z, x=X, x_ld=0, stream=0)
GEMM = dict(groups=2, rows=16, n=32, k=64, dtype=BF16, a=X, a_sf=Y, b=Z, b_sf=V,
            offsets=V + 4096, counts=V + 8192, slots=0, y=W, y_ld=0, stream=0)

BAD_ROWS = [(dict(T=-1), INV), (dict(K=0), INV), (dict(R=-1), INV), (dict(width=0), INV),
            (dict(dtype=4), INV), (dict(dtype=-1), INV), (dict(K=1025), SHAPE),
            (dict(T=1 << 23, K=2), SHAPE), (dict(R=1 << 28), SHAPE), (dict(width=1 << 24), SHAPE),
            (dict(src_row=0), INV), (dict(src_row=Z + 2), INV)]


@pytest.mark.parametrize("name,base,changes", [
    ("moe_permute", PERMUTE, BAD_ROWS + [
        (dict(x=0), INV), (dict(row_src=0), INV), (dict(xp=0), INV), (dict(x=X + 1), INV),
        (dict(xp=W + 1), INV), (dict(x=X + 2, dtype=F32), INV), (dict(used=V + 1), INV),
        (dict(x_ld=63), INV), (dict(xp_ld=-1), INV), (dict(x_ld=(1 << 30) + 1), INV),
        (dict(xp=X), INV), (dict(xp=X + 4 * 64 * 2 - 2), INV), (dict(xp=Y), INV),
        (dict(xp=Z - 2), INV), (dict(xp=V), INV)]),
    ("moe_permute_bwd", PBWD, BAD_ROWS + [
        (dict(dtype=U8), INV), (dict(yp=0), INV), (dict(y=0), INV), (dict(y=W + 1), INV),
        (dict(yp_ld=1), INV), (dict(y_ld=63), INV), (dict(y=X), INV), (dict(y=Y), INV)]),
    ("moe_unpermute", SUMS, BAD_ROWS + [
        (dict(dtype=U8), INV), (dict(yp=0), INV), (dict(y=0), INV), (dict(topk_w=Z + 1), INV),
        (dict(y=Z), INV), (dict(yp=X + 1), INV), (dict(y=X + 16 * 64 * 2 - 2), INV)]),
    ("moe_unpermute_bwd", GRAD, BAD_ROWS + [
        (dict(dtype=U8), INV), (dict(dyp=0, dw=0), INV), (dict(dy=0), INV), (dict(yp=0), INV),
        (dict(dy_ld=8), INV), (dict(yp_ld=8), INV), (dict(dyp_ld=8), INV), (dict(dw=W), INV),
        (dict(dyp=X), INV), (dict(dyp=Y), INV), (dict(dw=Z), INV), (dict(dw=W + 2), INV),
        (dict(dyp=V + 4096), INV)]),
    ("moe_quantize_mxfp4", QUANT, [
        (dict(rows=-1), INV), (dict(cols=0), INV), (dict(cols=48), SHAPE),
        (dict(cols=1 << 24), SHAPE), (dict(rows=1 << 30, cols=1 << 12), SHAPE),
        (dict(dtype=U8), INV), (dict(dtype=9), INV), (dict(x=0), INV), (dict(codes=0), INV),
        (dict(sf=0), INV), (dict(x=X + 1), INV), (dict(codes=Y + 2), INV), (dict(x_ld=32), INV),
        (dict(codes=X), INV), (dict(sf=X + 510), INV), (dict(sf=Y + 127), INV)]),
    ("moe_dequantize_mxfp4", DEQUANT, [
        (dict(rows=-1), INV), (dict(cols=33), SHAPE), (dict(dtype=U8), INV), (dict(x=0), INV),
        (dict(codes=0), INV), (dict(sf=0), INV), (dict(x_ld=-64), INV), (dict(x=Y), INV)]),
    ("moe_gemm_mxfp4", GEMM, [
        (dict(groups=0), INV), (dict(rows=-1), INV), (dict(n=-1), INV), (dict(k=0), INV),
        (dict(dtype=U8), INV), (dict(offsets=0), INV), (dict(offsets=0, groups=1), INV), (dict(slots=-1), INV),
        (dict(k=80), SHAPE), (dict(k=(1 << 20) + 32), SHAPE), (dict(groups=1025), SHAPE),
        (dict(rows=1 << 28), SHAPE), (dict(n=1 << 28), SHAPE), (dict(a=0), INV), (dict(b=0), INV),
        (dict(a_sf=0), INV), (dict(b_sf=0), INV), (dict(y=0), INV), (dict(a=X + 8), INV),
        (dict(b=Z + 4), INV), (dict(y=W + 1), INV), (dict(y_ld=31), INV),
        (dict(offsets=V + 4097), INV), (dict(counts=V + 8193), INV), (dict(y=X), INV),
        (dict(y=Z + 2 * 32 * 32 - 2), INV), (dict(y=V + 4096), INV), (dict(y=V + 8192), INV)]),
])
def test_refusals(name, base, changes):
    for change, code in changes:
        assert call(name, base, **change) == code, (name, change)


def test_empty_calls_are_no_ops():
    assert call("moe_permute", PERMUTE, R=0, xp=0, row_src=0) == OK
    assert call("moe_permute_bwd", PBWD, T=0, y=0, src_row=0) == OK
    assert call("moe_unpermute", SUMS, T=0, y=0, yp=0, src_row=0, topk_w=0) == OK
    assert call("moe_unpermute_bwd", GRAD, T=0, dyp=0, dy=0, yp=0, src_row=0) == OK
    assert call("moe_unpermute_bwd", GRAD, T=0, R=0) == OK
    assert call("moe_quantize_mxfp4", QUANT, rows=0, x=0, codes=0, sf=0) == OK
    assert call("moe_dequantize_mxfp4", DEQUANT, rows=0, x=0) == OK
    assert call("moe_gemm_mxfp4", GEMM, rows=0, a=0, y=0) == OK
    assert call("moe_gemm_mxfp4", GEMM, n=0, b=0, y=0) == OK


def test_binding_refuses_host_tensors():
    x, i = torch.zeros(2, 32), torch.zeros(2, dtype=torch.int32)
    u = torch.zeros(2, 16, dtype=torch.uint8)
    for f in (lambda: moe.moe_permute(x, i, i, i), lambda: moe.moe_permute_bwd(x, i, 2),
              lambda: moe.moe_unpermute(x, i, 2), lambda: moe.moe_unpermute_bwd(x, x, i, i, i),
              lambda: moe.moe_quantize_mxfp4(x), lambda: moe.moe_dequantize_mxfp4(u, u[:, :1]),
              lambda: moe.moe_gemm_mxfp4(u, u[:, :1], u, u[:, :1])):
        with pytest.raises(ValueError, match="expected a GPU"):
            f()


TILES = [(16, 16), (32, 16), (32, 64), (32, 128), (64, 128), (128, 128), (256, 256)]


def test_product_tiles():
    info = lambda *a: tuple(moe.moe_gemm_mxfp4_info(*a).values())
    # measured points of the rule: the best or within 10 % of it
    for sizes, tile in (((1, 4096, 7168), 0), ((32, 4096, 4096), 1), ((128, 4096, 7168), 2),
                        ((512, 4096, 4096), 4), ((2048, 4096, 4096), 5), ((4096, 4096, 4096), 6),
                        ((32, 4096, 4096, 32), 3), ((768, 4096, 4096, 32), 5), ((100, 2048, 2048, 16), 2),
                        ((6144, 4096, 4096, 32), 5), ((12288, 4096, 4096, 32), 6)):
        assert info(*sizes) == TILES[tile], sizes
    # every size has a tile
    for rows in (0, 1, 7, 300, 1 << 27):
        for n in (0, 1, 4097, 1 << 27):
            for g in (0, 1, 1024):
                assert info(rows, n, 32, g) in TILES
    for bad, code in (((-1, 4, 32), INV), ((4, 4, 0), INV), ((4, 4, 48), SHAPE), ((4, 4, 32, -1), INV),
                      ((4, 4, 32, 1025), SHAPE)):
        with pytest.raises(moe.MoEError) as e:
            info(*bad)
        assert e.value.code == code
    for at in range(4):                                    # not wrapped into range
        sizes = [4, 4, 32, 1]
        sizes[at] += 1 << 32
        with pytest.raises(ValueError, match="beyond 32 bits"):
            info(*sizes)
    m = ctypes.c_int32()
    assert ops.ops_lib().moe_gemm_mxfp4_info(0, 4, 4, 32, None, ctypes.addressof(m)) == INV
