"""moe_quantize_mxfp4, moe_dequantize_mxfp4 and moe_gemm_mxfp4 on the GPU
against their definitions in float64: conversions have to be equal, products
within the float32 rounding of their sums."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_amd as moe
import ops_util as ou
import workload as wl
from parity_util import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def unpack(codes):
    c = codes.cpu().numpy()
    return np.stack([ou.E2M1[c & 15], ou.E2M1[c >> 4]], -1).reshape(c.shape[0], -1)


def check_quantised(x):
    codes, sf = moe.moe_quantize_mxfp4(x)
    q, e = ou.quantised(x.double().cpu().numpy())
    assert np.array_equal(sf.cpu().numpy().astype(np.int64) - 127, e)
    got = unpack(codes)
    assert np.array_equal(got, q) and np.array_equal(np.signbit(got), np.signbit(q))
    return codes, sf


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 4096), (3, 64), (65, 96), (129, 2080), (7, 8224), (1000, 160)])
def test_quantise_rows(rows, cols, dtype):
    say(f"quantise {rows} x {cols} {dtype}")
    rng = np.random.default_rng(rows + cols)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-12, 12, (rows, cols // 32))).repeat(32, 1)
    x = torch.from_numpy(x).to(DT[dtype]).cuda()
    codes, sf = check_quantised(x)
    v = ou.values(codes.cpu().numpy(), sf.cpu().numpy())
    for out in DT.values():
        assert np.array_equal(moe.moe_dequantize_mxfp4(codes, sf, out).double().cpu().numpy(), ou.rounded(v, out))


def test_quantise_ties_zeros_and_extremes():
    ties = [0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, .2500001, .7499999, 4.9999995, 5.0000005]
    row = np.array(ties + [-v for v in ties] + [0.5] * 6)
    rows = [row * 2.0 ** e for e in (-36, -30, -8, 0, 1, 40, 120)]   # amax 6: the scale is 2^e
    rows += [np.zeros(32), -np.zeros(32), np.full(32, 1e-10), np.full(32, 1e-12), np.full(32, 2.0 ** -149),
             np.full(32, 3.4028234663852886e38), np.linspace(-6.0000005, 6.0000005, 32),
             np.linspace(-7, 7, 32), np.linspace(-3.0000002, 3, 32), np.linspace(-1e-10, 6.1e-10, 32)]
    check_quantised(torch.from_numpy(np.stack(rows).astype(np.float32)).cuda())
    h = np.stack([np.linspace(-65504, 65504, 32), np.full(32, 2.0 ** -24), np.linspace(0, 2.0 ** -14, 32)])
    check_quantised(torch.from_numpy(h).half().cuda())
    b = np.stack([np.linspace(-3e38, 3e38, 32), np.full(32, 1e-40), np.linspace(0, 1e-9, 32)])
    check_quantised(torch.from_numpy(b).bfloat16().cuda())


def test_quantise_every_bf16_value_against_each_scale():
    # each finite bf16 magnitude up to 6 times the scale, beside a 6: every rounding of the type
    v = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()
    for e in (-20, 0, 60):
        x = v[(v <= 6 * 2.0 ** e) & (v >= 2.0 ** (e - 12))]
        x = torch.cat([x, torch.zeros(-x.numel() % 31, dtype=x.dtype)]).view(-1, 31)
        x = torch.cat([x, torch.full((x.shape[0], 1), 6 * 2.0 ** e, dtype=x.dtype)], 1)
        check_quantised(x.bfloat16().cuda())
        check_quantised((-x).float().cuda())


def test_quantise_matches_the_input_generator():
    x = torch.from_numpy(np.random.default_rng(8).standard_normal((48, 512)).astype(np.float32))
    codes, sf = moe.moe_quantize_mxfp4(x.cuda())
    want, wsf = wl.quantize_mx_e2m1(x)
    assert torch.equal(sf.cpu(), wsf) and np.array_equal(unpack(codes), unpack(want))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", list(DT))
def test_a_block_that_is_not_finite_is_nan(dtype, bad):
    x = torch.randn(5, 160, device="cuda").to(DT[dtype])
    want, wsf = moe.moe_quantize_mxfp4(x)
    y = x.clone()
    y[1, 40], y[4, 159] = bad, bad
    codes, sf = moe.moe_quantize_mxfp4(y)
    wsf[1, 1], wsf[4, 4] = 255, 255
    assert torch.equal(sf, wsf)
    v, wv = moe.moe_dequantize_mxfp4(codes, sf, DT[dtype]), moe.moe_dequantize_mxfp4(want, wsf, DT[dtype])
    nan = torch.zeros_like(v, dtype=torch.bool)
    nan[1, 32:64], nan[4, 128:] = True, True
    assert torch.equal(torch.isnan(v), nan) and torch.equal(torch.isnan(wv), nan)
    assert torch.equal(v[~nan], wv[~nan])


@pytest.mark.parametrize("dtype", list(DT))
def test_dequantise_every_code(dtype):
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(16, 16).repeat(16, 1)
    codes = codes.reshape(1, -1).repeat(256, 1).contiguous()       # every byte under every scale code
    sf = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None].repeat(1, codes.shape[1] // 16).contiguous()
    got = moe.moe_dequantize_mxfp4(codes.cuda(), sf.cuda(), DT[dtype]).double().cpu().numpy()
    with np.errstate(over="ignore"):
        want = ou.rounded(ou.values(codes.numpy(), sf.numpy()), DT[dtype])
    assert np.array_equal(got, want, equal_nan=True)
    fine = ~np.isnan(want)
    assert np.array_equal(np.signbit(got)[fine], np.signbit(want)[fine])


@pytest.mark.parametrize("dtype", list(DT))
def test_quantise_strided_rows(dtype):
    big = torch.randn(13, 203, device="cuda").to(DT[dtype])
    x = big[:, 3:3 + 160]                                   # odd addresses and row stride
    codes, sf = check_quantised(x)
    out = torch.full((13, 171), 9.0, dtype=DT[dtype], device="cuda")
    moe.moe_dequantize_mxfp4(codes, sf, DT[dtype], out=out[:, 1:161])
    assert torch.equal(out[:, 1:161], moe.moe_dequantize_mxfp4(codes, sf, DT[dtype]))
    assert torch.all(out[:, 0] == 9) and torch.all(out[:, 161:] == 9)


@pytest.mark.parametrize("rows,cols", [((1 << 26) + 77, 32), (3, (1 << 24) - 32), (70000, 33024)])
def test_quantise_past_32_bit_offsets(rows, cols):
    say(f"quantise {rows} x {cols}")
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    codes, sf = moe.moe_quantize_mxfp4(x)
    back = moe.moe_dequantize_mxfp4(codes, sf)
    for at in (0, rows // 2, max(0, rows - 100)):
        s = slice(at, at + 100)
        c, f = moe.moe_quantize_mxfp4(x[s].clone())
        assert torch.equal(codes[s], c) and torch.equal(sf[s], f)
        assert torch.equal(back[s], moe.moe_dequantize_mxfp4(c, f))
    del x, codes, sf, back
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- product

# One MFMA rounds its running f32 sum with an error of at most 2^-22 of the
# magnitudes that entered it (measured: 2^-22.9 over scales 2^62 apart); a sum
# passes at most K / 64 of them and 8 additions of partial sums.
def bound(k, mag, exact, dtype):
    inner = (k / 64 + 1 + 8) * 2.0 ** -22 * mag
    return inner + ou.half_step(dtype) * (abs(exact) + inner) + ou.least(dtype)


def operand(rng, rows, k, spread):
    codes = rng.integers(0, 256, (rows, k // 2)).astype(np.uint8)
    sf = rng.integers(127 - spread, 128 + spread, (rows, k // 32)).astype(np.uint8)
    return codes, sf


def exact(a, asf, b, bsf):
    va, vb = torch.from_numpy(ou.values(a, asf)), torch.from_numpy(ou.values(b, bsf))
    return (va @ vb.t()).numpy(), (va.abs() @ vb.abs().t()).numpy()


def check_product(got, ex, mag, k, dtype, what):
    got = got.double().cpu().numpy()
    # The largest finite value is (2 - eps) 2^E; half a step above it, at (2 - eps / 2) 2^E
    # (f16: 65504 + 16), rounding to nearest gives infinity.  The sum before that rounding
    # is within `inner` of ex, so only sums nearer than that to the edge may go either way.
    info = torch.finfo(dtype)
    edge = info.max / (2 - info.eps) * (2 - info.eps / 2)
    inner = (k / 64 + 1 + 8) * 2.0 ** -22 * mag
    inf = np.isinf(got)
    assert np.all(inf[abs(ex) - inner >= edge]) and not np.any(inf[abs(ex) + inner < edge]), what
    assert np.array_equal(np.sign(got[inf]), np.sign(ex[inf])), what
    off, lim = abs(got - ex)[~inf], bound(k, mag, ex, dtype)[~inf]
    assert np.all(off <= lim), (what, float((off / lim).max()), np.argwhere(~inf)[off > lim][:4])


DENSE = [(1, 1, 32), (1, 17, 64), (1, 256, 4096), (2, 100, 96), (5, 33, 8192), (15, 16, 160), (16, 16, 256),
         (17, 255, 288), (32, 48, 1024), (33, 257, 512), (48, 31, 224), (49, 64, 128), (64, 129, 2080),
         (100, 300, 256), (127, 512, 544), (128, 128, 32), (129, 127, 800), (200, 1000, 352), (256, 256, 256),
         (257, 255, 288), (512, 250, 480), (513, 513, 96), (600, 270, 1056), (1025, 40, 736), (2050, 600, 320),
         # long sums, some of them beyond the range of f16
         (3, 20, 131072), (40, 33, 65568), (300, 70, 16416)]


@pytest.mark.parametrize("m,n,k", DENSE)
def test_dense_product(m, n, k):
    say(f"dense product {m} x {n} x {k}")
    rng = np.random.default_rng(m + n + k)
    a, asf = operand(rng, m, k, 3)
    b, bsf = operand(rng, n, k, 3)
    ex, mag = exact(a, asf, b, bsf)
    d = [torch.from_numpy(v).cuda() for v in (a, asf, b, bsf)]
    for dtype in DT.values():
        y = torch.full((m + 1, n + 3), 77.0, dtype=dtype, device="cuda")
        got = moe.moe_gemm_mxfp4(*d, out=y[:m, 1:n + 1])
        check_product(got, ex, mag, k, dtype, dtype)
        assert torch.all(y[m] == 77) and torch.all(y[:, 0] == 77) and torch.all(y[:, n + 1:] == 77)
    again = moe.moe_gemm_mxfp4(*d, dtype=torch.float32)
    assert torch.equal(again, moe.moe_gemm_mxfp4(*d, dtype=torch.float32))


# Ragged sizes of every tile: rows, n, k, segments (0: dense), the tile
BY_TILE = [(11, 700, 1184, 0, (16, 16)), (29, 3000, 1056, 0, (32, 16)), (130, 1500, 2080, 0, (32, 64)),
           (300, 8190, 1024, 0, (32, 128)), (511, 3000, 2144, 0, (64, 128)), (2047, 2100, 800, 0, (128, 128)),
           (12001, 1001, 992, 0, (256, 256)), (45, 2050, 480, 20, (32, 64)), (333, 4000, 1056, 40, (32, 128)),
           (2100, 600, 512, 20, (64, 128)), (6100, 1900, 544, 30, (128, 128)), (12300, 1000, 1024, 7, (256, 256)),
           # b read once and past the caches
           (31, 7999, 4128, 5, (32, 128)), (31, 66010, 2080, 0, (32, 128)), (700, 3701, 2144, 17, (128, 128))]


@pytest.mark.parametrize("rows,n,k,groups,tile", BY_TILE, ids=str)
def test_product_by_tile(rows, n, k, groups, tile):
    say(f"product {rows} x {n} x {k}, {groups} segments: tile {tile}")
    assert tuple(moe.moe_gemm_mxfp4_info(rows, n, k, groups).values()) == tile
    rng = np.random.default_rng(rows)
    E = max(1, groups)
    a, asf = operand(rng, rows, k, 3)
    b, bsf = operand(rng, E * n, k, 3)
    table = torch.from_numpy(ou.E2M1).cuda()

    def on_gpu(codes, sf):
        v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
        return v * torch.exp2(sf.double() - 127).repeat_interleave(32, -1)

    d = [torch.from_numpy(v).cuda() for v in (a, asf, b, bsf)]
    va, vb = on_gpu(*d[:2]), on_gpu(*d[2:]).view(E, n, k)
    args, lens = d, [rows]
    kw = {}
    if groups:
        lens = rng.multinomial(rows, rng.dirichlet(np.full(E, 2.0)))
        lens[E // 2] += lens[0]
        lens[0] = 0                                         # an expert without rows
        off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        kw = dict(offsets=torch.from_numpy(off).cuda())
        args = [d[0], d[1], d[2].view(E, n, -1), d[3].view(E, n, -1)]
    for dtype in (torch.bfloat16, torch.float32):
        y = torch.full((rows, n), 5.0, dtype=dtype, device="cuda")
        moe.moe_gemm_mxfp4(*args, out=y, **kw)
        first = 0
        for e, c in enumerate(lens):
            if c:
                s = slice(first, first + int(c))
                ex, mag = va[s] @ vb[e].t(), va[s].abs() @ vb[e].abs().t()
                inner = (k / 64 + 1 + 8) * 2.0 ** -22 * mag
                off_by = (y[s].double() - ex).abs()
                lim = inner + ou.half_step(dtype) * (ex.abs() + inner) + ou.least(dtype)
                assert torch.all(off_by <= lim), (e, (off_by / lim).max().item())
            first += int(c)
    z = torch.full_like(y, 5.0)
    assert torch.equal(moe.moe_gemm_mxfp4(*args, out=z, **kw), y)


@pytest.mark.parametrize("spread", [8, 31])
@pytest.mark.parametrize("m,n,k", [(4, 40, 512), (40, 40, 512), (130, 140, 512), (700, 300, 512)])
def test_product_of_far_scales(m, n, k, spread):
    rng = np.random.default_rng(m + spread)
    a, asf = operand(rng, m, k, spread)
    b, bsf = operand(rng, n, k, spread)
    ex, mag = exact(a, asf, b, bsf)
    got = moe.moe_gemm_mxfp4(*[torch.from_numpy(v).cuda() for v in (a, asf, b, bsf)], dtype=torch.float32)
    check_product(got, ex, mag, k, torch.float32, spread)


GROUPS = [([1], 96, 64, 1), ([0, 0, 3, 0], 40, 128, 1), ([3, 0, 1, 17, 16], 100, 288, 16),
          ([2] * 70 + [0] * 9 + [5] * 60, 50, 256, 1), ([40, 0, 33, 16, 48], 130, 512, 16),
          ([24] * 32, 300, 1024, 1), ([128, 129, 0, 1, 127], 200, 352, 128), ([200, 0, 61, 300], 270, 96, 64),
          ([700, 3, 900], 260, 544, 1), ([600, 513, 0, 511], 515, 256, 128)]


@pytest.mark.parametrize("lens,n,k,align", GROUPS, ids=lambda v: str(v)[:24])
def test_grouped_product(lens, n, k, align):
    say(f"grouped product {str(lens)[:40]} {n} x {k}")
    rng = np.random.default_rng(sum(lens) + n)
    E = len(lens)
    offsets = np.concatenate([[0], np.cumsum([-(-c // align) * align for c in lens])]).astype(np.int32)
    rows = int(offsets[-1]) + 9                             # nine rows behind the last segment
    a, asf = operand(rng, rows, k, 3)
    b, bsf = zip(*[operand(rng, n, k, 3) for _ in lens])
    live = np.zeros(rows, bool)
    for e, c in enumerate(lens):
        live[offsets[e]:offsets[e] + c] = True
    asf[~live] = 255                                        # rows outside hold NaN
    d = [torch.from_numpy(v).cuda() for v in (a, asf, np.stack(b), np.stack(bsf), offsets)]
    counts = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for dtype in DT.values():
        y = torch.full((rows, n), 55.0, dtype=dtype, device="cuda")
        moe.moe_gemm_mxfp4(*d, counts=counts, out=y)
        assert torch.all(y[torch.from_numpy(~live).cuda()] == 55)
        for e, c in enumerate(lens):
            s = slice(offsets[e], offsets[e] + c)
            if c:
                check_product(y[s], *exact(a[s], asf[s], b[e], bsf[e]), k, dtype, (e, dtype))
    for slots in (sum(lens), sum(lens) + 5):                # the launch sized by the rows there are
        z = torch.full((rows, n), 55.0, dtype=torch.float32, device="cuda")
        moe.moe_gemm_mxfp4(*d, counts=counts, out=z, slots=slots)
        assert torch.all(z[torch.from_numpy(~live).cuda()] == 55)
        for e, c in enumerate(lens):
            s = slice(offsets[e], offsets[e] + c)
            if c:
                check_product(z[s], *exact(a[s], asf[s], b[e], bsf[e]), k, torch.float32, (e, slots))
    if align == 1:                                          # whole segments without counts
        z = torch.full_like(y, 55.0)
        assert torch.equal(moe.moe_gemm_mxfp4(*d, out=z), y)
    # without counts the padding rows belong to the segments, whatever slots says
    a2, asf2 = d[0], torch.where(d[1] == 255, 127, d[1])
    unset = torch.full_like(y, float("nan"))
    whole = [moe.moe_gemm_mxfp4(a2, asf2, *d[2:], out=unset.clone(), slots=v) for v in (0, 1, sum(lens))]
    used = int(offsets[-1])
    for z in whole:
        assert torch.equal(z[:used], whole[0][:used]) and torch.all(torch.isnan(z[used:]))


@pytest.mark.parametrize("rows", [6, 40, 200, 900])
def test_nan_scales_and_cut_segments(rows):
    rng = np.random.default_rng(rows)
    n, k = 90, 352
    a, asf = operand(rng, rows, k, 2)
    b, bsf = operand(rng, n, k, 2)
    asf[rows // 2, 3], bsf[17, 10] = 255, 255
    d = [torch.from_numpy(v).cuda() for v in (a, asf, b, bsf)]
    y = moe.moe_gemm_mxfp4(*d, dtype=torch.float32).cpu().numpy()
    nan = np.zeros((rows, n), bool)
    nan[rows // 2], nan[:, 17] = True, True
    assert np.array_equal(np.isnan(y), nan)
    # segments that start or end outside the matrix are cut to it
    off = torch.tensor([-5, rows - 2, rows + 10, 3], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([9, 100, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    z = torch.full((rows, n), 3.0, device="cuda")
    moe.moe_gemm_mxfp4(d[0], d[1], d[2].expand(3, n, k // 2).contiguous(), d[3].expand(3, n, k // 32).contiguous(),
                       offsets=off, counts=cnt, out=z)
    assert torch.all(z[:rows - 2] == 3)
    # (a grouped call of few rows an expert may take another tile than the dense one)
    ex, mag = exact(a[-2:], asf[-2:], b, bsf)
    fine = ~nan[-2:]
    got = z[rows - 2:].cpu().numpy()
    assert np.array_equal(np.isnan(got), ~fine)
    assert np.all(abs(got - ex)[fine] <= bound(k, mag, ex, torch.float32)[fine])


@pytest.mark.parametrize("rows,n", [(1, (1 << 28) - 1), (3, (1 << 27) + 5), ((1 << 28) - 1, 1), ((1 << 27) + 300, 3)])
def test_largest_sizes(rows, n):
    # One block of K: sums of 32 products of e2m1 values under one scale are exact in
    # f32, whatever the tile, so pieces of the long side can be compared as calls of their own.
    say(f"product {rows} x {n} x 32")
    side = max(rows, n)
    g = torch.Generator(device="cuda").manual_seed(7)
    wide = torch.randint(0, 256, (side, 16), dtype=torch.uint8, device="cuda", generator=g)
    wide_sf = torch.randint(120, 134, (side, 1), dtype=torch.uint8, device="cuda", generator=g)
    few, few_sf = wide[1000:1000 + min(rows, n)].clone(), wide_sf[1000:1000 + min(rows, n)].clone()
    call = lambda w, f: (moe.moe_gemm_mxfp4(few, few_sf, w, f) if n > rows else moe.moe_gemm_mxfp4(w, f, few, few_sf))
    y = call(wide, wide_sf)
    for at in (0, 65536, (1 << 26) - 500, (1 << 27) - 777, side - 1001):
        part = call(wide[at:at + 1001], wide_sf[at:at + 1001].clone())
        assert torch.equal(y[:, at:at + 1001] if n > rows else y[at:at + 1001], part), at
    del wide, wide_sf, y
    torch.cuda.empty_cache()


def test_segments_that_overlap():
    # (not allowed; whatever they leave in their rows, the others stay)
    rows, n, k, E = 300, 40, 64, 130
    d = [torch.randint(0, 128, s, dtype=torch.uint8, device="cuda")
         for s in ((rows, k // 2), (rows, k // 32), (E, n, k // 2), (E, n, k // 32))]
    off = torch.full((E + 1,), 20, dtype=torch.int32, device="cuda")
    cnt = torch.full((E,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    for slots in (0, 7):
        y = torch.full((rows + 1, n), 5.0, device="cuda")
        moe.moe_gemm_mxfp4(*d, offsets=off, counts=cnt, slots=slots, out=y[:rows])
        assert torch.all(y[:20] == 5) and torch.all(y[rows] == 5)


def test_product_refusals():
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    a, asf, b, bsf = u(8, 32), u(8, 2), u(16, 32), u(16, 2)
    bad = [lambda: moe.moe_gemm_mxfp4(a, asf, u(16, 16), bsf), lambda: moe.moe_gemm_mxfp4(a, u(8, 4), b, bsf),
           lambda: moe.moe_gemm_mxfp4(a, asf, b, u(16, 1)), lambda: moe.moe_gemm_mxfp4(a, asf, b[None], bsf[None]),
           lambda: moe.moe_gemm_mxfp4(a, asf, b, bsf, offsets=i(0, 8)), lambda: moe.moe_gemm_mxfp4(a, asf, b, bsf, counts=i(8)),
           lambda: moe.moe_gemm_mxfp4(a, asf, b[None], bsf[None], offsets=i(0, 4, 8)),
           lambda: moe.moe_gemm_mxfp4(a, asf, b, bsf, dtype=torch.float64),
           lambda: moe.moe_gemm_mxfp4(a, asf, b, bsf, out=torch.zeros(8, 15, device="cuda")),
           lambda: moe.moe_gemm_mxfp4(a, asf, b, bsf, dtype=torch.float16, out=torch.zeros(8, 16, device="cuda")),
           lambda: moe.moe_gemm_mxfp4(a.t(), asf, b, bsf), lambda: moe.moe_gemm_mxfp4(a, asf, b.cpu(), bsf),
           lambda: moe.moe_quantize_mxfp4(torch.zeros(2, 64, device="cuda").t()),
           lambda: moe.moe_quantize_mxfp4(torch.zeros(2, 64, device="cuda", dtype=torch.float64)),
           lambda: moe.moe_quantize_mxfp4(torch.zeros(2, 64, device="cuda"), codes=u(2, 31)),
           lambda: moe.moe_dequantize_mxfp4(a, u(8, 1)), lambda: moe.moe_dequantize_mxfp4(a, asf, torch.int32)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: moe.moe_quantize_mxfp4(torch.zeros(2, 48, device="cuda")),
              lambda: moe.moe_gemm_mxfp4(u(8, 24), u(8, 1), u(16, 24), u(16, 1))):
        with pytest.raises(moe.MoEError):
            f()
