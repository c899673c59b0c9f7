"""moe_gemm_wgrad on the GPU against plain float64 forms."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_amd as moe
import layer_util as lu
import ops_util as ou
from parity_util import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
# rows, experts (0: dense), n, k, alignment: tiles and their edges, experts without rows, shares of rows
SHAPES = [(1, 0, 1, 32, 1), (31, 0, 7, 96, 1), (32, 0, 128, 128, 1), (33, 0, 129, 160, 1), (200, 0, 40, 384, 1),
          (5, 8, 33, 64, 1), (64, 3, 127, 256, 16), (300, 8, 136, 640, 1), (77, 1, 257, 128, 64), (1000, 5, 264, 288, 16),
          (3000, 0, 50, 128, 1), (2500, 2, 130, 96, 8), (9000, 0, 300, 256, 1), (700, 40, 16, 128, 128), (513, 0, 512, 512, 1)]


def x_values(codes, sf, dtype):
    """What the codes stand for in dy's type: a float32 product, rounded."""
    c = torch.from_numpy(lu.E4M3[codes.cpu().numpy()]).float()
    s = torch.from_numpy(lu.scales(sf)).float()
    return (c * s.repeat_interleave(codes.shape[1] // s.shape[1], 1)).to(dtype)


def make(shape, dtype, fmt, seed=0):
    """dy, codes, sf and lists (None: dense) of a pool whose padding rows are NaN."""
    rows, E, n, k, align = shape
    rng = np.random.default_rng(seed + rows + 3 * n + k)
    lists = None
    R = rows
    if E:
        idx = rng.integers(0, E, (rows, 1))
        idx[idx == E // 2] = 0 if E > 1 else E // 2           # an expert without rows
        lists = ou.route(idx, E, align)
        R = lists["pool"]
    dy = torch.from_numpy(rng.standard_normal((R, n))).to(dtype)
    codes, sf = lu.quantised(torch.from_numpy(rng.standard_normal((R, k)) * (1 + 9 * (rng.random((1, k)) < 0.05))).float(), fmt)
    if lists is not None:
        dead = torch.from_numpy(lists["row_src"] < 0)
        dy[dead] = float("nan")
        codes[dead] = 0x7F
    return dy, codes, sf, lists


def plain(dy, xv, lists, E, whole=False):
    """(sums, sums of magnitudes, most rows of an expert) in float64."""
    dy, xv = lu.f64(dy), lu.f64(xv)
    out, mag, most = [], [], 0
    for e in range(max(1, E)):
        a, m = (0, dy.shape[0]) if not E else (lists["offsets"][e], lists["counts"][e])
        if E and whole:
            m = lists["offsets"][e + 1] - a
        out.append(dy[a:a + m].T @ xv[a:a + m])
        mag.append(abs(dy[a:a + m]).T @ abs(xv[a:a + m]))
        most = max(most, m)
    return (out[0], mag[0], most) if not E else (np.stack(out), np.stack(mag), most)


def bound_of(want, mag, most, dtype):
    # exact products; each of the sum's `most` additions, and those of 16 shares, cut or rounded to 24 bits
    return lu.rounded_bound(want, (most + 18) * 2.0 ** -23 * mag, dtype)


def seg(lists):
    return {} if lists is None else {k: torch.from_numpy(lists[k]).cuda() for k in ("offsets", "counts")}


@pytest.mark.parametrize("fmt", [0, 1], ids=["f32", "ue8m0"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_product_against_the_plain_form(shape, dtype, fmt):
    if shape[3] % lu.BLOCK[fmt]:
        pytest.skip("columns are no whole blocks")
    say(f"weight gradient {shape} {dtype} {fmt}")
    dt = DT[dtype]
    dy, codes, sf, lists = make(shape, dt, fmt)
    want, mag, most = plain(dy, x_values(codes, sf, dt), lists, shape[1])
    d = (dy.cuda(), codes.cuda(), sf.cuda())
    got = moe.moe_gemm_wgrad(*d, **seg(lists))
    assert got.dtype == torch.float32
    lu.within(got, want, bound_of(want, mag, most, torch.float32))
    for out in (torch.bfloat16, torch.float16):
        v = moe.moe_gemm_wgrad(*d, dtype=out, **seg(lists))
        assert torch.equal(v, got.to(out))                    # the same sum, rounded once
    again = moe.moe_gemm_wgrad(*d, **seg(lists))
    assert torch.equal(again, got)
    # added to what is there, experts without rows left as they were
    for out in (torch.float32, torch.bfloat16):
        old = torch.randn(got.shape, device="cuda").to(out)
        v = moe.moe_gemm_wgrad(*d, out=old.clone(), accumulate=True, **seg(lists))
        assert torch.equal(v, (old.float() + got).to(out))


@pytest.mark.parametrize("dtype", list(DT))
def test_whole_numbers_are_exact(dtype):
    # values and sums that float32 holds: every layout mistake shows, no rounding does
    say("whole numbers")
    dt = DT[dtype]
    for rows, E, n, k in ((257, 0, 333, 480), (700, 6, 200, 224), (4100, 0, 65, 96)):
        rng = np.random.default_rng(n)
        idx = rng.integers(0, max(1, E), (rows, 1))
        lists = ou.route(idx, E, 8) if E else None
        R = lists["pool"] if E else rows
        dy = torch.from_numpy(rng.integers(-8, 9, (R, n))).to(dt)
        codes = torch.from_numpy(rng.integers(0, 256, (R, k)).astype(np.uint8))
        codes[(codes & 127) == 127] = 0
        codes = torch.where((codes & 120) >= 64, codes & 0xBF, codes)      # magnitudes below 4
        sf = torch.from_numpy(rng.integers(127, 130, (R, k // 32)).astype(np.uint8))
        want = plain(dy, x_values(codes, sf, dt), lists, E)[0]
        got = moe.moe_gemm_wgrad(dy.cuda(), codes.cuda(), sf.cuda(), **seg(lists))
        # (multiples of 2^-9 below 2^7 * rows in all: 24 bits hold 2^15, so sums of up to 200 rows or so;
        # longer ones round, each addition to 2^-24 of at most the magnitudes)
        m = plain(dy, x_values(codes, sf, dt), lists, E)[1]
        lu.within(got, want, np.where(m * 512 < 2 ** 24, 0.0, m * (rows + 18) * 2.0 ** -23))


def test_segments_without_counts_and_bad_lists():
    say("segments")
    shape = (200, 4, 70, 64, 16)
    dy, codes, sf, lists = make(shape, torch.bfloat16, 1, 5)
    dy, codes = torch.nan_to_num(dy, nan=0.5), torch.where(codes == 0x7F, 0x38, codes)
    xv = x_values(codes, sf, torch.bfloat16)
    off = torch.from_numpy(lists["offsets"]).cuda()
    d = (dy.cuda(), codes.cuda(), sf.cuda())
    want, mag, most = plain(dy, xv, lists, 4, whole=True)
    lu.within(moe.moe_gemm_wgrad(*d, offsets=off), want, bound_of(want, mag, most, torch.float32))
    # cut at the rows there are; an empty or negative length is no rows
    R = dy.shape[0]
    bad_off = torch.tensor([0, R - 5, R + 50, 7, 7], dtype=torch.int32).cuda()
    counts = torch.tensor([3, 100, 4, -2], dtype=torch.int32).cuda()
    got = moe.moe_gemm_wgrad(*d, offsets=bad_off, counts=counts)
    for e, rows in enumerate((slice(0, 3), slice(R - 5, R), slice(0, 0), slice(0, 0))):
        w, m, n = plain(dy[rows], xv[rows], None, 0)
        lu.within(got[e], w, bound_of(w, m, n, torch.float32))
    for kw in (dict(offsets=off, counts=torch.zeros_like(counts)), dict(offsets=torch.zeros_like(off))):
        old = torch.full((4, 70, 64), 3.0, device="cuda")
        assert torch.all(moe.moe_gemm_wgrad(*d, out=old.clone(), **kw) == 0)
        assert torch.equal(moe.moe_gemm_wgrad(*d, out=old.clone(), accumulate=True, **kw), old)


def test_shares_of_experts_with_and_without_rows():
    # rows of few experts split over workgroups, added to what is there: the experts' planes meet inside a wave
    say("shares of experts")
    R, n, k = 6000, 130, 96
    dy, codes, sf, _ = make((R, 0, n, k, 1), torch.bfloat16, 1, 4)
    d = (dy.cuda(), codes.cuda(), sf.cuda())
    assert moe.moe_gemm_wgrad_workspace_bytes(3, R, n, k) > 3 * n * k * 4
    for counts in ((0, R, 0), (R, 0, 0), (5, 0, R - 5), (0, 0, 0)):
        off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
        old = torch.randn(3, n, k, device="cuda")
        fresh = moe.moe_gemm_wgrad(*d, offsets=off)
        added = moe.moe_gemm_wgrad(*d, offsets=off, out=old.clone(), accumulate=True)
        for e, c in enumerate(counts):
            rows = slice(sum(counts[:e]), sum(counts[:e]) + c)
            w, m, most = plain(dy[rows], x_values(codes[rows], sf[rows], torch.bfloat16), None, 0)
            lu.within(fresh[e], w, bound_of(w, m, most, torch.float32))
            assert torch.equal(added[e], old[e] + fresh[e] if c else old[e])


def test_strides_and_odd_addresses():
    say("weight gradient strides")
    for n in (64, 71, 130):
        dy, codes, sf, _ = make((90, 0, n, 96, 1), torch.float16, 1, 2)
        big = torch.full((90, n + 5), float("nan"), dtype=torch.float16, device="cuda")
        big[:, 3:3 + n] = dy.cuda()
        want = moe.moe_gemm_wgrad(dy.cuda(), codes.cuda(), sf.cuda())
        assert torch.equal(moe.moe_gemm_wgrad(big[:, 3:3 + n], codes.cuda(), sf.cuda()), want)
        odd = torch.zeros(n * 96 + 1, dtype=torch.bfloat16, device="cuda")
        moe.moe_gemm_wgrad(dy.cuda(), codes.cuda(), sf.cuda(), out=odd[1:].view(n, 96))
        assert torch.equal(odd[1:].view(n, 96), want.bfloat16()) and odd[0] == 0


def test_special_values():
    say("weight gradient: infinities and NaN")
    dy, codes, sf, _ = make((50, 0, 40, 64, 1), torch.bfloat16, 1, 3)
    dy[49, 3] = float("inf")
    dy[10, 5] = float("nan")
    codes[20, 7] = 0xFF
    sf[30, 1] = 0xFF
    codes[49, 8], codes[49, 9] = 0, 0x38
    got = moe.moe_gemm_wgrad(dy.cuda(), codes.cuda(), sf.cuda()).cpu()
    nan = torch.isnan(got)
    want = torch.zeros(40, 64, dtype=torch.bool)
    want[5], want[:, 7], want[:, 32:], want[3, 8] = True, True, True, True
    assert torch.equal(nan | torch.isinf(got), want | (torch.arange(40) == 3)[:, None])
    assert torch.all(nan[want & (torch.arange(40) != 3)[:, None]]) and got[3, 9] == float("inf") and nan[3, 8]
    # a float32 result beyond f16 becomes an infinity
    big = torch.full((8, 4), 3e4, dtype=torch.float16, device="cuda")
    c, s = torch.full((8, 32), 0x48, dtype=torch.uint8, device="cuda"), torch.full((8, 1), 127, dtype=torch.uint8, device="cuda")
    assert torch.all(moe.moe_gemm_wgrad(big, c, s, dtype=torch.float16) == float("inf"))
    assert torch.all(moe.moe_gemm_wgrad(big, c, s) == 960000)
    # x beyond f16's range rounds to an infinity of its type
    s[:] = 127 + 15
    assert torch.all(torch.isinf(moe.moe_gemm_wgrad(big, c, s)))


def test_empty():
    say("weight gradient: nothing to do")
    e = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    c, s = torch.empty(0, 64, dtype=torch.uint8, device="cuda"), torch.empty(0, 2, dtype=torch.uint8, device="cuda")
    assert torch.all(moe.moe_gemm_wgrad(e, c, s, out=torch.ones(40, 64, device="cuda")) == 0)
    assert torch.all(moe.moe_gemm_wgrad(e, c, s, out=torch.ones(40, 64, device="cuda"), accumulate=True) == 1)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert torch.all(moe.moe_gemm_wgrad(e, c, s, offsets=off, out=torch.ones(3, 40, 64, device="cuda")) == 0)
    none = torch.empty(5, 0, dtype=torch.bfloat16, device="cuda")
    assert moe.moe_gemm_wgrad(none, torch.zeros(5, 64, dtype=torch.uint8, device="cuda"),
                              torch.zeros(5, 2, dtype=torch.uint8, device="cuda")).shape == (0, 64)


def test_rows_past_32_bit_offsets():
    R, n, k = 600000, 4096, 4096                              # 4.9 GB of dy, 2.5 GB of codes
    say(f"weight gradient of {R} rows")
    dy = torch.zeros(R, n, dtype=torch.bfloat16, device="cuda")
    codes, sf = torch.zeros(R, k, dtype=torch.uint8, device="cuda"), torch.full((R, k // 32), 127, dtype=torch.uint8, device="cuda")
    tail = slice(R - 40, R)
    dy[tail] = torch.randn(40, n, device="cuda").bfloat16()
    codes[tail] = torch.randint(0, 0x7F, (40, k), device="cuda").to(torch.uint8)
    off = torch.tensor([0, R - 40, R], dtype=torch.int32, device="cuda")
    got = moe.moe_gemm_wgrad(dy, codes, sf, offsets=off)
    assert torch.all(got[0] == 0)
    want = moe.moe_gemm_wgrad(dy[tail].clone(), codes[tail].clone(), sf[tail].clone())
    assert torch.equal(got[1], want)
    del dy, codes, got
    torch.cuda.empty_cache()


# rows, experts (0: dense), n, k, alignment, shares: sizes that the larger tiles take, whole and in shares of the rows
LARGER = [(5805, 8, 399, 2048, 1, False), (4686, 0, 391, 2304, 1, True), (300, 8, 519, 1664, 1, False), (5679, 0, 1037, 2432, 1, True)]


@pytest.mark.parametrize("dtype,fmt", [("bf16", 1), ("f16", 0)], ids=["bf16-ue8m0", "f16-f32"])
@pytest.mark.parametrize("shape", LARGER, ids=str)
def test_larger_products_against_the_plain_form(shape, dtype, fmt):
    say(f"weight gradient {shape} {dtype} {fmt}")
    dt, (rows, E, n, k, _, shares) = DT[dtype], shape
    dy, codes, sf, lists = make(shape[:5], dt, fmt, 5)
    assert (moe.moe_gemm_wgrad_workspace_bytes(max(1, E), len(dy), n, k) > 0) == shares
    want, mag, most = plain(dy, x_values(codes, sf, dt), lists, E)
    d = (dy.cuda(), codes.cuda(), sf.cuda())
    got = moe.moe_gemm_wgrad(*d, **seg(lists))
    lu.within(got, want, bound_of(want, mag, most, torch.float32))
    assert torch.equal(moe.moe_gemm_wgrad(*d, dtype=torch.bfloat16, **seg(lists)), got.bfloat16())
    old = torch.randn(got.shape, device="cuda")
    none = torch.zeros(got.shape, dtype=torch.bool)
    if E:
        none[lists["counts"] == 0] = True
    assert torch.equal(moe.moe_gemm_wgrad(*d, out=old.clone(), accumulate=True, **seg(lists)),
                       torch.where(none.cuda(), old, old + got))
    old = old.half()
    assert torch.equal(moe.moe_gemm_wgrad(*d, out=old.clone(), accumulate=True, **seg(lists)),
                       torch.where(none.cuda(), old, (old.float() + got).half()))


@pytest.mark.parametrize("n", [1, 2, 3, 5, 7, 9, 15, 129, 255])
def test_rows_that_end_inside_a_piece(n):
    # columns that are no whole eights, around the ends of stages; whole numbers, so that the sums are exact
    say(f"weight gradient of {n} columns")
    g = torch.Generator().manual_seed(n)
    for rows in (1, 7, 8, 63, 64, 65, 66, 71, 72, 73, 127, 128, 129, 136, 200):
        dy = torch.randint(-8, 9, (rows, n), generator=g).half()
        codes = torch.randint(0x38, 0x40, (rows, 64), generator=g).to(torch.uint8)
        sf = torch.full((rows, 2), 127, dtype=torch.uint8)
        want = torch.from_numpy(lu.f64(dy).T @ lu.E4M3[codes.numpy()]).float()
        assert torch.equal(moe.moe_gemm_wgrad(dy.cuda(), codes.cuda(), sf.cuda()).cpu(), want), rows
        off = torch.tensor([0, rows // 3, rows // 3, rows], dtype=torch.int32).cuda()
        got = moe.moe_gemm_wgrad(dy.cuda(), codes.cuda(), sf.cuda(), offsets=off).cpu()
        assert torch.equal(got[0] + got[2], want) and torch.all(got[1] == 0), rows


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32], ids=str)
def test_accumulation_at_odd_addresses_and_edges(out):
    say(f"weight gradient added to {out}")
    for R, n, k in ((40, 5, 32), (70, 131, 96), (300, 300, 288)):
        dy, codes, sf, _ = make((R, 0, n, k, 1), torch.bfloat16, 1, 8)
        d = (dy.cuda(), codes.cuda(), sf.cuda())
        got = moe.moe_gemm_wgrad(*d)
        buf = torch.full((n * k + 2,), 7.0, dtype=out, device="cuda")
        buf[1:-1].normal_()
        old = buf.clone()
        moe.moe_gemm_wgrad(*d, out=buf[1:-1].view(n, k), accumulate=True)
        assert torch.equal(buf[1:-1].view(n, k), (old[1:-1].view(n, k).float() + got).to(out))
        assert buf[0] == 7 and buf[-1] == 7


def test_widest_stride():
    # 130 rows 2^24 elements apart: stages that span all but 2^31 bytes
    say("weight gradient of rows 32 MB apart")
    for n in (40, 37):
        dy, codes, sf, _ = make((130, 0, n, 64, 1), torch.bfloat16, 1, 6)
        far = torch.empty(129 * (1 << 24) + n, dtype=torch.bfloat16, device="cuda").as_strided((130, n), (1 << 24, 1))
        far.copy_(dy)
        assert torch.equal(moe.moe_gemm_wgrad(far, codes.cuda(), sf.cuda()), moe.moe_gemm_wgrad(dy.cuda(), codes.cuda(), sf.cuda()))
    del far
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n,k", [((1 << 20) - 1, 32), (3, 1 << 20)])
def test_widest_matrices(n, k):
    say(f"weight gradient {n} x {k}")
    g = torch.Generator().manual_seed(7)
    dy = torch.randint(-8, 9, (2, n), generator=g).bfloat16().cuda()
    codes = torch.randint(0x30, 0x48, (2, k), generator=g).to(torch.uint8)  # 0.5 to 3.75 in sixteenths
    sf = torch.full((2, k // 32), 127, dtype=torch.uint8, device="cuda")
    xv = torch.from_numpy(lu.E4M3).float().cuda()[codes.cuda().long()]
    got = moe.moe_gemm_wgrad(dy, codes.cuda(), sf)
    assert torch.equal(got, dy[0].float()[:, None] * xv[0] + dy[1].float()[:, None] * xv[1])  # (whole sixteenths: exact)


def test_workspace_and_refusals():
    say("weight gradient: refusals")
    dy, codes, sf, _ = (t.cuda() if isinstance(t, torch.Tensor) else t for t in make((3000, 0, 50, 128, 1), torch.bfloat16, 1))
    need = moe.moe_gemm_wgrad_workspace_bytes(1, 3000, 50, 128)
    assert need > 0
    want = moe.moe_gemm_wgrad(dy, codes, sf)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")      # NaN, whatever it holds
    assert torch.equal(moe.moe_gemm_wgrad(dy, codes, sf, workspace=ws), want)
    with pytest.raises(moe.MoEError) as e:
        moe.moe_gemm_wgrad(dy, codes, sf, workspace=ws[:-16])
    assert e.value.code == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    off = torch.tensor([0, 3000], dtype=torch.int32, device="cuda")
    leaf = torch.zeros(50, 128, device="cuda", requires_grad=True)
    bad = [lambda: moe.moe_gemm_wgrad(dy.float(), codes, sf), lambda: moe.moe_gemm_wgrad(dy.t(), codes, sf),
           lambda: moe.moe_gemm_wgrad(dy[1:], codes, sf), lambda: moe.moe_gemm_wgrad(dy, codes.view(torch.int8), sf),
           lambda: moe.moe_gemm_wgrad(dy, codes, sf.float()), lambda: moe.moe_gemm_wgrad(dy, codes, sf.half()),
           lambda: moe.moe_gemm_wgrad(dy, codes, sf[:, :3]), lambda: moe.moe_gemm_wgrad(dy, codes, sf, counts=off),
           lambda: moe.moe_gemm_wgrad(dy, codes, sf, offsets=off[:1]), lambda: moe.moe_gemm_wgrad(dy, codes, sf, offsets=off.long()),
           lambda: moe.moe_gemm_wgrad(dy, codes, sf, offsets=off, counts=off), lambda: moe.moe_gemm_wgrad(dy, codes, sf, accumulate=True),
           lambda: moe.moe_gemm_wgrad(dy, codes, sf, dtype=torch.float64), lambda: moe.moe_gemm_wgrad(dy, codes, sf, out=leaf),
           lambda: moe.moe_gemm_wgrad(dy.clone().requires_grad_(), codes, sf), lambda: moe.moe_gemm_wgrad(dy, codes[0], sf),
           lambda: moe.moe_gemm_wgrad(dy, codes, sf, out=want.t())]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with torch.no_grad():
        moe.moe_gemm_wgrad(dy, codes, sf, out=leaf)
