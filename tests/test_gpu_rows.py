"""moe_permute, moe_unpermute and their gradients on the GPU against plain
float64 forms.  Copies have to be equal; a sum of n float32 terms may be off
by n roundings of its magnitudes' sum, and its result by one rounding to the
output type."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_amd as moe
import ops_util as ou
from parity_util import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# tokens, slots, width, experts, alignment, masked share
SHAPES = [
    (1, 1, 1, 1, 1, 0.0), (1, 6, 64, 8, 16, 0.0), (3, 2, 7, 5, 4, 0.3), (17, 3, 8, 16, 1, 0.0),
    (5, 9, 17, 12, 3, 0.2), (33, 8, 130, 8, 16, 0.1), (64, 4, 256, 4, 64, 0.5),
    (20, 5, 515, 9, 8, 0.1), (9, 2, 2048, 3, 2, 0.0), (6, 4, 4097, 7, 5, 0.25),
    (130, 6, 24, 40, 16, 1.0), (257, 1, 40, 30, 1, 0.05), (2, 13, 1000, 13, 160, 0.1),
]


def make(shape, dtype, seed=0):
    T, K, W, E, align, masked = shape
    rng = np.random.default_rng(1000 * seed + T + K + W)
    idx = ou.draw_idx(rng, T, K, E, masked)
    if T > 2:
        idx[1] = -1                                   # a token with no slot
    lists = ou.route(idx, E, align)
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(dtype)
    w = torch.from_numpy(rng.random((T, K)).astype(np.float32))
    return lists, ou.dev(lists), draw, w


def f64(t):
    return t.double().cpu().numpy()


def same(got, want):
    assert np.array_equal(f64(got), want, equal_nan=True)


def check_sums(got, exact, mag, terms, dtype):
    off = abs(f64(got) - exact)
    inner = terms * ou.U32 * mag
    bound = inner + ou.half_step(dtype) * (abs(exact) + inner) + ou.least(dtype)
    assert np.all(off <= bound), float((off / np.maximum(bound, 1e-300)).max())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rows_against_plain_forms(shape, dtype):
    say(f"rows {shape} {dtype}")
    dt = DT[dtype]
    T, K, W, E, align, masked = shape
    lists, d, draw, w = make(shape, dt)
    R = lists["pool"]
    x, before = draw(T, W), draw(R, W)
    got = moe.moe_permute(x.cuda(), d["row_src"], d["src_row"], d["offsets"], out=before.cuda())
    same(got, ou.permute(f64(x), lists, f64(before)))
    # rows no slot names are not read: NaN there and in masked weights
    yp = draw(R, W)
    yp[torch.from_numpy(lists["row_src"]) < 0] = float("nan")
    wm = w.clone()
    wm.view(-1)[torch.from_numpy(lists["src_row"]) < 0] = float("nan")
    ypd, wd = yp.cuda(), wm.cuda()
    got = moe.moe_permute_bwd(ypd, d["src_row"], T)
    check_sums(got, *ou.token_sums(f64(yp), lists, T), K, dt)
    got = moe.moe_unpermute(ypd, d["src_row"], T, wd)
    check_sums(got, *ou.token_sums(f64(yp), lists, T, f64(wm)), K, dt)
    got = moe.moe_unpermute(ypd, d["src_row"], T)
    check_sums(got, *ou.token_sums(f64(yp), lists, T), K, dt)
    dy = draw(T, W)
    dyp, dw = moe.moe_unpermute_bwd(dy.cuda(), ypd, d["row_src"], d["src_row"], d["offsets"], wd,
                                    dyp=before.cuda())
    edyp, edw, mag = ou.unpermute_grads(f64(dy), f64(yp), lists, f64(wm), f64(before))
    # one float32 product rounded to the type: dyp within half a step of the product's half step
    check_sums(dyp, edyp, abs(edyp), 1, dt)
    # each lane sums at most W / 64 + 8 products, then 6 levels of a tree
    assert np.all(abs(f64(dw) - edw) <= (W / 64 + 8 + 6) * ou.U32 * mag)
    # either gradient alone has the same bits
    a, none = moe.moe_unpermute_bwd(dy.cuda(), None, d["row_src"], d["src_row"], d["offsets"], wd,
                                    dyp=before.cuda(), need_dw=False)
    assert none is None and torch.equal(a.view(torch.uint8), dyp.view(torch.uint8))
    none, b = moe.moe_unpermute_bwd(dy.cuda(), ypd, d["row_src"], d["src_row"], d["offsets"], wd,
                                    need_dyp=False)
    assert none is None and torch.equal(b, dw)


@pytest.mark.parametrize("width", [1, 3, 15, 16, 17, 64, 224, 1001])
def test_permute_bytes(width):
    lists, d, _, _ = make((19, 3, width, 6, 8, 0.2), torch.float32)
    rng = np.random.default_rng(width)
    x = torch.from_numpy(rng.integers(0, 256, (19, width)).astype(np.uint8))
    before = torch.full((lists["pool"], width), 7, dtype=torch.uint8)
    got = moe.moe_permute(x.cuda(), d["row_src"], d["src_row"], d["offsets"], out=before.cuda())
    same(got, ou.permute(f64(x), lists, f64(before)))


@pytest.mark.parametrize("dtype", list(DT))
def test_row_strides_and_odd_addresses(dtype):
    dt = DT[dtype]
    T, K, W = 21, 3, 77
    lists, d, draw, w = make((T, K, W, 5, 4, 0.1), dt)
    R = lists["pool"]

    def inside(t, pad, first):
        """t's values as the columns first .. of a wider matrix, and that matrix."""
        big = torch.full((t.shape[0], t.shape[1] + pad), 99.0, dtype=dt, device="cuda")
        big[:, first:first + t.shape[1]] = t.cuda()
        return big[:, first:first + t.shape[1]], big

    x, yp, dy, before = draw(T, W), draw(R, W), draw(T, W), draw(R, W)
    xs, _ = inside(x, 5, 1)
    out, big = inside(before, 7, 3)
    moe.moe_permute(xs, d["row_src"], d["src_row"], d["offsets"], out=out)
    same(out, ou.permute(f64(x), lists, f64(before)))
    assert torch.all(big[:, :3] == 99) and torch.all(big[:, 3 + W:] == 99)
    ys, _ = inside(yp, 3, 2)
    out, big = inside(dy, 9, 1)
    moe.moe_unpermute(ys, d["src_row"], T, w.cuda(), out=out)
    check_sums(out, *ou.token_sums(f64(yp), lists, T, f64(w)), K, dt)
    assert torch.all(big[:, :1] == 99) and torch.all(big[:, 1 + W:] == 99)
    ds, _ = inside(dy, 1, 1)
    out, big = inside(before, 2, 1)
    _, dw = moe.moe_unpermute_bwd(ds, ys, d["row_src"], d["src_row"], d["offsets"], w.cuda(), dyp=out)
    edyp, edw, mag = ou.unpermute_grads(f64(dy), f64(yp), lists, f64(w), f64(before))
    check_sums(out, edyp, abs(edyp), 1, dt)
    assert np.all(abs(f64(dw) - edw) <= (W / 64 + 14) * ou.U32 * mag)
    assert torch.all(big[:, :1] == 99) and torch.all(big[:, 1 + W:] == 99)


def test_gradients_are_the_adjoints_and_match_differences():
    # whole numbers small enough that float32 holds every sum exactly
    T, K, W, E = 40, 4, 96, 11
    rng = np.random.default_rng(3)
    lists = ou.route(ou.draw_idx(rng, T, K, E, 0.2), E, 8)
    d = ou.dev(lists)
    R = lists["pool"]
    whole = lambda *s: torch.from_numpy(rng.integers(-8, 9, s).astype(np.float32)).cuda()
    routed = (d["row_src"] >= 0)[:, None]
    x, g, yp, dy, w = whole(T, W), whole(R, W), whole(R, W), whole(T, W), whole(T, K)
    fwd = lambda v: moe.moe_permute(v, d["row_src"], d["src_row"], d["offsets"], out=torch.zeros(R, W, device="cuda"))
    dx = moe.moe_permute_bwd(g, d["src_row"], T)
    assert (fwd(x) * g).sum().item() == (x * dx).sum().item()
    back = lambda p, v: moe.moe_unpermute(p, d["src_row"], T, v)
    dyp, dw = moe.moe_unpermute_bwd(dy, yp, d["row_src"], d["src_row"], d["offsets"], w,
                                    dyp=torch.zeros(R, W, device="cuda"))
    # differences along whole directions: the maps are linear in each argument
    p, v = whole(R, W) * routed, whole(T, K)
    loss = lambda q, u: (back(q, u).double() * dy.double()).sum().item()
    assert loss(yp + p, w) - loss(yp - p, w) == 2 * (dyp.double() * p.double()).sum().item()
    assert loss(yp, w + v) - loss(yp, w - v) == 2 * (dw.double() * v.double()).sum().item()


def test_the_planner_lists_and_a_cut_list():
    # moe_route's own lists, and entries out of range (skipped, not followed)
    T, K, E, W, align = 300, 4, 32, 72, 16
    rng = np.random.default_rng(5)
    idx = ou.draw_idx(rng, T, K, E, 0.1)
    lists = ou.route(idx, E, align)
    R = lists["pool"]
    plan = moe.moe_plan_create(256, 128, E, K, T)
    new = lambda n: torch.full((n,), -7, dtype=torch.int32, device="cuda")
    counts, offsets, row_src, src_row = new(E), new(E + 1), new(R), new(T * K)
    ws = torch.empty(moe.moe_route_workspace_bytes(plan, T), dtype=torch.uint8, device="cuda")
    moe.moe_route(plan, T, torch.from_numpy(idx.astype(np.int32)).cuda(), align, counts, offsets,
                  row_src, src_row, ws)
    for got, want in ((counts, "counts"), (offsets, "offsets"), (row_src, "row_src"), (src_row, "src_row")):
        assert np.array_equal(got.cpu().numpy(), lists[want]), want
    moe.moe_plan_destroy(plan)
    x = torch.from_numpy(rng.standard_normal((T, W))).float()
    before = torch.full((R, W), 5.0)
    got = moe.moe_permute(x.cuda(), row_src, src_row, offsets, out=before.cuda())
    same(got, ou.permute(f64(x), lists, f64(before)))
    # slots 3 and 8 point past the pool, pool row 0 names a slot past the last
    bad = src_row.clone()
    bad[3], bad[8] = R, 2 ** 31 - 1
    brow = row_src.clone()
    brow[0] = T * K
    cut = {**lists, "src_row": bad.cpu().numpy().copy()}
    cut["src_row"][[3, 8]] = -1
    yp = torch.from_numpy(rng.standard_normal((R, W))).float()
    got = moe.moe_unpermute(yp.cuda(), bad, T)
    check_sums(got, *ou.token_sums(f64(yp), cut, T), K, torch.float32)
    got = moe.moe_permute(x.cuda(), brow, bad, offsets, out=before.cuda())
    assert got.shape == (R, W) and torch.isfinite(got).all()
    _, dw = moe.moe_unpermute_bwd(x.cuda(), yp.cuda(), brow, bad, offsets)
    assert dw.view(-1)[3] == 0 and dw.view(-1)[8] == 0


def test_a_token_that_names_an_expert_twice():
    T, K, E, W = 12, 4, 3, 50
    rng = np.random.default_rng(9)
    idx = rng.integers(0, E, (T, K))
    idx[3] = 1
    lists = ou.route(idx, E, 4)
    d = ou.dev(lists)
    x = torch.from_numpy(rng.standard_normal((T, W)).astype(np.float32))
    before = torch.zeros(lists["pool"], W)
    xp = moe.moe_permute(x.cuda(), d["row_src"], d["src_row"], d["offsets"], out=before.cuda())
    same(xp, ou.permute(f64(x), lists, f64(before)))
    w = torch.from_numpy(rng.random((T, K)).astype(np.float32))
    check_sums(moe.moe_unpermute(xp, d["src_row"], T, w.cuda()), *ou.token_sums(f64(xp), lists, T, f64(w)), K,
               torch.float32)
    dyp, dw = moe.moe_unpermute_bwd(x.cuda(), xp, d["row_src"], d["src_row"], d["offsets"], w.cuda(),
                                    dyp=before.cuda())
    edyp, edw, mag = ou.unpermute_grads(f64(x), f64(xp), lists, f64(w), f64(before))
    check_sums(dyp, edyp, abs(edyp), 1, torch.float32)
    assert np.all(abs(f64(dw) - edw) <= (W / 64 + 14) * ou.U32 * mag)


def test_no_tokens_and_all_masked():
    e = torch.empty(0, 32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    row_src = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    got = moe.moe_permute(e, row_src, none, offsets, out=torch.full((6, 32), 3.0, device="cuda"))
    assert torch.all(got[:4] == 0) and torch.all(got[4:] == 3)
    assert moe.moe_unpermute(got, none, 0).shape == (0, 32)
    dyp, dw = moe.moe_unpermute_bwd(e, got, row_src, none, offsets, dyp=got.clone())
    assert torch.all(dyp[:4] == 0) and torch.all(dyp[4:] == 3) and dw.numel() == 0
    src_row = torch.full((10,), -1, dtype=torch.int32, device="cuda")
    x = torch.randn(5, 32, device="cuda")
    assert torch.all(moe.moe_unpermute(got, src_row, 5) == 0)
    assert torch.all(moe.moe_permute_bwd(got, src_row, 5) == 0)
    dyp, dw = moe.moe_unpermute_bwd(x, got, row_src, src_row, offsets, dyp=got.clone())
    assert torch.all(dw == 0) and torch.all(dyp[:4] == 0) and torch.all(dyp[4:] == 3)


def test_pool_past_32_bit_offsets():
    # 4.9 GB of pool rows; the routed ones are its first and last
    R, W, T, K = 600000, 4096, 2, 2
    rows = torch.tensor([R - 1, 0, -1, R - 2], dtype=torch.int32)
    row_src = torch.full((R,), 3, dtype=torch.int32)      # (other rows count as routed: not cleared)
    row_src[rows[0]], row_src[rows[1]], row_src[rows[3]] = 0, 1, 3
    d = rows.cuda()
    pool = torch.zeros(R, W, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(T, W, device="cuda").bfloat16()
    moe.moe_permute(x, row_src.cuda(), d, None, out=pool)
    assert torch.equal(pool[R - 1], x[0]) and torch.equal(pool[0], x[0]) and torch.equal(pool[R - 2], x[1])
    assert not pool[1:1000].any() and not pool[R - 1000:R - 2].any()
    y = moe.moe_unpermute(pool, d, T)
    assert torch.equal(y[0], 2 * x[0]) and torch.equal(y[1], x[1])
    w = torch.tensor([[0.5, 2.0], [3.0, 4.0]], device="cuda")
    _, dw = moe.moe_unpermute_bwd(x, pool, row_src.cuda(), d, None, w, dyp=torch.empty_like(pool))
    s = (x.double() ** 2).sum(1)
    want = torch.stack([s[0], s[0], 0 * s[1], s[1]]).view(2, 2)
    assert torch.all((dw.double() - want).abs() <= (W / 64 + 14) * ou.U32 * want)
    del pool
    torch.cuda.empty_cache()


def test_binding_refusals():
    lists, d, draw, w = make((8, 2, 64, 4, 4, 0.0), torch.float32)
    R = lists["pool"]
    x, yp, w = draw(8, 64).cuda(), draw(R, 64).cuda(), w.cuda()
    bad = [
        lambda: moe.moe_permute(x.t(), d["row_src"], d["src_row"], d["offsets"]),
        lambda: moe.moe_permute(x.double(), d["row_src"], d["src_row"], d["offsets"]),
        lambda: moe.moe_permute(x, d["row_src"].long(), d["src_row"], d["offsets"]),
        lambda: moe.moe_permute(x, d["row_src"].cpu(), d["src_row"], d["offsets"]),
        lambda: moe.moe_permute(x, d["row_src"], d["src_row"][:15], d["offsets"]),
        lambda: moe.moe_permute(x, d["row_src"], d["src_row"], d["offsets"], out=yp[1:]),
        lambda: moe.moe_permute(x, d["row_src"], d["src_row"], d["offsets"], out=yp.half()),
        lambda: moe.moe_permute(x[0], d["row_src"], d["src_row"], d["offsets"]),
        lambda: moe.moe_permute(x[:1].expand(8, 64), d["row_src"], d["src_row"], d["offsets"]),
        lambda: moe.moe_unpermute(yp, d["src_row"], 8, w.half()),
        lambda: moe.moe_unpermute(yp, d["src_row"], 8, w[:, :1]),
        lambda: moe.moe_unpermute(yp, d["src_row"], 7, w),
        lambda: moe.moe_unpermute(yp.to(torch.uint8), d["src_row"], 8),
        lambda: moe.moe_unpermute_bwd(x, yp.half(), d["row_src"], d["src_row"], d["offsets"], w),
        lambda: moe.moe_unpermute_bwd(x, yp, d["row_src"], d["src_row"], d["offsets"], w, dw=w[:4]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(moe.MoEError):                     # the output over its input
        moe.moe_permute(yp[:8], d["row_src"], d["src_row"], d["offsets"], out=yp)
    with pytest.raises(moe.MoEError):
        moe.moe_unpermute_bwd(x, None, d["row_src"], d["src_row"], d["offsets"], need_dyp=False, need_dw=False)


def test_sizes_beyond_32_bits_are_refused():
    # (their low 32 bits alone would name a small call that fits)
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = torch.empty(1, (1 << 32) + 32, dtype=torch.uint8, device="cuda")
    half = wide.view(torch.float16)
    u = torch.zeros(1, 16, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(1, 1, dtype=torch.uint8, device="cuda")
    for f in (lambda: moe.moe_permute(wide, i, i, None), lambda: moe.moe_permute_bwd(half, i, 1),
              lambda: moe.moe_quantize_mxfp4(half), lambda: moe.moe_dequantize_mxfp4(wide, sf),
              lambda: moe.moe_gemm_mxfp4(wide[:, :-16], sf, u, sf),
              lambda: moe.moe_gemm_mxfp4(u, sf, wide.view(-1, 16), sf),
              lambda: moe.moe_gemm_mxfp4(u, sf, u[None], sf[None], offsets=torch.cat([i, i]), slots=(1 << 32) + 1)):
        with pytest.raises((ValueError, moe.MoEError)) as e:
            f()
        print(e.value)
    del wide, half
    torch.cuda.empty_cache()
