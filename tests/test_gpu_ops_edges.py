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


# Launches of 2^32 threads and more, whose workgroups go on along the grid's y axis.

def done(*tensors):
    for t in tensors:
        t.untyped_storage().resize_(0)
    torch.cuda.empty_cache()


def test_padding_of_the_largest_pool():
    R = (1 << 28) - 1                                         # 2^24 workgroups look for padding
    say(f"padding of {R} pool rows")
    rows = [R - 1, 0, 1 << 27, -1, 5, R - 2]                  # of 3 tokens, top-2
    src_row, row_src = ints(*rows), torch.full((R,), -1, dtype=torch.int32, device="cuda")
    for f, r in enumerate(rows):
        if r >= 0:
            row_src[r] = f
    x = torch.tensor([[11], [22], [33]], dtype=torch.uint8, device="cuda")
    xp = torch.full((R, 1), 7, dtype=torch.uint8, device="cuda")
    moe.moe_permute(x, row_src, src_row, None, out=xp)
    want = torch.zeros_like(xp)
    for f, r in enumerate(rows):
        if r >= 0:
            want[r] = x[f // 2]
    assert torch.equal(xp, want)
    done(xp, want)
    dy, yp = torch.tensor([[2.0], [4.0], [8.0]], device="cuda").bfloat16(), torch.ones(R, 1, device="cuda").bfloat16()
    dyp = torch.full_like(yp, 7.0)
    _, dw = moe.moe_unpermute_bwd(dy, yp, row_src, src_row, None, dyp=dyp)
    for f, r in enumerate(rows):
        assert dw.view(-1)[f] == (dy[f // 2] if r >= 0 else 0)
        if r >= 0:
            assert dyp[r] == dy[f // 2]
            dyp[r] = 0
    assert not dyp.any()
    done(yp, dyp, row_src)


def test_sums_of_the_most_tokens():
    T, W = 1 << 23, 1028                                      # two workgroups a token: 2^24
    say(f"sums of {T} tokens of {W} f32")
    pool = torch.randn(3, W, device="cuda")
    src_row = (torch.arange(T, device="cuda") * 7 % 4 - 1).int()        # every fourth is masked
    y = moe.moe_unpermute(pool, src_row, T)
    rows = torch.cat([torch.zeros(1, W, device="cuda"), pool])
    for at in range(0, T, T // 8):
        s = slice(at, at + T // 8)
        assert torch.equal(y[s], rows[src_row[s].long() + 1]), at
    done(y)


def test_permute_of_the_most_tokens():
    T, W, R = 1 << 23, 4100, 5
    say(f"permute {T} tokens of {W} bytes")
    x = torch.zeros(T, W, dtype=torch.uint8, device="cuda")
    src_row = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    row_src = ints(0, 1 << 22, -1, T - 1, T - 2)
    for r, f in enumerate(row_src.tolist()):
        if f >= 0:
            src_row[f] = r
            x[f] = torch.randint(0, 256, (W,), device="cuda").to(torch.uint8)
    xp = moe.moe_permute(x, row_src, src_row, None, out=torch.full((R, W), 7, dtype=torch.uint8, device="cuda"))
    for r, f in enumerate(row_src.tolist()):
        assert torch.equal(xp[r], x[f] if f >= 0 else torch.zeros_like(xp[r])), r
    done(x)


def test_quantise_the_most_rows():
    rows, cols = (1 << 29) + 77, 32                           # 32 rows a workgroup
    say(f"quantise {rows} x {cols}")
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    codes, sf = moe.moe_quantize_mxfp4(x)
    back = torch.full_like(x, float("nan"))
    moe.moe_dequantize_mxfp4(codes, sf, out=back)
    for at in (0, 1 << 28, (1 << 29) - 50, rows - 100):
        s = slice(at, at + 100)
        c, f = moe.moe_quantize_mxfp4(x[s].clone())
        assert torch.equal(codes[s], c) and torch.equal(sf[s], f), at
        assert torch.equal(back[s], moe.moe_dequantize_mxfp4(c, f)), at
    done(x, codes, sf, back)


def test_product_of_the_most_tiles():
    # one row for each of 1024 experts: 2^24 tiles and more of 32 x 128.  (One block of K: sums
    # exact in f32 whatever the tile, so each expert's row equals its own dense product's.)
    E, N, K = 1024, (1 << 21) + 129, 32
    say(f"{E} segments of one row, {N} columns")
    assert tuple(moe.moe_gemm_mxfp4_info(E, N, K, E).values()) == (32, 128)
    g = torch.Generator(device="cuda").manual_seed(3)
    u = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, device="cuda", generator=g)
    a, a_sf = u(0, 256, E, K // 2), u(120, 134, E, 1)
    b, b_sf = u(0, 256, E, N, K // 2), u(120, 134, E, N, 1)
    y = moe.moe_gemm_mxfp4(a, a_sf, b, b_sf, offsets=torch.arange(E + 1, dtype=torch.int32, device="cuda"),
                           out=torch.full((E, N), float("nan"), dtype=torch.bfloat16, device="cuda"))
    for e in (0, 1, 500, E - 2, E - 1):
        assert torch.equal(y[e:e + 1], moe.moe_gemm_mxfp4(a[e:e + 1], a_sf[e:e + 1], b[e], b_sf[e])), e
    assert not torch.isnan(y).any()
    done(b, b_sf, y)


def test_gradients_without_the_pool_list():
    T, K, W, R = 6, 2, 70, 20
    say("gradients without row_src")
    src_row = (torch.randperm(R, device="cuda")[:T * K]).int()
    src_row[3] = -1
    row_src = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    for f, r in enumerate(src_row.tolist()):
        if r >= 0:
            row_src[r] = f
    dy, yp, w = torch.randn(T, W, device="cuda"), torch.randn(R, W, device="cuda"), torch.rand(T, K, device="cuda")
    want, dw = moe.moe_unpermute_bwd(dy, yp, row_src, src_row, None, w)
    before = torch.randn(R, W, device="cuda")
    want = torch.where((row_src >= 0)[:, None], want, before)        # the padding stays
    for p in (yp, None):                                             # the pool's rows by yp, or by dyp
        got, dw2 = moe.moe_unpermute_bwd(dy, p, None, src_row, None, w, dyp=before.clone(), need_dw=p is not None)
        assert torch.equal(got, want) and (dw2 is None if p is None else torch.equal(dw2, dw))
    none, dw2 = moe.moe_unpermute_bwd(dy, yp, None, src_row, None, w, need_dyp=False)
    assert none is None and torch.equal(dw2, dw)
    new, _ = moe.moe_unpermute_bwd(dy, yp, None, src_row, None, w)
    assert torch.equal(new[row_src >= 0], want[row_src >= 0])
    for bad in (lambda: moe.moe_unpermute_bwd(dy, None, row_src, src_row, None, w),
                lambda: moe.moe_unpermute_bwd(dy, None, None, src_row, None, w, need_dw=False),
                lambda: moe.moe_unpermute_bwd(dy, yp, None, src_row, None, w, dyp=before[1:].clone()),
                lambda: moe.moe_unpermute_bwd(dy, yp[0], None, src_row, None, w)):
        with pytest.raises(ValueError):
            bad()


class Permute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, row_src, src_row, offsets):
        ctx.lists, ctx.tokens = src_row, x.shape[0]
        return moe.moe_permute(x, row_src, src_row, offsets)

    @staticmethod
    def backward(ctx, dxp):
        return moe.moe_permute_bwd(dxp, ctx.lists, ctx.tokens), None, None, None


class Unpermute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, yp, w, row_src, src_row, offsets):
        ctx.lists = row_src, src_row, offsets
        ctx.save_for_backward(yp, w)
        return moe.moe_unpermute(yp, src_row, w.shape[0], w)

    @staticmethod
    def backward(ctx, dy):
        return *moe.moe_unpermute_bwd(dy, ctx.saved_tensors[0], *ctx.lists, ctx.saved_tensors[1]), None, None, None


def test_gradients_are_not_lost_silently():
    say("tensors that require grad")
    T, W = 4, 32
    i, offsets = torch.arange(T, dtype=torch.int32, device="cuda"), ints(0, T)
    leaf = lambda *s: torch.randn(*s, device="cuda", requires_grad=True)
    x, w, plain, one = leaf(T, W), leaf(T, 1), torch.randn(T, W, device="cuda"), torch.ones(T, 1, device="cuda")
    codes, sf = moe.moe_quantize_mxfp4(x)                     # codes have no gradient
    calls = [lambda: moe.moe_permute(x, i, i, offsets), lambda: moe.moe_permute(plain, i, i, offsets, out=x),
             lambda: moe.moe_permute_bwd(x, i, T), lambda: moe.moe_permute_bwd(plain, i, T, out=x),
             lambda: moe.moe_unpermute(x, i, T), lambda: moe.moe_unpermute(plain, i, T, w),
             lambda: moe.moe_unpermute(plain, i, T, one, out=x),
             lambda: moe.moe_unpermute_bwd(x, plain, i, i, offsets),
             lambda: moe.moe_unpermute_bwd(plain, x, i, i, offsets),
             lambda: moe.moe_unpermute_bwd(plain, plain, i, i, offsets, w),
             lambda: moe.moe_unpermute_bwd(plain, plain, i, i, offsets, dyp=x),
             lambda: moe.moe_unpermute_bwd(plain, plain, i, i, offsets, dw=w),
             lambda: moe.moe_dequantize_mxfp4(codes, sf, torch.float32, out=x),
             lambda: moe.moe_gemm_mxfp4(codes, sf, codes, sf, out=leaf(T, T))]
    for n, f in enumerate(calls):
        with pytest.raises(ValueError, match="requires grad"):
            f()
        if n in (0, 2, 4, 5, 9):
            with torch.no_grad():                             # without grad mode they run
                f()
    # in autograd.Functions: rows, weighted, there and back
    y = Unpermute.apply(Permute.apply(x, i, i, offsets), w, i, i, offsets)
    dx, dw = torch.autograd.grad(y, (x, w), plain)
    assert torch.equal(dx, plain * w)
    terms = plain.double() * x.detach().double()              # a lane's products, then 6 levels of a tree
    assert torch.all((dw[:, 0] - terms.sum(1)).abs() <= (W / 64 + 14) * 2.0 ** -24 * terms.abs().sum(1))


def test_autograd_sees_writes_into_given_outputs():
    # a tensor that a graph saved and a call overwrote is refused in the backward pass
    say("outputs that autograd saved")
    T, W = 4, 32
    i, offsets = torch.arange(T, dtype=torch.int32, device="cuda"), ints(0, T)
    x, w = torch.randn(T, W, device="cuda"), torch.rand(T, 1, device="cuda")
    codes, sf = moe.moe_quantize_mxfp4(x)
    calls = [lambda o: moe.moe_permute(x, i, i, offsets, out=o), lambda o: moe.moe_permute_bwd(x, i, T, out=o),
             lambda o: moe.moe_unpermute(x, i, T, w, out=o),
             lambda o: moe.moe_unpermute_bwd(x, x, i, i, offsets, w, dyp=o),
             lambda o: moe.moe_unpermute_bwd(x, x, i, i, offsets, w, dw=o),
             lambda o: moe.moe_dequantize_mxfp4(codes, sf, torch.float32, out=o),
             lambda o: moe.moe_gemm_mxfp4(codes, sf, torch.cat([codes] * 8), torch.cat([sf] * 8), out=o)]
    for n, f in enumerate(calls):
        saved = torch.randn(T, 1 if n == 4 else W, device="cuda")
        y = (saved * torch.randn_like(saved).requires_grad_()).sum()
        f(saved)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    for given in (dict(codes=codes), dict(sf=sf), dict(codes=codes, sf=sf)):
        before = {k: v._version for k, v in given.items()}
        moe.moe_quantize_mxfp4(x, **given)
        assert all(v._version > before[k] for k, v in given.items())
    # a call that is refused, and one that writes nothing given, leave them
    before = x._version
    with pytest.raises(moe.MoEError):
        moe.moe_permute(x, i, i, offsets, out=x)
    moe.moe_permute(x, i, i, offsets)
    moe.moe_unpermute_bwd(x, x, i, i, offsets, w, dyp=x, need_dyp=False)
    assert x._version == before
    with torch.inference_mode():                              # tensors without a version
        moe.moe_permute(x, i, i, offsets, out=torch.empty(T, W, device="cuda"))
