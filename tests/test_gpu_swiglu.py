"""moe_swiglu and moe_swiglu_bwd on the GPU against plain float64 forms."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_amd as moe
import layer_util as lu
import ops_util as ou
from parity_util import say

pytestmark = pytest.mark.gpu

# rows, inner width
SHAPES = [(1, 1), (5, 7), (3, 32), (9, 96), (17, 128), (4, 130), (33, 256), (6, 1000), (130, 2048), (3, 2176), (2, 4100)]
# float32 roundings: exp(-|g|) 2 (1 ulp), 1 + e, its reciprocal 2 (1 ulp), their product, g sg, times u
STEPS = 9


def steps_of(g, dtype):
    """16-bit types: 2^x of a rounded product, |g| more roundings (of values above 2^-126, |g| < 88)."""
    return STEPS + (dtype != torch.float32) * np.minimum(abs(g), 88)


# where exp(-|g|) is subnormal (|g| > 87) a rounding is a part of no value but a step of 2^-149: one of
# exp's last place and a half each of e r and g sg, so 2^-148 in all, carried on by |g| and |u| (or |dh|)
SUB = 2.0 ** -148


def sub_of(dtype):
    """16-bit types: 2^x is zero below 2^-126, so that sg and 1 - sg may be off by that (float32: see above)."""
    return SUB if dtype == torch.float32 else 2.0 ** -126


def make(shape, dtype, seed=0):
    R, inner = shape
    g = torch.Generator().manual_seed(100 * seed + R + inner)
    gu = 3 * torch.randn(R, 2 * inner, generator=g)
    if R > 2:
        gu[1] *= 40                                           # both tails of the sigmoid
        gu[2] *= 1e-4
    dh = torch.randn(R, inner, generator=g)
    row_src = torch.arange(R, dtype=torch.int32)
    row_src[torch.rand(R, generator=g) < 0.3] = -1
    return gu.to(dtype), dh.to(dtype), row_src, torch.tensor([0, max(0, R - R // 4)], dtype=torch.int32)


def live_rows(row_src, offsets):
    return ((row_src >= 0) & (torch.arange(row_src.numel()) < offsets[-1])).numpy()


@pytest.mark.parametrize("dtype", list(lu.DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_activation_against_the_plain_form(shape, dtype):
    say(f"swiglu {shape} {dtype}")
    dt = lu.DT[dtype]
    R, inner = shape
    gu, _, row_src, offsets = make(shape, dt)
    live = live_rows(row_src, offsets)
    masked = gu.clone()
    masked[torch.from_numpy(~live)] = float("nan")            # not read
    for clamp in (0.0, 2.5):
        want = lu.swiglu(lu.f64(gu), clamp)
        g64, u64 = np.split(np.clip(lu.f64(gu), -clamp, clamp) if clamp else lu.f64(gu), 2, 1)
        bound = steps_of(g64, dt) * lu.U32 * abs(want) + sub_of(dt) * (1 + abs(g64)) * abs(u64)
        h, *none = moe.moe_swiglu(gu.cuda(), clamp=clamp)
        assert none == [None] * 4
        lu.within(h, lu.overflowed(want, dt), lu.rounded_bound(want, bound, dt))
        before = torch.full((R, inner), 7.0, dtype=dt, device="cuda")
        got = moe.moe_swiglu(masked.cuda(), row_src.cuda(), offsets.cuda(), clamp=clamp, h=before)[0]
        assert got is before and torch.all(got[~live] == 7) and torch.equal(got[live], h[live])
        for fmt in (moe.MOE_SF_F32_128, moe.MOE_SF_UE8M0_32):
            kw = dict(clamp=clamp, sf_format=fmt, need_h8=True, need_gu8=True)
            if inner % lu.BLOCK[fmt]:
                with pytest.raises(moe.MoEError):
                    moe.moe_swiglu(gu.cuda(), **kw)
                continue
            h2, hc, hsf, gc, gsf = moe.moe_swiglu(gu.cuda(), **kw)
            assert torch.equal(h2, h)
            # (16-bit types: what 2^x loses at |g| > 16 is of values below 2^-19 of what else the block holds; all of it
            # counted, a code's value is off by a step's 2^-17)
            lu.near_codes(hc, hsf, want, (STEPS if dtype == "f32" else STEPS + 88) * lu.U32, fmt)
            lu.same_codes(gc, gsf, gu, fmt)                   # the copy is of the input, not clamped
            if dtype == "f32":
                lu.same_codes(hc, hsf, h, fmt)
            # one output alone, rows without a slot left as they were
            u8 = lambda cols: torch.full((R, cols), 5, dtype=torch.uint8, device="cuda")
            sf = lambda like: torch.full_like(like, 3)
            a, c1, s1, c2, s2 = moe.moe_swiglu(masked.cuda(), row_src.cuda(), offsets.cuda(), need_h=False, h_codes=u8(inner),
                                               h_sf=sf(hsf), **{**kw, "need_gu8": False})
            assert a is None and c2 is None and s2 is None
            b, n1, n2, c2, s2 = moe.moe_swiglu(masked.cuda(), row_src.cuda(), offsets.cuda(), need_h=False,
                                               gu_codes=u8(2 * inner), gu_sf=sf(gsf), **{**kw, "need_h8": False})
            assert b is None and n1 is None and n2 is None
            for t, full, old in ((c1, hc, 5), (s1, hsf, 3), (c2, gc, 5), (s2, gsf, 3)):
                assert torch.equal(t[live], full[live]) and torch.all(t[~live] == old)


@pytest.mark.parametrize("dtype", list(lu.DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradient_against_the_formula(shape, dtype):
    say(f"swiglu gradient {shape} {dtype}")
    dt = lu.DT[dtype]
    R, inner = shape
    gu, dh, row_src, offsets = make(shape, dt, 1)
    live = live_rows(row_src, offsets)
    inputs = [dict(gu=gu.cuda())]
    values = [lu.f64(gu)]
    for fmt in (moe.MOE_SF_F32_128, moe.MOE_SF_UE8M0_32):
        if inner % lu.BLOCK[fmt] == 0:
            codes, sf = lu.quantised(gu, fmt)
            inputs.append(dict(gu_codes=codes.cuda(), gu_sf=sf.cuda()))
            values.append(lu.read(codes, sf))
    for kw, v in zip(inputs, values):
        for clamp in (0.0, 2.5):
            got = moe.moe_swiglu_bwd(dh.cuda(), clamp=clamp, **kw)
            if clamp > 0:                                     # (a code's float32 value may be a rounding off the bound)
                v = np.where(abs(abs(v) - clamp) <= 2 * lu.U32 * clamp, np.copysign(clamp, v), v)
            want, mag = lu.swiglu_grads(lu.f64(dh), v, clamp)
            # the float32 value of a code with a float32 scale, and its way through the sigmoid: |g| of them
            half = np.split(v, 2, 1)[0]
            steps = np.tile(steps_of(half, dt), 2) + 6 + (0 if "gu" in kw else 2 + np.tile(abs(half), 2))
            d64, (g64, u64) = lu.f64(dh), np.split(np.clip(v, -clamp, clamp) if clamp else v, 2, 1)
            sub = sub_of(dt) * abs(np.concatenate([d64 * u64, d64], 1)) * np.tile(1 + abs(g64), 2)
            lu.within(got, lu.overflowed(want, dt), lu.rounded_bound(want, steps * lu.U32 * mag + sub, dt))
            before = torch.full((R, 2 * inner), 7.0, dtype=dt, device="cuda")
            part = moe.moe_swiglu_bwd(dh.cuda(), row_src=row_src.cuda(), offsets=offsets.cuda(), clamp=clamp, out=before, **kw)
            assert part is before and torch.equal(part[live], got[live]) and torch.all(part[~live] == 7)
    onto = gu.cuda()                                          # in place
    assert moe.moe_swiglu_bwd(dh.cuda(), gu=onto, out=onto) is onto
    assert torch.equal(onto, moe.moe_swiglu_bwd(dh.cuda(), gu=gu.cuda()))


def test_gradient_against_differences():
    say("swiglu gradient by differences")
    g = torch.Generator().manual_seed(2)
    gu, dh, v = (torch.randn(4, n, generator=g) for n in (60, 30, 60))
    got = moe.moe_swiglu_bwd(dh.cuda(), gu=gu.cuda()).double().cpu()
    h = 2.0 ** -10
    loss = lambda x: (lu.swiglu(lu.f64(x)) * lu.f64(dh)).sum()
    slope = (loss(gu.double() + h * v.double()) - loss(gu.double() - h * v.double())) / (2 * h)
    # third derivatives of silu(g) u along v stay below 12 of the slope's size here, h^2 = 2^-20
    assert abs((got * v).sum().item() - slope) <= 2.0 ** -16 * (got * v).abs().sum().item()


def test_codes_are_those_of_the_activation_quantiser():
    say("swiglu: the library's own quantiser")
    R, inner = 40, 256
    gu = make((R, inner), torch.bfloat16)[0].cuda()
    for recipe, fmt in ((moe.MOE_RECIPE_FP8_BLOCK128, 0), (moe.MOE_RECIPE_MXFP4, 1)):
        plan = moe.moe_plan_create(2 * inner, 128, 4, 2, R, recipe=recipe)
        _, _, _, codes, sf = moe.moe_swiglu(gu, need_h=False, need_gu8=True, sf_format=fmt)
        x, x_sf = torch.empty_like(codes), torch.empty_like(sf)
        moe.moe_quantize_act(plan, R, gu, x, x_sf)
        assert torch.equal(codes, x) and torch.equal(sf, x_sf)
        moe.moe_plan_destroy(plan)


def test_special_values():
    say("swiglu: infinities, NaN, tails")
    nan, inf = float("nan"), float("inf")
    g = torch.tensor([[200.0, -200.0, 95.0, -95.0, inf, nan, 0.0, -0.0]], device="cuda")
    u = torch.tensor([[2.0, 2.0, nan, 1.0, 1.0, 1.0, 3.0, inf]], device="cuda")
    h = moe.moe_swiglu(torch.cat([g, u], 1))[0][0]
    assert h[0] == 400 and h[1] == 0 and torch.isnan(h[2]) and 0 <= -h[3] < 1e-38 and h[4] == inf
    assert torch.isnan(h[5]) and h[6] == 0 and torch.isnan(h[7])
    h = moe.moe_swiglu(torch.cat([g, u], 1), clamp=5.0)[0][0]   # a clamp passes NaN on
    assert torch.isnan(h[2]) and torch.isnan(h[5]) and torch.isfinite(h[[0, 1, 3, 4, 6, 7]]).all()
    d = moe.moe_swiglu_bwd(torch.ones(1, 8, device="cuda"), gu=torch.cat([g, u], 1), clamp=5.0)[0]
    assert torch.all(d[[0, 1, 2, 3, 4]] == 0) and torch.isnan(d[5]) and d[15] == 0
    # scale codes 0xFF and 0 of a copy: NaN, and 2^-127
    codes = torch.full((2, 64), 0x38, dtype=torch.uint8, device="cuda")
    sf = torch.tensor([[255, 127], [0, 127]], dtype=torch.uint8, device="cuda")
    d = moe.moe_swiglu_bwd(torch.ones(2, 32, device="cuda"), gu_codes=codes, gu_sf=sf)
    assert torch.isnan(d[0]).all() and torch.all(d[1, :32] == 0.5) and torch.all(d[1, 32:].abs() <= 2.0 ** -127)


def test_strides_and_empty():
    say("swiglu strides")
    R, inner, dt = 21, 77, torch.float16
    gu, dh, row_src, offsets = make((R, inner), dt)

    def inside(t, pad, first):
        big = torch.full((R, t.shape[1] + pad), 99.0, dtype=dt, device="cuda")
        big[:, first:first + t.shape[1]] = t.cuda()
        return big[:, first:first + t.shape[1]], big

    out, big = inside(dh, 4, 3)
    moe.moe_swiglu(inside(gu, 5, 1)[0], h=out)
    assert torch.equal(out, moe.moe_swiglu(gu.cuda())[0])
    assert torch.all(big[:, :3] == 99) and torch.all(big[:, 3 + inner:] == 99)
    out, big = inside(gu, 3, 1)
    moe.moe_swiglu_bwd(inside(dh, 1, 1)[0], gu=inside(gu, 5, 2)[0], out=out)
    assert torch.equal(out, moe.moe_swiglu_bwd(dh.cuda(), gu=gu.cuda()))
    assert torch.all(big[:, :1] == 99) and torch.all(big[:, 1 + 2 * inner:] == 99)
    e = torch.empty(0, 64, device="cuda")
    assert moe.moe_swiglu(e)[0].shape == (0, 32) and moe.moe_swiglu_bwd(e[:, :32].contiguous(), gu=e).shape == (0, 64)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")   # no row in use; and more named than there are
    h = torch.full((R, inner), 7.0, dtype=dt, device="cuda")
    assert torch.all(moe.moe_swiglu(gu.cuda(), offsets=zero, h=h)[0] == 7)
    assert torch.equal(moe.moe_swiglu(gu.cuda(), offsets=zero + 1000, h=h)[0], moe.moe_swiglu(gu.cuda())[0])


def test_pool_past_32_bit_offsets():
    R, inner = (1 << 20) + 7, 2048                            # 8.6 GB of gate and up
    say(f"swiglu of {R} x {inner}")
    gu = torch.zeros(R, 2 * inner, dtype=torch.bfloat16, device="cuda")
    gu[-100:].normal_()
    h, hc, hsf, gc, gsf = moe.moe_swiglu(gu, need_h8=True, need_gu8=True, sf_format=1)
    part = moe.moe_swiglu(gu[-100:].clone(), need_h8=True, need_gu8=True, sf_format=1)
    for a, b in zip((h, hc, hsf, gc, gsf), part):
        assert torch.equal(a[-100:], b)
    want = moe.moe_swiglu_bwd(part[0], gu_codes=part[3], gu_sf=part[4])
    assert torch.equal(moe.moe_swiglu_bwd(h, gu_codes=gc, gu_sf=gsf, out=gu)[-100:], want)
    del gu, h, hc, gc
    torch.cuda.empty_cache()


def test_widest_rows():
    test_activation_against_the_plain_form((3, (1 << 23) - 128), "bf16")
    test_gradient_against_the_formula((1, (1 << 23) - 1), "f16")


def test_binding_refusals():
    gu, dh = torch.randn(4, 256, device="cuda"), torch.randn(4, 128, device="cuda")
    codes, sf = torch.zeros(4, 256, dtype=torch.uint8, device="cuda"), torch.zeros(4, 8, dtype=torch.uint8, device="cuda")
    leaf = gu.clone().requires_grad_()
    bad = [lambda: moe.moe_swiglu(gu.double()), lambda: moe.moe_swiglu(gu[:, :255]), lambda: moe.moe_swiglu(gu.t()),
           lambda: moe.moe_swiglu(leaf), lambda: moe.moe_swiglu(gu, h=gu), lambda: moe.moe_swiglu(gu, need_h8=True),
           lambda: moe.moe_swiglu(gu, need_gu8=True, sf_format=1, gu_sf=sf.float()),
           lambda: moe.moe_swiglu(gu, row_src=torch.zeros(3, dtype=torch.int32, device="cuda")),
           lambda: moe.moe_swiglu_bwd(dh), lambda: moe.moe_swiglu_bwd(dh, gu=gu, gu_codes=codes, gu_sf=sf),
           lambda: moe.moe_swiglu_bwd(dh, gu_codes=codes), lambda: moe.moe_swiglu_bwd(dh, gu_codes=codes, gu_sf=sf.half()),
           lambda: moe.moe_swiglu_bwd(dh, gu_codes=codes, gu_sf=sf.float()), lambda: moe.moe_swiglu_bwd(dh, gu=gu.half()),
           lambda: moe.moe_swiglu_bwd(dh, gu=leaf), lambda: moe.moe_swiglu_bwd(dh, gu=gu, out=leaf)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: moe.moe_swiglu(gu, need_h=False), lambda: moe.moe_swiglu(gu, h=gu[:, :128]),
              lambda: moe.moe_swiglu_bwd(gu[:, :128], gu=gu, out=gu)):
        with pytest.raises(moe.MoEError):
            f()
