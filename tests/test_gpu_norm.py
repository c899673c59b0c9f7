"""moe_rms_norm and moe_rms_norm_bwd on the GPU against plain float64 forms."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_amd as moe
import layer_util as lu
import ops_util as ou
from parity_util import say

pytestmark = pytest.mark.gpu

# rows, width: each kernel's widths and their edges
SHAPES = [(1, 1), (3, 7), (5, 128), (9, 511), (4, 512), (7, 515), (6, 1024), (3, 1025), (11, 1280), (5, 2048),
          (2, 2049), (130, 4096), (3, 4104), (9, 7168), (2, 8191), (3, 8320), (2, 16384), (2, 16385), (3, 20480),
          (700, 96), (301, 64), (45, 65), (1000, 200), (77, 256), (33, 257), (40000, 32), (9000, 128)]
EPS = 1e-5


def make(shape, dtype, seed=0):
    g = torch.Generator().manual_seed(1000 * seed + shape[0] + shape[1])
    rows = lambda s: (s * torch.randn(shape, generator=g)).to(dtype)
    return rows(1.0), rows(4.0), 1 + 0.2 * torch.randn(shape[1], generator=g)


def check_y(y, z64, weight, dtype):
    rstd, want = lu.norm(z64, weight, EPS)
    steps = lu.norm_steps(z64.shape[1])
    lu.within(y, want, lu.rounded_bound(want, steps * lu.U32 * abs(want), dtype))


@pytest.mark.parametrize("dtype", list(lu.DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm_against_the_plain_form(shape, dtype):
    say(f"norm {shape} {dtype}")
    dt = lu.DT[dtype]
    T, W = shape
    x, res, w = make(shape, dt)
    sums = ou.rounded(lu.f64(x) + lu.f64(res), dt)            # (of two such values the float32 sum rounds as the exact one)
    steps = lu.norm_steps(W)
    for residual in (None, res):
        for weight in (None, w.to(dt), w):
            z, rstd, y, codes, sf = moe.moe_rms_norm(x.cuda(), None if weight is None else weight.cuda(),
                                                     residual=None if residual is None else residual.cuda(), eps=EPS)
            assert codes is None and sf is None
            z64 = lu.f64(x) if residual is None else sums
            w64 = np.ones(W) if weight is None else lu.f64(weight)
            if residual is None:
                assert z is None
            else:
                assert np.array_equal(lu.f64(z), z64)
            want = lu.norm(z64, w64, EPS)[0]
            lu.within(rstd, want, steps * lu.U32 * want)
            check_y(y, z64, w64, dt)
    for fmt in (moe.MOE_SF_F32_128, moe.MOE_SF_UE8M0_32):
        if W % lu.BLOCK[fmt]:
            with pytest.raises(moe.MoEError):
                moe.moe_rms_norm(x.cuda(), sf_format=fmt)
            continue
        for need_y in (True, False):
            z, _, y, codes, sf = moe.moe_rms_norm(x.cuda(), w.cuda(), residual=res.cuda(), eps=EPS, need_y=need_y,
                                                  sf_format=fmt)
            want = lu.norm(sums, lu.f64(w), EPS)[1]
            lu.near_codes(codes, sf, want, steps * lu.U32, fmt)
            assert np.array_equal(lu.f64(z), sums) and (y is not None) == need_y
            if need_y:
                check_y(y, sums, lu.f64(w), dt)
                if dtype == "f32":                            # y is what was quantised
                    lu.same_codes(codes, sf, y, fmt)


@pytest.mark.parametrize("dtype", list(lu.DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients_against_the_formula(shape, dtype):
    say(f"norm gradient {shape} {dtype}")
    dt = lu.DT[dtype]
    T, W = shape
    z, dy, w = make(shape, dt, 1)
    dz = make(shape, dt, 2)[0]
    rstd = torch.from_numpy(lu.norm(lu.f64(z), 1.0, EPS)[0]).float()
    for other in (None, dz):
        for weight in (None, w.to(dt), w):
            args = (dy.cuda(), z.cuda(), rstd.cuda(), None if weight is None else weight.cuda())
            kw = dict(dz=None if other is None else other.cuda())
            dx, dw = moe.moe_rms_norm_bwd(*args, **kw)
            w64 = np.ones(W) if weight is None else lu.f64(weight)
            wx, mx, ww, mw = lu.norm_grads(lu.f64(dy), lu.f64(z), lu.f64(rstd), w64, 0.0 if other is None else lu.f64(dz))
            # a thread's run, the trees, five products and sums (xh, g, mean, two fused)
            steps = max(16, W / 1024 + 8) + 22 + 6
            lu.within(dx, wx, lu.rounded_bound(wx, steps * lu.U32 * mx, dt))
            # 256 workgroups of 1 to 16 rows at a time: a run over a sixteenth at least, 16 that meet; a run over 1/32 of
            # the workgroups, 32 that meet; two products
            lu.within(dw, ww, (T / 256 + 1 + 16 + 256 / 32 + 32 + 2) * lu.U32 * mw + 2.0 ** -140)
            a, none = moe.moe_rms_norm_bwd(*args, need_dw=False, **kw)
            assert none is None and torch.equal(a, dx)
            none, b = moe.moe_rms_norm_bwd(*args, need_dx=False, **kw)
            assert none is None and torch.equal(b, dw)


def test_gradients_against_differences():
    say("norm gradient by differences")
    T, W = 5, 200
    g = torch.Generator().manual_seed(4)
    x, res, w, dy, dz, v, vw = (torch.randn(s, generator=g) for s in ((T, W), (T, W), (W,), (T, W), (T, W), (T, W), (W,)))
    z, rstd, y, _, _ = moe.moe_rms_norm(x.cuda(), w.cuda(), residual=res.cuda(), eps=EPS)
    dx, dw = moe.moe_rms_norm_bwd(dy.cuda(), z, rstd, w.cuda(), dz=dz.cuda())

    def loss(x, w):
        s = lu.f64(x + res.double())
        return (lu.norm(s, lu.f64(w), EPS)[1] * lu.f64(dy)).sum() + (s * lu.f64(dz)).sum()

    h = 2.0 ** -10
    x, w = x.double(), w.double()
    for d, slope in ((dx.double().cpu() * v, loss(x + h * v.double(), w) - loss(x - h * v.double(), w)),
                     (dw.double().cpu() * vw, loss(x, w + h * vw.double()) - loss(x, w - h * vw.double()))):
        # third derivatives along v: below 6 |v|^2 / W of the slope's size, times h^2 = 2^-20; float32 z on top
        assert abs(d.sum().item() - slope / (2 * h)) <= 2.0 ** -14 * d.abs().sum().item()


@pytest.mark.parametrize("shape", [(6, 96), (9, 640), (5, 4096), (3, 8192), (3, 16512)], ids=str)
def test_in_place_and_strides(shape):
    say(f"norm in place {shape}")
    T, W = shape
    dt = torch.bfloat16
    x, res, w = (t.cuda() for t in make(shape, dt, 5))
    fmt = moe.MOE_SF_UE8M0_32
    want = moe.moe_rms_norm(x, w, residual=res, sf_format=fmt)
    for onto in ("x", "residual"):                            # z on an input, y on an input without z's way
        a, b = x.clone(), res.clone()
        got = moe.moe_rms_norm(a, w, residual=b, sf_format=fmt, z=a if onto == "x" else b)
        assert all(torch.equal(p, q) for p, q in zip(got, want)) and torch.equal(a if onto == "x" else b, want[0])
        a, b = x.clone(), res.clone()
        got = moe.moe_rms_norm(a, w, residual=b, sf_format=fmt, z=a if onto == "x" else b, y=b if onto == "x" else a)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    a = x.clone()
    assert torch.equal(moe.moe_rms_norm(a, w, y=a)[2], moe.moe_rms_norm(x, w)[2])

    def inside(t, pad, first):
        big = torch.full((T, W + pad), 99.0, dtype=dt, device="cuda")
        big[:, first:first + W] = t
        return big[:, first:first + W], big

    views = [inside(x, 3, 1)[0], inside(res, 5, 2)[0]]
    (z, zb), (y, yb) = inside(x, 7, 3), inside(x, 2, 1)
    got = moe.moe_rms_norm(views[0], w, residual=views[1], sf_format=fmt, z=z, y=y)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    for big, first in ((zb, 3), (yb, 1)):
        assert torch.all(big[:, :first] == 99) and torch.all(big[:, first + W:] == 99)
    dy, dz = torch.randn(T, W, device="cuda").to(dt), torch.randn(T, W, device="cuda").to(dt)
    dx, dw = moe.moe_rms_norm_bwd(dy, want[0], want[1], w, dz=dz)
    for onto in (0, 1):
        a, b = dy.clone(), dz.clone()
        p, q = moe.moe_rms_norm_bwd(a, want[0], want[1], w, dz=b, dx=(a, b)[onto])
        assert torch.equal(p, dx) and torch.equal(q, dw) and p is (a, b)[onto]
    out, big = inside(x, 4, 3)
    moe.moe_rms_norm_bwd(inside(dy, 1, 1)[0], inside(want[0], 3, 2)[0], want[1], w, dz=inside(dz, 9, 5)[0], dx=out)
    assert torch.equal(out, dx) and torch.all(big[:, :3] == 99) and torch.all(big[:, 3 + W:] == 99)
    # a workspace of one's own, whatever it holds
    ws = torch.full((moe.moe_rms_norm_bwd_workspace_bytes(T, W),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(moe.moe_rms_norm_bwd(dy, want[0], want[1], w, dz=dz, workspace=ws)[1], dw)
    with pytest.raises(moe.MoEError) as e:
        moe.moe_rms_norm_bwd(dy, want[0], want[1], w, workspace=ws[:-16])
    assert e.value.code == moe.MOE_ERR_WORKSPACE_TOO_SMALL


def test_empty_rows_and_special_values():
    say("norm: no rows, zeros, infinities, NaN")
    e, w = torch.empty(0, 256, device="cuda"), torch.randn(256, device="cuda")
    z, rstd, y, codes, sf = moe.moe_rms_norm(e, w, residual=e, sf_format=0)
    assert z.shape == y.shape == (0, 256) and codes.shape == (0, 256) and sf.shape == (0, 2) and rstd.shape == (0,)
    dx, dw = moe.moe_rms_norm_bwd(e, z, rstd, w, dw=torch.full((256,), 5.0, device="cuda"))
    assert dx.shape == (0, 256) and torch.all(dw == 0)
    x = torch.randn(5, 256, device="cuda")
    x[0] = 0
    x[1, 7] = float("inf")
    x[2, 9] = float("nan")
    x[3] *= 1e-20                                             # squares below float32's range: eps alone counts
    _, rstd, y, codes, sf = moe.moe_rms_norm(x, w, eps=EPS, sf_format=0)
    assert torch.all(y[0] == 0) and torch.all(codes[0] & 127 == 0) and torch.isfinite(sf[0]).all()
    assert rstd[1] == 0 and torch.isnan(y[1, 7]) and torch.isnan(rstd[2]) and torch.isnan(y[2]).all()
    assert torch.all(codes[2] & 127 == 127) and codes[1, 7] & 127 == 127
    lu.within(y[[3, 4]], lu.norm(lu.f64(x[[3, 4]]), lu.f64(w), EPS)[1],
              lu.norm_steps(256) * lu.U32 * abs(lu.norm(lu.f64(x[[3, 4]]), lu.f64(w), EPS)[1]))


def test_rows_past_32_bit_offsets():
    T, W = (1 << 20) + 3, 4096                                # 8.6 GB a matrix
    say(f"norm of {T} x {W}")
    x = torch.zeros(T, W, dtype=torch.bfloat16, device="cuda")
    x[-600:].normal_()
    x[0].normal_()
    w = torch.randn(W, device="cuda")
    z, rstd, y, codes, sf = moe.moe_rms_norm(x, w, residual=x, sf_format=1)
    s = moe.moe_rms_norm(x[-600:].clone(), w, residual=x[-600:].clone(), sf_format=1)
    for a, b in zip((z, rstd, y, codes, sf), s):
        assert torch.equal(a[-600:], b)
    del y, codes
    dx, dw = moe.moe_rms_norm_bwd(x, z, rstd, w, dx=x.clone())
    a, _ = moe.moe_rms_norm_bwd(x[-600:].clone(), s[0], s[1], w)
    assert torch.equal(dx[-600:], a)
    rows = torch.cat([x[:1], x[-600:]]).double() * torch.cat([z[:1], z[-600:]]).double() * torch.cat([rstd[:1], rstd[-600:]])[:, None]
    bound = (T / 256 + 1 + 16 + 8 + 32 + 2) * lu.U32 * rows.abs().sum(0)
    assert torch.all((dw.double() - rows.sum(0)).abs() <= bound)
    del x, z, dx
    torch.cuda.empty_cache()


def test_widest_rows():
    T, W = 2, (1 << 24) - 1
    say(f"norm of {T} x {W}")
    z, dy, w = make((T, W), torch.bfloat16, 3)
    _, rstd, y, _, _ = moe.moe_rms_norm(z.cuda(), w.cuda(), eps=EPS)
    want = lu.norm(lu.f64(z), 1.0, EPS)[0]
    lu.within(rstd, want, lu.norm_steps(W) * lu.U32 * want)
    check_y(y, lu.f64(z), lu.f64(w), torch.bfloat16)
    r = torch.from_numpy(want).float()
    dx, dw = moe.moe_rms_norm_bwd(dy.cuda(), z.cuda(), r.cuda(), w.cuda())
    wx, mx, ww, mw = lu.norm_grads(lu.f64(dy), lu.f64(z), lu.f64(r), lu.f64(w), 0.0)
    # as for the narrower rows: a thread's run, the trees, five products and sums; for dw two products and the rows' sum
    lu.within(dx, wx, lu.rounded_bound(wx, (W / 1024 + 8 + 22 + 6) * lu.U32 * mx, torch.bfloat16))
    lu.within(dw, ww, 4 * lu.U32 * mw + 2.0 ** -140)


def test_binding_refusals():
    x, w, r = torch.randn(4, 64, device="cuda"), torch.randn(64, device="cuda"), torch.ones(4, device="cuda")
    leaf = x.clone().requires_grad_()
    bad = [lambda: moe.moe_rms_norm(x.double()), lambda: moe.moe_rms_norm(x.t()), lambda: moe.moe_rms_norm(x, w[:63]),
           lambda: moe.moe_rms_norm(x, w.half()), lambda: moe.moe_rms_norm(x, w.cpu()), lambda: moe.moe_rms_norm(x, z=x),
           lambda: moe.moe_rms_norm(x, residual=x[:3]), lambda: moe.moe_rms_norm(x, residual=x.half()),
           lambda: moe.moe_rms_norm(x, sf_format=2), lambda: moe.moe_rms_norm(x, sf_format=1, sf=torch.zeros(4, 2, device="cuda")),
           lambda: moe.moe_rms_norm(leaf), lambda: moe.moe_rms_norm(x, w.clone().requires_grad_()),
           lambda: moe.moe_rms_norm(x, y=leaf), lambda: moe.moe_rms_norm(x, rstd=r.half()),
           lambda: moe.moe_rms_norm_bwd(x, x.half(), r), lambda: moe.moe_rms_norm_bwd(x, x, r[:3]),
           lambda: moe.moe_rms_norm_bwd(leaf, x, r), lambda: moe.moe_rms_norm_bwd(x, leaf, r),
           lambda: moe.moe_rms_norm_bwd(x, x, r, dw=w.clone().requires_grad_()), lambda: moe.moe_rms_norm_bwd(x, x, r, dz=w)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: moe.moe_rms_norm(x, need_y=False), lambda: moe.moe_rms_norm(x, sf_format=0),
              lambda: moe.moe_rms_norm_bwd(x, x, r, need_dx=False, need_dw=False)):
        with pytest.raises(moe.MoEError):
            f()
    z = x.clone()
    with pytest.raises(moe.MoEError):                         # dx on z, which the sum for dw still needs
        moe.moe_rms_norm_bwd(x, z, r, dx=z)
