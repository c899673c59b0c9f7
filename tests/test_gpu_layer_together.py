"""The operators around the experts' products as a layer uses them: the norm and the
router before the fused forward, a training step whose activations are kept in 8
bits (each step held to float64 on the input it received, and the whole to a float64
model), captured and replayed graphs, other streams, and autograd."""
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import fp8_grouped_gemm_amd as moe
import layer_util as lu
import ops_util as ou
import oracle
from parity_util import say

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EPS = 1e-6


def planner(idx, experts, align):
    """moe_route's lists on the GPU for expert ids idx int32 [T, K]."""
    T, K = idx.shape
    plan = moe.moe_plan_create(256, 128, experts, K, T)
    pool = T * K + experts * (align - 1)
    new = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    r = {"counts": new(experts), "offsets": new(experts + 1), "row_src": new(pool), "src_row": new(T * K)}
    ws = torch.empty(moe.moe_route_workspace_bytes(plan, T), dtype=torch.uint8, device="cuda")
    moe.moe_route(plan, T, idx, align, r["counts"], r["offsets"], r["row_src"], r["src_row"], ws)
    moe.moe_plan_destroy(plan)
    return r


@pytest.mark.parametrize("tokens", [1, 37])
def test_norm_and_router_before_the_fused_forward(tokens):
    say(f"norm, router and forward, {tokens} tokens")
    H, I, E, K = 256, 128, 8, 2
    g = torch.Generator().manual_seed(tokens)
    rand = lambda *s: torch.randn(*s, generator=g)
    x, res, w = rand(tokens, H).to(BF16).cuda(), rand(tokens, H).to(BF16).cuda(), (1 + 0.1 * rand(H)).cuda()
    wg, bias = rand(H, E).cuda(), (0.1 * rand(E)).cuda()
    z, _, y, codes, sf = moe.moe_rms_norm(x, w, residual=res, eps=EPS, sf_format=moe.MOE_SF_F32_128)
    logits = y.float() @ wg
    idx, tw = moe.moe_gate(logits, K, bias=bias, score=moe.MOE_SCORE_SIGMOID, groups=4, top_groups=2, group_top=2)
    want = lu.gate(lu.f64(logits), K, lu.f64(bias), None, True, 4, 2, 2, True, 1.0)
    assert np.array_equal(idx.cpu().numpy(), want[0])
    w1, w1_sf = torch.empty(E, 2 * I, H, dtype=torch.uint8), torch.empty(E, 2 * I // 128, H // 128)
    w2, w2_sf = torch.empty(E, H, I, dtype=torch.uint8), torch.empty(E, H // 128, I // 128)
    import workload as wl
    for e in range(E):
        w1[e], w1_sf[e] = wl.quantize_blocks(rand(2 * I, H) / H ** 0.5, 128, 128)
        w2[e], w2_sf[e] = wl.quantize_blocks(rand(H, I) / I ** 0.5, 128, 128)
    runner = moe.MoEForward(H, I, E, K, tokens)
    out = runner.forward(codes, sf, idx, tw, w1.cuda(), w1_sf.cuda(), w2.cuda(), w2_sf.cuda()).view(BF16)
    n = lambda t: t.cpu().numpy()
    ref = oracle.moe_forward(n(codes), n(sf), n(idx), n(tw), *[[t[e].numpy() for e in range(E)] for t in (w1, w1_sf, w2, w2_sf)])["y"]
    ref = (ref.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    # (the forward's own bound against the oracle, over the case: one code of h at a rounding's border on the other
    # side moves a token by a sixteenth of one of its 2 * 128 values, which alone may be over 1e-2 of a token)
    assert np.linalg.norm(lu.f64(out) - ref) <= 1e-2 * np.linalg.norm(ref)


@pytest.mark.parametrize("T,align", [(1, 16), (45, 16), (45, 1)])
def test_four_bit_layer(T, align):
    # a layer of 4-bit experts between the router and the tokens' order, padding rows never written by the activation
    say(f"4-bit layer, {T} tokens")
    H, I, E, K = 256, 96, 6, 2
    g = torch.Generator().manual_seed(T + align)
    rand = lambda *s: torch.randn(*s, generator=g).cuda()
    x, logits = rand(T, H).to(BF16), rand(T, E)
    (w1, w1_sf), (w2, w2_sf) = [[t.view(E, n, -1) for t in moe.moe_quantize_mxfp4(rand(E * n, k).to(BF16) / k ** 0.5)]
                                for n, k in ((2 * I, H), (H, I))]
    idx, tw = moe.moe_gate(logits, K)
    r = planner(idx, E, align)
    seg = dict(offsets=r["offsets"], counts=r["counts"], slots=T * K)
    codes, sf = moe.moe_quantize_mxfp4(x)
    xp, xps = (moe.moe_permute(t, r["row_src"], r["src_row"], r["offsets"]) for t in (codes, sf))
    gu = moe.moe_gemm_mxfp4(xp, xps, w1, w1_sf, **seg)
    h = torch.full((gu.shape[0], I), float("nan"), dtype=BF16, device="cuda")
    moe.moe_swiglu(gu, r["row_src"], r["offsets"], h=h)
    used = torch.arange(h.shape[0], device="cuda") < r["offsets"][-1]
    live = used & (r["row_src"] >= 0)
    want = lu.swiglu(lu.f64(gu[live]))
    # (bf16 of float32 with at most 128 roundings: the sigmoid's |g| and ten)
    lu.within(h[live], want, lu.rounded_bound(want, 128 * lu.U32 * abs(want) + 2.0 ** -120, BF16))
    assert torch.isnan(h[~live]).all()
    yp = moe.moe_gemm_mxfp4(*moe.moe_quantize_mxfp4(h), w2, w2_sf, **seg)
    y = moe.moe_unpermute(yp, r["src_row"], T, tw)
    # the same layer token by token
    for t in range(T):
        out = torch.zeros(H, dtype=torch.float64, device="cuda")
        for j in range(K):
            e = idx[t, j].item()
            a = moe.moe_gemm_mxfp4(codes[t:t + 1], sf[t:t + 1], w1[e], w1_sf[e])
            b = moe.moe_gemm_mxfp4(*moe.moe_quantize_mxfp4(moe.moe_swiglu(a)[0]), w2[e], w2_sf[e])
            out += tw[t, j].double() * b[0].double()
        # other tiles add in another order: a bf16 step in gate or up, and a 4-bit code of h beside a border (half of its
        # value) on the other side, of I of them
        assert torch.linalg.vector_norm(y[t].double() - out) <= 0.1 * torch.linalg.vector_norm(out) + 1e-3


class Layer:
    """Tokens of width H, residual, norm, a router and E experts of inner width I; activations that the
    backward pass needs are kept in 8 bits."""

    def __init__(self, T, H, I, E, K, align, seed):
        self.dims = T, H, I, E, K, align
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g).cuda()
        self.x, self.res, self.dz = rand(T, H).to(BF16), rand(T, H).to(BF16), 0.1 * rand(T, H).to(BF16)
        self.w, self.wg = 1 + 0.1 * rand(H), rand(H, E) / H ** 0.5
        self.w1, self.w2 = (rand(E, 2 * I, H) / H ** 0.5).to(BF16), (rand(E, H, I) / I ** 0.5).to(BF16)
        self.dy = rand(T, H).to(BF16)
        self.mask = (torch.rand(T, generator=g) < 0.9).cuda()

    def experts(self, rows, w, turn):
        """Each expert's product over all rows, its own rows kept (fixed sizes, for graphs)."""
        out = 0
        for e in range(w.shape[0]):
            m = w[e].float() if turn else w[e].float().t().contiguous()
            out = out + torch.where((self.owner == e)[:, None], rows.float() @ m, 0.0)
        return out.to(BF16)

    def step(self):
        T, H, I, E, K, align = self.dims
        o = {}
        z, rstd, y, xc, xs = moe.moe_rms_norm(self.x, self.w, residual=self.res, eps=EPS, sf_format=moe.MOE_SF_UE8M0_32)
        logits = y.float() @ self.wg
        idx, tw = moe.moe_gate(logits, K, mask=self.mask)
        r = planner(idx, E, align)
        rows = torch.arange(r["row_src"].numel(), device="cuda")
        owner = torch.bucketize(rows, r["offsets"][1:].long(), right=True)
        self.owner = torch.where(r["row_src"] >= 0, owner, -1)
        xp, xps = (moe.moe_permute(t, r["row_src"], r["src_row"], r["offsets"], out=torch.zeros(rows.numel(), t.shape[1], dtype=torch.uint8, device="cuda"))
                   for t in (xc, xs))
        gu = self.experts(self.read(xp, xps), self.w1, False)
        zero = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
        R = rows.numel()
        _, hc, hs, gc, gs = moe.moe_swiglu(gu, r["row_src"], r["offsets"], sf_format=moe.MOE_SF_UE8M0_32, need_h=False,
                                           need_h8=True, need_gu8=True, h_codes=zero(R, I), h_sf=zero(R, I // 32),
                                           gu_codes=zero(R, 2 * I), gu_sf=zero(R, I // 16))
        yp = self.experts(self.read(hc, hs), self.w2, False)
        out = moe.moe_unpermute(yp, r["src_row"], T, tw)
        # backwards, from the 8-bit copies
        dyp, dtw = moe.moe_unpermute_bwd(self.dy, yp, r["row_src"], r["src_row"], r["offsets"], tw, dyp=torch.zeros_like(yp))
        seg = dict(offsets=r["offsets"], counts=r["counts"])
        dw2 = moe.moe_gemm_wgrad(dyp, hc, hs, **seg)
        dh = self.experts(dyp, self.w2, True)
        dgu = moe.moe_swiglu_bwd(dh, gu_codes=gc, gu_sf=gs, row_src=r["row_src"], offsets=r["offsets"], out=torch.zeros_like(gu))
        dw1 = moe.moe_gemm_wgrad(dgu, xp, xps, **seg)
        dxp = self.experts(dgu, self.w1, True)
        dx8 = moe.moe_permute_bwd(dxp, r["src_row"], T)
        dlogits = moe.moe_gate_bwd(logits, idx, dtw)
        dwg = y.float().t().contiguous() @ dlogits
        dyn = (dx8.float() + dlogits @ self.wg.t().contiguous()).to(BF16)
        dx, dw = moe.moe_rms_norm_bwd(dyn, z, rstd, self.w, dz=self.dz)
        o.update(locals())
        return {k: v for k, v in o.items() if isinstance(v, (torch.Tensor, dict)) and k != "o"}

    @staticmethod
    def read(codes, sf):
        v = codes.view(torch.float8_e4m3fn).float()
        s = torch.ldexp(torch.ones((), device=v.device), sf.int() - 127)
        return v * s.repeat_interleave(32, 1)


@pytest.mark.parametrize("T,H,I,E,K,align", [(1, 64, 32, 4, 2, 1), (50, 128, 96, 6, 3, 8), (90, 256, 128, 8, 2, 16)])
def test_training_step(T, H, I, E, K, align):
    say(f"training step T={T} H={H} I={I} E={E} K={K}")
    a = Layer(T, H, I, E, K, align, 3)
    o = a.step()
    torch.cuda.synchronize()
    n = lu.f64
    # the forward steps on what they received
    z = ou.rounded(n(a.x) + n(a.res), BF16)
    assert np.array_equal(n(o["z"]), z)
    lu.near_codes(o["xc"], o["xs"], lu.norm(z, n(a.w), EPS)[1], lu.norm_steps(H) * lu.U32, 1)
    mask = a.mask.cpu().numpy()
    idx, tw = lu.gate(n(o["logits"]), K, None, mask, False, 1, 1, 1, True, 1.0)
    assert np.array_equal(o["idx"].cpu().numpy(), idx)
    lists = ou.route(idx, E, align)
    live = lists["row_src"] >= 0
    lu.near_codes(o["hc"][live], o["hs"][live], lu.swiglu(n(o["gu"]))[live], 97 * lu.U32, 1)
    lu.same_codes(o["gc"][live], o["gs"][live], o["gu"][live], 1)
    # the backward steps
    gv = lu.read(o["gc"], o["gs"])
    want, mag = lu.swiglu_grads(n(o["dh"]), gv)
    assert np.all(abs(n(o["dgu"]) - want)[live] <= lu.rounded_bound(want, 120 * lu.U32 * mag + 2.0 ** -100, BF16)[live])
    for dw, rows, codes, sf in ((o["dw2"], o["dyp"], o["hc"], o["hs"]), (o["dw1"], o["dgu"], o["xp"], o["xps"])):
        v, d = lu.read(codes, sf), n(rows)
        for e in range(E):
            s = slice(lists["offsets"][e], lists["offsets"][e] + lists["counts"][e])
            lu.within(n(dw[e]), d[s].T @ v[s], (lists["counts"][e] + 18) * 2.0 ** -23 * (abs(d[s]).T @ abs(v[s])))
    want, mag = lu.gate_grad(n(o["logits"]), idx, n(o["dtw"]), False, True, 1.0)
    lu.within(o["dlogits"], want, (4 * lu.gate_steps(n(o["logits"]), E) + 2 * K + 25) * lu.U32 * mag + 2.0 ** -140)
    wx, mx, ww, mw = lu.norm_grads(n(o["dyn"]), z, n(o["rstd"]), n(a.w), n(a.dz))
    lu.within(o["dx"], wx, lu.rounded_bound(wx, 60 * lu.U32 * mx, BF16))
    lu.within(o["dw"], ww, (T / 256 + 59) * lu.U32 * mw + 2.0 ** -140)
    # the whole against a float64 model whose 8-bit rows pass gradients straight through
    leaf = {k: getattr(a, k).double().cpu().requires_grad_() for k in ("x", "w", "wg", "w1", "w2")}
    zz = leaf["x"] + a.res.double().cpu()
    y = zz / torch.sqrt((zz * zz).mean(1, keepdim=True) + EPS) * leaf["w"]
    through = lambda v, q: v + (torch.from_numpy(q) - v).detach()
    x8 = through(y, lu.read(o["xc"], o["xs"]))
    s = torch.softmax(y @ leaf["wg"], 1).gather(1, torch.from_numpy(idx).clamp(min=0)) * torch.from_numpy(idx >= 0)
    weights = s / (s.sum(1, keepdim=True) + 1e-20)
    total = torch.zeros(T, H, dtype=torch.float64)
    hv = lu.read(o["hc"], o["hs"])
    for t in range(T):
        for j in range(K):
            e = int(idx[t, j])
            if e >= 0:
                row = lists["src_row"][t * K + j]
                gu = through(leaf["w1"][e] @ x8[t], gv[row])
                h = through(torch.nn.functional.silu(gu[:I]) * gu[I:], hv[row])
                total[t] = total[t] + weights[t, j] * (leaf["w2"][e] @ h)
    loss = (total * a.dy.double().cpu()).sum() + (zz * a.dz.double().cpu()).sum()
    grads = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()), allow_unused=True, materialize_grads=True)))
    # ten bf16 roundings at most lie between an input and a gradient, each of half a step (2^-8)
    for name, got in (("x", o["dx"]), ("w", o["dw"]), ("wg", o["dwg"]), ("w1", o["dw1"]), ("w2", o["dw2"])):
        far, size = np.linalg.norm(n(got) - grads[name].numpy()), np.linalg.norm(grads[name].numpy())
        assert far <= 10 * 2.0 ** -8 * size, (name, far, size)


def test_graph_replays():
    # two captured steps, replayed in turn with new inputs and eager work between: each equal to the eager result
    say("layer graphs")
    layers = [Layer(60, 128, 64, 8, 2, 16, s) for s in (1, 2)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for a in layers:
        with torch.cuda.stream(side):
            a.step()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(a.step())
        graphs.append(g)
    names = ("out", "idx", "dw1", "dw2", "dx", "dw", "dlogits", "dwg")
    for k in range(4):
        for a, g, o in zip(layers, graphs, outs):
            for t in (a.x, a.res, a.dy, a.dz):
                t.copy_(torch.randn_like(t.float()))
            a.mask.copy_(torch.rand_like(a.w[:60]) < 0.8)
            g.replay()
            torch.cuda.synchronize()
            got = [o[v].clone() for v in names]
            eager = a.step()
            torch.cuda.synchronize()
            for v, t in zip(names, got):
                assert torch.equal(t, eager[v]), (k, v)


def test_shared_rows_of_a_weight_gradient_in_a_graph():
    # rows split over workgroups: the sums meet in a workspace that the graph keeps; two graphs share one of their own
    say("weight gradient graphs")
    R, n, k = 9000, 70, 96
    need = moe.moe_gemm_wgrad_workspace_bytes(1, R, n, k)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    jobs = []
    for s in range(2):
        dy = torch.randn(R, n, device="cuda").to(BF16)
        codes, sf = torch.randint(0, 0x78, (R, k), device="cuda").to(torch.uint8), torch.full((R, k // 32), 127, dtype=torch.uint8, device="cuda")
        run = lambda dy=dy, codes=codes, sf=sf: moe.moe_gemm_wgrad(dy, codes, sf, workspace=ws)
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        jobs.append((dy, run, g, out))
    for _ in range(3):
        for dy, run, g, out in jobs:
            dy.normal_()
            g.replay()
            torch.cuda.synchronize()
            got = out.clone()
            assert torch.equal(got, run())


def test_streams():
    say("layer streams")
    a, b = Layer(70, 128, 64, 8, 2, 16, 5), Layer(70, 128, 64, 8, 2, 16, 6)
    names = ("out", "idx", "dw1", "dw2", "dx", "dw", "dlogits")
    want = [{k: l.step()[k].clone() for k in names} for l in (a, b)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):                                        # two steps at once
        got = []
        for l, st in zip((a, b), s):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(l.step())
        torch.cuda.synchronize()
        assert all(torch.equal(g[k], w[k]) for g, w in zip(got, want) for k in names)
    # the stream argument, as a Stream and as a handle
    x, w, l = a.x, a.w, torch.randn(70, 16, device="cuda")
    gu, dh = torch.randn(70, 128, device="cuda"), torch.randn(70, 64, device="cuda")
    torch.cuda.synchronize()

    def calls(**kw):
        z, rstd, y, c, f = moe.moe_rms_norm(x, w, residual=a.res, sf_format=1, **kw)
        idx, tw = moe.moe_gate(l, 3, **kw)
        h, hc, hs, gc, gs = moe.moe_swiglu(gu, sf_format=1, need_h8=True, need_gu8=True, **kw)
        return (z, rstd, y, c, f, idx, tw, h, hc, hs, gc, gs, *moe.moe_rms_norm_bwd(y, z, rstd, w, **kw),
                moe.moe_gate_bwd(l, idx, tw, **kw), moe.moe_swiglu_bwd(dh, gu_codes=gc, gu_sf=gs, **kw),
                moe.moe_gemm_wgrad(y, c, f, **kw))

    ref = calls()
    for st in (s[0], s[1].cuda_stream, 0):
        got = calls(stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, ref))


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w):
        _, rstd, y, _, _ = moe.moe_rms_norm(x, w, eps=EPS)
        ctx.save_for_backward(x, w, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w, rstd = ctx.saved_tensors
        dx, dw = moe.moe_rms_norm_bwd(dy, x, rstd, w)
        return dx, dw.to(w.dtype)


class Gate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k):
        idx, w = moe.moe_gate(logits, k)
        ctx.save_for_backward(logits, idx)
        ctx.mark_non_differentiable(idx)
        return w, idx

    @staticmethod
    def backward(ctx, dw, _):
        return moe.moe_gate_bwd(*ctx.saved_tensors, dw.contiguous()), None


class SwiGLU(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gu):
        h, _, _, codes, sf = moe.moe_swiglu(gu, sf_format=moe.MOE_SF_UE8M0_32, need_gu8=True)
        ctx.save_for_backward(codes, sf)
        return h

    @staticmethod
    def backward(ctx, dh):
        codes, sf = ctx.saved_tensors
        return moe.moe_swiglu_bwd(dh, gu_codes=codes, gu_sf=sf)


def test_autograd_functions_and_versions():
    say("autograd")
    leaf = lambda *s: torch.randn(*s, device="cuda", requires_grad=True)
    x, w, gu = leaf(6, 64), leaf(64), leaf(6, 64)
    y = Norm.apply(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), torch.ones_like(y))
    xr = x.detach().double().requires_grad_()
    wr = w.detach().double().requires_grad_()
    ref = torch.autograd.grad(xr / torch.sqrt((xr * xr).mean(1, keepdim=True) + EPS) * wr, (xr, wr), torch.ones(6, 64, dtype=torch.float64, device="cuda"))
    for g, r in zip((dx, dw), ref):
        assert (g - r).abs().max() <= 200 * lu.U32 * r.abs().max()      # 64-term sums and a dozen roundings
    tw, idx = Gate.apply(x, 5)
    d, = torch.autograd.grad(tw, x, torch.randn_like(tw))
    assert d.shape == x.shape and torch.isfinite(d).all()
    d, = torch.autograd.grad(SwiGLU.apply(gu), gu, torch.ones(6, 32, device="cuda"))
    assert d.shape == gu.shape and torch.isfinite(d).all()
    # a tensor that a graph saved and a call overwrote is refused in the backward pass
    p, q = x.detach().clone(), gu.detach().clone()
    rstd = torch.ones(6, device="cuda")
    codes, sf = moe.moe_swiglu(q, need_gu8=True, sf_format=1)[3:]
    i5 = idx.clone()
    for f in (lambda o: moe.moe_rms_norm(p, y=o), lambda o: moe.moe_rms_norm(p, residual=p, z=o),
              lambda o: moe.moe_rms_norm_bwd(p, p, rstd, dx=o), lambda o: moe.moe_gate_bwd(p, i5, tw.detach(), out=o),
              lambda o: moe.moe_swiglu(torch.cat([q, q], 1), h=o), lambda o: moe.moe_swiglu_bwd(p[:, :32].contiguous(), gu=q, out=o),
              lambda o: moe.moe_gemm_wgrad(torch.zeros(6, 6, device="cuda").to(BF16), codes, sf, out=o)):
        saved = torch.randn(6, 64, device="cuda")
        loss = (saved * torch.randn_like(saved).requires_grad_()).sum()
        f(saved)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    before = [t._version for t in (i5, codes, sf, rstd)]
    moe.moe_gate(p, 5, topk_idx=i5)
    moe.moe_swiglu(q, need_gu8=True, sf_format=1, gu_codes=codes, gu_sf=sf)
    moe.moe_rms_norm(p, rstd=rstd)
    assert all(t._version > v for t, v in zip((i5, codes, sf, rstd), before))


PROGRAM = """
import torch
import fp8_grouped_gemm_amd as moe
T, H = {sizes}
x, w, l = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(H, device="cuda"), torch.randn(T, 96, device="cuda")
bias = torch.zeros(96, device="cuda")
torch.cuda.synchronize()
def run():
    z, rstd, y, c, f = moe.moe_rms_norm(x, w, residual=x, sf_format=1)
    idx, tw = moe.moe_gate(l, 4, bias=bias, groups=8, top_groups=3, group_top=2)
    h, hc, hs, gc, gs = moe.moe_swiglu(y, sf_format=1, need_h8=True, need_gu8=True)
    return (z, y, c, f, idx, tw, h, hc, hs, gc, gs, *moe.moe_rms_norm_bwd(y, z, rstd, w), moe.moe_gate_bwd(l, idx, tw),
            moe.moe_swiglu_bwd(h, gu_codes=gc, gu_sf=gs), moe.moe_gemm_wgrad(y, hc, hs))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = run()
for _ in range(3):
    x.normal_(), l.normal_()
    graph.replay()
    torch.cuda.synchronize()
    got = [v.clone() for v in out]
    assert all(torch.equal(v, w) for v, w in zip(got, run()))
print("replays equal")
"""


@pytest.mark.parametrize("sizes", [(5, 128), (3000, 1024)])
def test_first_call_is_captured(sizes):
    run = subprocess.run([sys.executable, "-c", PROGRAM.format(sizes=sizes)], cwd=Path(__file__).parents[1],
                         capture_output=True, text=True, timeout=100)
    assert run.returncode == 0 and "replays equal" in run.stdout, run.stdout + run.stderr
