"""The row operators as a layer uses them: a 4-bit expert layer over the
planner's lists (each step held to float64 on the input it received), a
training step with the permutations' gradients, captured and replayed graphs,
and calls on other streams."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_amd as moe
import ops_util as ou
from parity_util import say

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


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


class Layer:
    """T tokens of width H through E experts of inner width I, 4-bit weights and activations."""

    def __init__(self, T, H, I, E, K, align, masked, seed):
        self.dims = T, H, I, E, K, align
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
        rng = np.random.default_rng(seed)
        self.idx = torch.from_numpy(ou.draw_idx(rng, T, K, E, masked).astype(np.int32)).cuda()
        self.w = torch.rand(T, K, generator=g, device="cuda")
        self.x = rand(T, H).bfloat16()
        quant = lambda rows, cols: [t.view(E, rows, -1) for t in moe.moe_quantize_mxfp4(
            (rand(E * rows, cols) / cols ** 0.5).bfloat16())]
        self.w1, self.w1_sf = quant(2 * I, H)
        self.w2, self.w2_sf = quant(H, I)

    def forward(self):
        T, H, I, E, K, align = self.dims
        r = planner(self.idx, E, align)
        codes, sf = moe.moe_quantize_mxfp4(self.x)
        xp = moe.moe_permute(codes, r["row_src"], r["src_row"], r["offsets"])
        xp_sf = moe.moe_permute(sf, r["row_src"], r["src_row"], r["offsets"])
        seg = dict(offsets=r["offsets"], counts=r["counts"], slots=T * K)
        gu = torch.zeros(xp.shape[0], 2 * I, dtype=torch.bfloat16, device="cuda")
        moe.moe_gemm_mxfp4(xp, xp_sf, self.w1, self.w1_sf, out=gu, **seg)
        g, u = gu.float().chunk(2, 1)
        h = (torch.nn.functional.silu(g) * u).bfloat16()
        hc, h_sf = moe.moe_quantize_mxfp4(h)
        yp = moe.moe_gemm_mxfp4(hc, h_sf, self.w2, self.w2_sf, **seg)
        y = moe.moe_unpermute(yp, r["src_row"], T, self.w)
        return dict(r=r, codes=codes, sf=sf, xp=xp, xp_sf=xp_sf, gu=gu, h=h, hc=hc, h_sf=h_sf, yp=yp, y=y)


def check_quantised(x, codes, sf):
    q, e = ou.quantised(f64(x))
    c = codes.cpu().numpy()
    got = np.stack([ou.E2M1[c & 15], ou.E2M1[c >> 4]], -1).reshape(q.shape)
    assert np.array_equal(got, q) and np.array_equal(sf.cpu().numpy().astype(np.int64) - 127, e)


def check_products(y, a, a_sf, b, b_sf, lists, dtype):
    va, vb = ou.values(a.cpu().numpy(), a_sf.cpu().numpy()), ou.values(b.cpu().numpy(), b_sf.cpu().numpy())
    k = va.shape[1]
    for e, (first, n) in enumerate(zip(lists["offsets"], lists["counts"])):
        if n == 0:
            continue
        s = slice(first, first + n)
        ex, mag = va[s] @ vb[e].T, abs(va[s]) @ abs(vb[e]).T
        inner = (k / 64 + 9) * 2.0 ** -22 * mag          # one MFMA per 64 columns, 2^-22 each
        assert np.all(abs(f64(y[s]) - ex) <= inner + ou.half_step(dtype) * (abs(ex) + inner) + ou.least(dtype))


@pytest.mark.parametrize("T,H,I,E,K,align,masked", [
    (1, 256, 128, 8, 2, 16, 0.0), (37, 160, 96, 5, 3, 1, 0.2), (200, 512, 256, 16, 4, 128, 0.1), (64, 96, 64, 6, 2, 8, 1.0)])
def test_four_bit_layer(T, H, I, E, K, align, masked):
    say(f"4-bit layer T={T} H={H} I={I} E={E} K={K} align={align}")
    layer = Layer(T, H, I, E, K, align, masked, 5)
    o = layer.forward()
    lists = ou.route(layer.idx.cpu().numpy(), E, align)
    for name in ("counts", "offsets", "row_src", "src_row"):
        assert np.array_equal(o["r"][name].cpu().numpy(), lists[name]), name
    used = lists["offsets"][-1]
    check_quantised(layer.x, o["codes"], o["sf"])
    for rows, moved in ((o["codes"], o["xp"]), (o["sf"], o["xp_sf"])):
        want = ou.permute(f64(rows), lists, np.zeros(tuple(moved.shape)))
        assert np.array_equal(f64(moved)[:used], want[:used])
    check_products(o["gu"], o["xp"], o["xp_sf"], layer.w1, layer.w1_sf, lists, torch.bfloat16)
    live = torch.from_numpy(lists["row_src"] >= 0).cuda()
    check_quantised(o["h"][live], o["hc"][live], o["h_sf"][live])
    check_products(o["yp"], o["hc"], o["h_sf"], layer.w2, layer.w2_sf, lists, torch.bfloat16)
    s, m = ou.token_sums(f64(o["yp"]), lists, T, f64(layer.w))
    inner = K * ou.U32 * m
    assert np.all(abs(f64(o["y"]) - s) <= inner + ou.half_step(torch.bfloat16) * (abs(s) + inner) + ou.least(torch.bfloat16))


def train_step(x, w, v, r, T, dy):
    """y of a layer of one matrix v[e] per expert, and the gradients of x, w and v, in float32
    torch products between the permutations."""
    E = v.shape[0]
    off, n = r["offsets"].tolist(), r["counts"].tolist()
    xp = moe.moe_permute(x, r["row_src"], r["src_row"], r["offsets"])
    yp = torch.zeros(xp.shape[0], v.shape[2], device="cuda")
    for e in range(E):
        yp[off[e]:off[e] + n[e]] = xp[off[e]:off[e] + n[e]] @ v[e]
    y = moe.moe_unpermute(yp, r["src_row"], T, w)
    dyp, dw = moe.moe_unpermute_bwd(dy, yp, r["row_src"], r["src_row"], r["offsets"], w)
    dxp = torch.zeros_like(xp)
    dv = torch.zeros_like(v)
    for e in range(E):
        s = slice(off[e], off[e] + n[e])
        dxp[s] = dyp[s] @ v[e].t().contiguous()
        dv[e] = xp[s].t().contiguous() @ dyp[s]
    return y, moe.moe_permute_bwd(dxp, r["src_row"], T), dw, dv


def test_training_step_against_the_formula_and_differences():
    T, K, E, H, N, align = 50, 3, 6, 72, 40, 8
    rng = np.random.default_rng(11)
    idx = ou.draw_idx(rng, T, K, E, 0.15)
    r = planner(torch.from_numpy(idx.astype(np.int32)).cuda(), E, align)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s))
    x, w, v, dy = t(T, H), t(T, K), t(E, H, N), t(T, N)
    got = train_step(*(a.float().cuda() for a in (x, w, v)), r, T, dy.float().cuda())
    x, w, v, dy = (a.float().double() for a in (x, w, v, dy))

    def loss(x, w, v):
        y = torch.zeros(T, N, dtype=torch.float64)
        for j in range(K):
            on = torch.from_numpy(idx[:, j] >= 0)
            e = torch.from_numpy(idx[:, j])[on]
            y[on] = y[on] + w[on, j, None] * torch.matmul(x[on].unsqueeze(1), v[e]).squeeze(1)
        return y, (y * dy).sum()

    leaves = [a.clone().requires_grad_() for a in (x, w, v)]
    y, total = loss(*leaves)
    grads = torch.autograd.grad(total, leaves)
    # sums of at most T K H N float32 products of values below 5; errors of order one rounding per
    # term over the terms of an element: at most 600 (rows of an expert times 1, or N, or H) at 2^-24
    for g, want, terms in zip(got, (y.detach(), *grads), (K * H, K * N, H + N, T * K)):
        scale = want.abs().max().item()
        assert (g.double().cpu() - want).abs().max().item() <= 4 * terms * ou.U32 * scale, terms
    # central differences of the loss along a direction, in float64 (the loss is trilinear: a step of
    # 2^-10 leaves a relative error of 2^-20)
    h = 2.0 ** -10
    for i, g in enumerate(got[1:]):
        d = torch.from_numpy(rng.standard_normal(tuple(leaves[i].shape)))
        at = lambda s: loss(*[a + s * h * d if k == i else a for k, a in enumerate((x, w, v))])[1].item()
        slope = (at(1) - at(-1)) / (2 * h)
        size = (g.double().cpu().abs() * d.abs()).sum().item()
        assert abs((g.double().cpu() * d).sum().item() - slope) <= 2.0 ** -14 * size


def test_graph_replays():
    # two captured layers, replayed in turn with new inputs and eager work between: every replay equal
    # to the eager result
    layers = [Layer(60, 256, 128, 8, 2, 16, 0.1, s) for s in (1, 2)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for a in layers:
        with torch.cuda.stream(side):
            a.forward()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(a.forward()["y"])
        graphs.append(g)
    for k in range(4):
        for a, g, y in zip(layers, graphs, outs):
            a.x.copy_(torch.randn_like(a.x.float()))
            a.w.uniform_()
            a.idx.copy_(a.idx.roll(7, 0))
            g.replay()
            torch.cuda.synchronize()
            got = y.clone()
            eager = a.forward()["y"]
            torch.cuda.synchronize()
            assert torch.equal(got, eager), k


@pytest.mark.parametrize("rows,n,k,groups", [(3, 500, 512, 0), (300, 1000, 544, 4), (2047, 2100, 800, 0), (4200, 3000, 1056, 0)])
def test_product_in_a_graph(rows, n, k, groups):
    # (one size for each kind of kernel)
    g = torch.Generator(device="cuda").manual_seed(rows)
    q = lambda *s: torch.randn(*s, generator=g, device="cuda")
    a, a_sf = moe.moe_quantize_mxfp4(q(rows, k))
    b, b_sf = moe.moe_quantize_mxfp4(q(max(1, groups) * n, k))
    kw = {}
    if groups:
        b, b_sf = b.view(groups, n, -1), b_sf.view(groups, n, -1)
        kw = dict(offsets=torch.linspace(0, rows, groups + 1, device="cuda").int())
    run = lambda: moe.moe_gemm_mxfp4(a, a_sf, b, b_sf, **kw)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run()
    for _ in range(3):
        c, f = moe.moe_quantize_mxfp4(q(rows, k))
        a.copy_(c), a_sf.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, run())


def test_gradients_in_a_graph():
    T, K, E, W = 70, 4, 9, 200
    rng = np.random.default_rng(2)
    r = planner(torch.from_numpy(ou.draw_idx(rng, T, K, E, 0.1).astype(np.int32)).cuda(), E, 16)
    R = r["row_src"].numel()
    yp, dy, w = torch.randn(R, W, device="cuda"), torch.randn(T, W, device="cuda"), torch.rand(T, K, device="cuda")
    dyp = torch.zeros(R, W, device="cuda")
    step = lambda: (*moe.moe_unpermute_bwd(dy, yp, r["row_src"], r["src_row"], r["offsets"], w, dyp=dyp),
                    moe.moe_permute_bwd(yp, r["src_row"], T))
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for _ in range(4):
        dy.normal_(), yp.normal_(), w.uniform_()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_streams():
    a, b = Layer(90, 256, 128, 8, 2, 16, 0.0, 3), Layer(90, 256, 128, 8, 2, 16, 0.0, 4)
    want = [l.forward()["y"].clone() for l in (a, b)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):                                      # two layers at once
        got = []
        for l, st in zip((a, b), s):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(l.forward()["y"])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    # the stream argument: outputs made there, as a Stream and as a handle
    codes, sf = moe.moe_quantize_mxfp4(a.x)
    r = planner(a.idx, 8, 16)
    xp = moe.moe_permute(a.x, r["row_src"], r["src_row"], r["offsets"])
    y = moe.moe_unpermute(xp, r["src_row"], 90, a.w)
    torch.cuda.synchronize()
    for st in (s[0], s[1].cuda_stream, 0):
        c2, f2 = moe.moe_quantize_mxfp4(a.x, stream=st)
        v2 = moe.moe_dequantize_mxfp4(c2, f2, stream=st)
        x2 = moe.moe_permute(a.x, r["row_src"], r["src_row"], r["offsets"], stream=st)
        y2 = moe.moe_unpermute(x2, r["src_row"], 90, a.w, stream=st)
        d2, w2 = moe.moe_unpermute_bwd(y2, x2, r["row_src"], r["src_row"], r["offsets"], a.w, stream=st)
        b2 = moe.moe_permute_bwd(x2, r["src_row"], 90, stream=st)
        g2 = moe.moe_gemm_mxfp4(a.w2[0], a.w2_sf[0], a.w2[1], a.w2_sf[1], stream=st)
        torch.cuda.synchronize()
        assert torch.equal(c2, codes) and torch.equal(f2, sf) and torch.equal(y2, y)
        assert torch.equal(v2, moe.moe_dequantize_mxfp4(codes, sf))
        used = r["offsets"][-1].item()
        assert torch.equal(x2[:used], xp[:used])
        d, w = moe.moe_unpermute_bwd(y, xp, r["row_src"], r["src_row"], r["offsets"], a.w)
        assert torch.equal(d2[:used], d[:used]) and torch.equal(w2, w)
        assert torch.equal(b2, moe.moe_permute_bwd(xp, r["src_row"], 90))
        assert torch.equal(g2, moe.moe_gemm_mxfp4(a.w2[0], a.w2_sf[0], a.w2[1], a.w2_sf[1]))
