"""Measured cases of the operators around the experts' products: the router's
choice of experts, the residual's addition with a root-mean-square norm and an
8-bit result, SwiGLU with its inputs kept in 8 bits, and the experts' weight
gradients from 8-bit rows; each with its gradient.

`run` computes a case with the library's entry points when `own` is true and
in elementary torch operations otherwise.

8-bit rows are e4m3 codes with a scale per block of columns, in one of two
formats: "f32" (128 columns, sf = max(amax, 1e-10) / 448 in float32) and "ue8m0"
(32 columns, the smallest power of two at or above that).  Codes and scales are
returned as the values they stand for.  Routing lists are those of the library's
planner: expert e's rows are offsets[e] .. offsets[e] + counts[e] - 1 of the pool,
row_src[r] is the slot of pool row r (-1: padding).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = {"f32": 128, "ue8m0": 32}
SF_BYTES = {"f32": 4 / 128, "ue8m0": 1 / 32, "": 0}        # per column
EPS = 1e-6
# the most a drawn case of each kind handles: what the largest listed one does
MOST_LOGITS = 32768 * 384
MOST_NORM = 8192 * 7168
MOST_SWIGLU = 49152 * 2048
MOST_FLOP = 2 * 12288 * 4096 * 4096
MOST_WEIGHTS = 32 * 4096 * 4096


def listed():
    return [
        # One token's router in a decode step: latency alone.
        dict(name="gate 1 token", op="gate", dtype="f32", tokens=1, experts=384, top_k=6, score="softmax",
             bias=False, groups=1, top_groups=1, group_top=1, renorm=True, masked=0.0),
        # A prompt batch of a router with a balance bias and expert groups, float32 logits.
        dict(name="gate prompt", op="gate", dtype="f32", tokens=8192, experts=256, top_k=8, score="sigmoid",
             bias=True, groups=8, top_groups=4, group_top=2, renorm=True, masked=0.0),
        # The router's gradient in a training step of long sequences, a tenth of it padding.
        dict(name="gate gradient", op="gate_grad", dtype="bf16", tokens=32768, experts=384, top_k=6,
             score="softmax", bias=False, groups=1, top_groups=1, group_top=1, renorm=True, masked=0.1),
        # A decode batch of the flash layer: residual, norm and the FP8 forward's operand.
        dict(name="norm decode", op="norm", dtype="bf16", rows=128, width=4096, residual=True, y=False, sf="f32"),
        # The pro layer's prompt batch: residual, norm, rows for the router and 8-bit rows for the experts.
        dict(name="norm prompt", op="norm", dtype="bf16", rows=8192, width=7168, residual=True, y=True, sf="ue8m0"),
        # Its gradient in a training step, with the residual's gradient and the weight's.
        dict(name="norm gradient", op="norm_grad", dtype="bf16", rows=8192, width=4096, residual=True),
        # A decode batch's 768 routed rows between the two products, 8-bit operand of the second.
        dict(name="swiglu decode", op="swiglu", dtype="bf16", rows=768, inner=2048, experts=32, align=16, sf="f32",
             h=False, keep=False),
        # A training batch of 8192 tokens, top-6: 8-bit h and the 8-bit copy of gate and up that the gradient
        # reads, segments aligned to 128 rows.
        dict(name="swiglu prompt", op="swiglu", dtype="bf16", rows=49152, inner=2048, experts=256, align=128,
             sf="ue8m0", h=False, keep=True),
        # Its gradient from that copy.
        dict(name="swiglu gradient", op="swiglu_grad", dtype="bf16", rows=49152, inner=2048, experts=256, align=128,
             sf="ue8m0"),
        # A small odd step: few rows an expert, ragged sizes, float32 scales, half precision.
        dict(name="weights few rows", op="wgrad", dtype="f16", out="f32", experts=8, rows=301, n=520, k=896,
             align=1, sf="f32"),
        # The router's or a dense layer's weight: one matrix, many rows.
        dict(name="weights dense", op="wgrad", dtype="bf16", out="f32", experts=1, rows=8192, n=384, k=7168,
             align=1, sf="ue8m0"),
        # The 32 resident experts of the flash layer, a training batch of 12288 routed rows.
        dict(name="weights prompt", op="wgrad", dtype="bf16", out="bf16", experts=32, rows=12288, n=4096, k=4096,
             align=16, sf="ue8m0"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "gate", "gate_grad", "norm", "norm", "norm_grad", "swiglu", "swiglu_grad", "wgrad",
                     "wgrad"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op in ("gate", "gate_grad"):
        group = _log(rng, 2, 64)
        groups = rng.choice([1, 1, rng.randint(2, 8)])
        experts = min(512, max(4, group * groups if groups > 1 else _log(rng, 4, 512)))
        groups = groups if experts % groups == 0 else 1
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(12, experts // groups * top_groups))
        tokens = max(1, min(_log(rng, 1, 32768), MOST_LOGITS // 2 // experts))
        # (a router that sums a group's best has a bias: without one sigmoid(x) + sigmoid(-x) would tie;
        # one weight alone is not renormalised: it would be 1, and its gradient nothing but roundings)
        group_top = min(rng.choice([1, 2]), experts // groups)
        return dict(op=op, dtype=dtype, tokens=tokens, experts=experts, top_k=top_k,
                    score=rng.choice(["softmax", "sigmoid"]), bias=group_top == 2 or rng.random() < 0.5,
                    groups=groups, top_groups=top_groups, group_top=group_top,
                    renorm=top_k > 1 and rng.random() < 0.7, masked=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op in ("norm", "norm_grad"):
        sf = rng.choice(["", "f32", "ue8m0"]) if op == "norm" else ""
        width = BLOCK[sf] * _log(rng, 1, 8192 // BLOCK[sf]) if sf else _log(rng, 16, 8192)
        rows = max(1, min(_log(rng, 1, 16384), MOST_NORM // 2 // width))
        case = dict(op=op, dtype=dtype, rows=rows, width=width, residual=rng.random() < 0.7)
        return {**case, "y": not sf or rng.random() < 0.5, "sf": sf} if op == "norm" else case
    if op in ("swiglu", "swiglu_grad"):
        sf = rng.choice(["", "f32", "ue8m0"])
        inner = BLOCK[sf] * _log(rng, 1, 8192 // BLOCK[sf]) if sf else _log(rng, 16, 8192)
        rows = max(1, min(_log(rng, 1, 49152), MOST_SWIGLU // 4 // inner))
        experts, align = _log(rng, 1, 256), rng.choice([1, 16, 64])
        case = dict(op=op, dtype=dtype, rows=rows, inner=inner, experts=max(1, min(experts, rows)), align=align, sf=sf)
        if op == "swiglu":
            case.update(h=not sf or rng.random() < 0.3, keep=bool(sf) and rng.random() < 0.6)
        return case
    sf = rng.choice(["f32", "ue8m0"])
    experts = rng.choice([1, _log(rng, 2, 64)])
    n, k = _log(rng, 16, 4096), BLOCK[sf] * _log(rng, 1, 4096 // BLOCK[sf])
    if rng.random() < 0.5:
        n = max(16, n // 16 * 16)
    experts = max(1, min(experts, MOST_WEIGHTS // 2 // (n * k)))
    rows = max(1, min(_log(rng, 1, 12288), MOST_FLOP // 4 // (n * k)))
    return dict(op=op, dtype=rng.choice(["bf16", "f16"]), out=rng.choice(["f32", "bf16", "f16"]), experts=experts,
                rows=rows, n=n, k=k, align=rng.choice([1, 16, 128]), sf=sf)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, cols):
    """Gaussian rows with a few columns of larger values."""
    return _randn(g, rows, cols) * (1 + 15 * (_rand(g, 1, cols) < 0.01).float())


def _segments(g, rows, experts, align):
    """The planner's lists for `rows` slots of a skewed router; the pool has room for each expert's padding."""
    e = torch.argmax(_randn(g, rows, experts) + 0.5 * _randn(g, 1, experts), 1)
    counts = torch.bincount(e, minlength=experts)
    ends = torch.cumsum((counts + align - 1) // align * align, 0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    order = torch.argsort(e, stable=True)
    rank = torch.arange(rows, device="cuda") - (torch.cumsum(counts, 0) - counts)[e[order]]
    row_src = torch.full((rows + experts * (align - 1),), -1, dtype=torch.int64, device="cuda")
    row_src[offsets[e[order]] + rank] = order
    return {"counts": counts.int(), "offsets": offsets.int(), "row_src": row_src.int()}


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if op in ("gate", "gate_grad"):
        T, E, K = case["tokens"], case["experts"], case["top_k"]
        s["logits"] = (1.5 * _randn(g, T, E) + 0.5 * _randn(g, 1, E)).to(dt)
        s["bias"] = 0.05 * _randn(g, E) if case["bias"] else None
        s["mask"] = (_rand(g, T) >= case["masked"]) if case["masked"] else None
        if op == "gate_grad":                               # of the choice that the forward pass made
            s["idx"], _ = _gate(s)
            s["dw"] = _randn(g, T, K)
    elif op == "norm":
        T, W = case["rows"], case["width"]
        s["x"] = _activations(g, T, W).to(dt)
        s["residual"] = (4 * _randn(g, T, W)).to(dt) if case["residual"] else None
        s["weight"] = (1 + 0.1 * _randn(g, W)).to(dt)
    elif op == "norm_grad":
        T, W = case["rows"], case["width"]
        s["dy"], s["z"] = _randn(g, T, W).to(dt), _activations(g, T, W).to(dt)
        s["dz"] = _randn(g, T, W).to(dt) if case["residual"] else None
        s["weight"] = (1 + 0.1 * _randn(g, W)).to(dt)
        s["rstd"] = _rstd(s["z"].double()).float()
    elif op in ("swiglu", "swiglu_grad"):
        lists = _segments(g, case["rows"], case["experts"], case["align"])
        s.update(row_src=lists["row_src"], offsets=lists["offsets"])
        R, I = s["row_src"].numel(), case["inner"]
        gu = _activations(g, R, 2 * I).to(dt)
        if op == "swiglu":
            s["gu"] = gu
            if case["h"]:
                s["h"] = torch.zeros(R, I, dtype=dt, device="cuda")
            for name, cols in (("h", I),) * bool(case["sf"]) + (("gu", 2 * I),) * case["keep"]:
                s[name + "_codes"] = torch.zeros(R, cols, dtype=torch.uint8, device="cuda")
                s[name + "_sf"] = torch.zeros(R, cols // BLOCK[case["sf"]], device="cuda",
                                              dtype=torch.float32 if case["sf"] == "f32" else torch.uint8)
        else:
            s["dh"] = _randn(g, R, I).to(dt)
            s["dgu"] = torch.zeros(R, 2 * I, dtype=dt, device="cuda")
            if case["sf"]:
                s["gu_codes"], s["gu_sf"] = _codes(gu.float(), case["sf"])
            else:
                s["gu"] = gu
    else:
        E, n, k = case["experts"], case["n"], case["k"]
        R = case["rows"]
        if E > 1:
            lists = _segments(g, R, E, case["align"])
            s.update(counts=lists["counts"], offsets=lists["offsets"], most=int(lists["counts"].max()))
            R = lists["row_src"].numel()
        s["dy"] = _randn(g, R, n).to(dt)
        s["x"], s["x_sf"] = _codes(_activations(g, R, k), case["sf"])
    return s


# ---------------------------------------------------------------- plain forms

def _fp8(v, sf):
    """The e4m3 values of float32 rows in units of their block's scale, and the scales."""
    blk = v.unflatten(-1, (-1, BLOCK[sf]))
    scale = blk.abs().amax(-1).clamp(min=1e-10) / 448
    if sf == "ue8m0":
        m, e = torch.frexp(scale)
        scale = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))
    q = (blk / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.flatten(-2), scale


def _codes(v, sf):
    q, scale = _fp8(v, sf)
    if sf == "ue8m0":
        scale = (torch.frexp(scale)[1] + 126).to(torch.uint8)
    return q.view(torch.uint8), scale


def _read(codes, sf):
    """float32 values of codes with scales (uint8 codes of powers of two, or float32)."""
    if sf.dtype == torch.uint8:
        sf = torch.ldexp(torch.ones((), device=sf.device), sf.to(torch.int32) - 127)
    return (codes.view(torch.float8_e4m3fn).float().unflatten(-1, (sf.shape[-1], -1)) * sf[..., None]).flatten(-2)


def _stands_for(codes, sf):
    """The values that codes and scales stand for, without a copy."""
    return codes.view(torch.float8_e4m3fn), sf if sf.dtype == torch.float32 else sf.view(torch.float8_e8m0fnu)


def _scores(case, logits):
    """float64 scores: neighbours of the choice are nearer than float32 tells apart."""
    l = logits.double()
    if case["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    p = torch.exp(l - l.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _gate(s):
    case = s["case"]
    T, E, K, G = case["tokens"], case["experts"], case["top_k"], case["groups"]
    score = _scores(case, s["logits"])
    choice = score + s["bias"] if s["bias"] is not None else s["logits"].double()
    if G > 1:
        best = (choice if case["group_top"] == 1 or s["bias"] is not None else score).view(T, G, E // G)
        best = torch.sort(best, dim=-1, descending=True).values[..., :case["group_top"]].sum(-1)
        keep = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        on = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, keep, True)
        choice = torch.where(on.repeat_interleave(E // G, 1), choice, -math.inf)
    idx = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :K]
    w = torch.gather(score, 1, idx)
    if case["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    if s["mask"] is not None:
        idx = torch.where(s["mask"][:, None], idx, -1)
        w = torch.where(s["mask"][:, None], w, 0.0)
    return idx.int(), w.float()


def _gate_grad(s):
    case, idx = s["case"], s["idx"].long()
    score = _scores(case, s["logits"])
    on = idx >= 0
    p = torch.where(on, torch.gather(score, 1, idx.clamp(min=0)), 0.0)
    dp = torch.where(on, s["dw"].double(), 0.0)
    if case["renorm"]:
        total = p.sum(1, keepdim=True) + 1e-20
        dp = torch.where(on, (dp - (dp * p).sum(1, keepdim=True) / total) / total, 0.0)
    ds = torch.zeros_like(score).scatter_add_(1, idx.clamp(min=0), dp)
    if case["score"] == "sigmoid":
        out = ds * score * (1 - score)
    else:
        out = score * (ds - (dp * p).sum(1, keepdim=True))
    return torch.where(on.any(1, keepdim=True), out, 0.0).to(s["logits"].dtype)


def _rstd(z):
    return torch.rsqrt((z * z).mean(1) + EPS)


def _norm(s):
    case, x = s["case"], s["x"]
    out = {}
    z = x.float()
    if case["residual"]:
        out["z"] = (z + s["residual"].float()).to(x.dtype)
        z = out["z"].float()
    out["rstd"] = _rstd(z)
    y = z * out["rstd"][:, None] * s["weight"].float()
    if case["y"]:
        out["y"] = y.to(x.dtype)
    if case["sf"]:
        out["codes"], out["sf"] = _stands_for(*_codes(y, case["sf"]))
    return out


def _norm_grad(s):
    xh = s["z"].float() * s["rstd"][:, None]
    g = s["dy"].float()
    dw = (g.double() * xh.double()).sum(0).float()
    g = g * s["weight"].float()
    dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dz"] is not None:
        dx = dx + s["dz"].float()
    return {"dx": dx.to(s["dy"].dtype), "dw": dw}


def _live(s):
    """Pool rows that hold a slot, [R, 1]."""
    r = torch.arange(s["row_src"].numel(), device="cuda")
    return ((s["row_src"] >= 0) & (r < s["offsets"][-1]))[:, None]


def _swiglu(s):
    case, live = s["case"], _live(s)
    gu = s["gu"].float()
    g, u = gu.chunk(2, 1)
    h = g / (1 + torch.exp(-g)) * u
    out = {}
    if case["h"]:
        out["h"] = torch.where(live, h.to(s["gu"].dtype), s["h"])
    for name, v in (("h", h),) * bool(case["sf"]) + (("gu", gu),) * case["keep"]:
        codes, sf = _codes(v, case["sf"])
        out[name + "_codes"], out[name + "_sf"] = _stands_for(torch.where(live, codes, s[name + "_codes"]),
                                                              torch.where(live, sf, s[name + "_sf"]))
    return out


def _swiglu_grad(s):
    gu = s["gu"].float() if "gu" in s else _read(s["gu_codes"], s["gu_sf"])
    g, u = gu.chunk(2, 1)
    dh, sg = s["dh"].float(), 1 / (1 + torch.exp(-g))
    dgu = torch.cat([dh * u * sg * (1 + g * (1 - sg)), dh * g * sg], 1)
    return {"dgu": torch.where(_live(s), dgu.to(s["dgu"].dtype), s["dgu"])}


def _wgrad(s):
    case, dy = s["case"], s["dy"].float()
    x = _read(s["x"], s["x_sf"]).to(s["dy"].dtype).float()   # the product takes x in dy's type
    if case["experts"] == 1:
        return {"dw": torch.matmul(dy.t(), x).to(DTYPES[case["out"]])}
    rank = torch.arange(s["most"], device="cuda")
    live = (rank < s["counts"][:, None])[..., None]
    at = (rank + s["offsets"][:-1, None]).clamp(max=dy.shape[0] - 1).long()
    dy, x = torch.where(live, dy[at], 0.0), torch.where(live, x[at], 0.0)
    return {"dw": torch.matmul(dy.transpose(1, 2).contiguous(), x).to(DTYPES[case["out"]])}


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "gate":
            idx, w = _gate(s)
            return {"idx": idx, "w": w}
        if op == "gate_grad":
            return {"dlogits": _gate_grad(s)}
        return {"norm": _norm, "norm_grad": _norm_grad, "swiglu": _swiglu, "swiglu_grad": _swiglu_grad,
                "wgrad": _wgrad}[op](s)
    import fp8_grouped_gemm_amd as moe
    if op in ("gate", "gate_grad"):
        score = moe.MOE_SCORE_SIGMOID if case["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX
        if op == "gate":
            idx, w = moe.moe_gate(s["logits"], case["top_k"], bias=s["bias"], mask=s["mask"], score=score,
                                  groups=case["groups"], top_groups=case["top_groups"],
                                  group_top=case["group_top"], renorm=case["renorm"])
            return {"idx": idx, "w": w}
        return {"dlogits": moe.moe_gate_bwd(s["logits"], s["idx"], s["dw"], score=score, renorm=case["renorm"])}
    if op == "norm":
        fmt = {"": None, "f32": moe.MOE_SF_F32_128, "ue8m0": moe.MOE_SF_UE8M0_32}[case["sf"]]
        z, rstd, y, codes, sf = moe.moe_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS,
                                                 need_y=case["y"], sf_format=fmt)
        out = {"rstd": rstd}
        if case["residual"]:
            out["z"] = z
        if case["y"]:
            out["y"] = y
        if case["sf"]:
            out["codes"], out["sf"] = _stands_for(codes, sf)
        return out
    if op == "norm_grad":
        dx, dw = moe.moe_rms_norm_bwd(s["dy"], s["z"], s["rstd"], s["weight"], dz=s["dz"])
        return {"dx": dx, "dw": dw}
    if op == "swiglu":
        given = {k: s[k] for k in ("h", "h_codes", "h_sf", "gu_codes", "gu_sf") if k in s}
        fmt = {"": None, "f32": moe.MOE_SF_F32_128, "ue8m0": moe.MOE_SF_UE8M0_32}[case["sf"]]
        h, h_codes, h_sf, gu_codes, gu_sf = moe.moe_swiglu(
            s["gu"], row_src=s["row_src"], offsets=s["offsets"], sf_format=fmt, need_h=case["h"],
            need_h8=bool(case["sf"]), need_gu8=case["keep"], **given)
        out = {"h": h} if case["h"] else {}
        if case["sf"]:
            out["h_codes"], out["h_sf"] = _stands_for(h_codes, h_sf)
        if case["keep"]:
            out["gu_codes"], out["gu_sf"] = _stands_for(gu_codes, gu_sf)
        return out
    if op == "swiglu_grad":
        return {"dgu": moe.moe_swiglu_bwd(s["dh"], gu=s.get("gu"), gu_codes=s.get("gu_codes"),
                                          gu_sf=s.get("gu_sf"), row_src=s["row_src"], offsets=s["offsets"],
                                          out=s["dgu"])}
    return {"dw": moe.moe_gemm_wgrad(s["dy"], s["x"], s["x_sf"], offsets=s.get("offsets"),
                                     counts=s.get("counts"), dtype=DTYPES[case["out"]])}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, size = case["op"], SIZE[case["dtype"]]
    if op in ("gate", "gate_grad"):
        T, E, K = case["tokens"] * (1 - case["masked"]), case["experts"], case["top_k"]
        if op == "gate":
            return {"bytes": T * E * size + 8 * case["tokens"] * K, "flops": 6 * T * E}
        return {"bytes": T * E * size + case["tokens"] * (E * size + 4 * K) + 4 * T * K, "flops": 8 * T * E}
    if op in ("norm", "norm_grad"):
        n = case["rows"] * case["width"]
        if op == "norm":
            moved = size * (1 + 2 * case["residual"] + case["y"]) + (1 + SF_BYTES[case["sf"]] if case["sf"] else 0)
            return {"bytes": n * moved + 4 * case["rows"], "flops": 5 * n}
        return {"bytes": n * size * (3 + case["residual"]) + 4 * case["rows"], "flops": 10 * n}
    if op in ("swiglu", "swiglu_grad"):
        n = case["rows"] * case["inner"]
        eight = 1 + SF_BYTES[case["sf"]] if case["sf"] else 0
        if op == "swiglu":
            return {"bytes": n * (size * (2 + case["h"]) + eight * (1 + 2 * case["keep"])), "flops": 6 * n}
        return {"bytes": n * (size * 3 + (2 * eight or 2 * size)), "flops": 12 * n}
    m, n, k = case["rows"], case["n"], case["k"]
    return {"bytes": m * (n * size + k * (1 + SF_BYTES[case["sf"]])) + case["experts"] * n * k * SIZE[case["out"]],
            "flops": 2 * m * n * k}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_fp8(v, sf):
    """(e4m3 values in units of the scale, scales) of float64 rows."""
    blk = v.reshape(v.shape[0], -1, BLOCK[sf])
    scale = blk.abs().amax(-1).clamp(min=1e-10) / 448
    if sf == "ue8m0":
        scale = torch.exp2(torch.ceil(torch.log2(scale) - 1e-12))
    q = blk / scale[..., None]
    # e4m3: 3 bits behind the leading one, the spacing of its smallest binade is 2^-9
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / step) * step).clamp(-448, 448).reshape(v.shape), scale


def _exact_read(codes, sf):
    c = codes.long()
    e, m = (c >> 3) & 15, c & 7
    v = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
    s = sf.double() if sf.dtype == torch.float32 else torch.exp2(sf.double() - 127)
    return torch.where(c > 127, -v, v) * s.repeat_interleave(codes.shape[1] // s.shape[1], 1)


def _exact_gate(s):
    case = s["case"]
    T, E, G = case["tokens"], case["experts"], case["groups"]
    l = s["logits"].double()
    score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    choice = l.clone() if s["bias"] is None else score + s["bias"].double()
    ids = torch.arange(E, device="cuda")

    def first_best(v):                                       # the lowest index of the largest value
        return torch.where(v == v.amax(1, keepdim=True), ids[:v.shape[1]], E).amin(1)

    if G > 1:
        by = choice if s["bias"] is not None or case["group_top"] == 1 else score
        total = torch.topk(by.view(T, G, E // G), case["group_top"], dim=2).values.sum(2)
        kept = torch.zeros(T, G, dtype=torch.bool, device="cuda")
        for _ in range(case["top_groups"]):
            at = first_best(total)[:, None]
            kept.scatter_(1, at, True)
            total.scatter_(1, at, -math.inf)
        choice[~kept[:, ids // (E // G)]] = -math.inf
    picked = []
    for _ in range(case["top_k"]):
        at = first_best(choice)
        picked.append(at)
        choice.scatter_(1, at[:, None], -math.inf)
    idx = torch.stack(picked, 1)
    w = score.gather(1, idx)
    if case["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    if s["mask"] is not None:
        idx[~s["mask"]] = -1
        w[~s["mask"]] = 0
    return {"idx": idx.int(), "w": w}


def _exact_gate_grad(s):
    # by automatic differentiation of the weights as a function of the logits
    case = s["case"]
    l = s["logits"].double().requires_grad_()
    score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    on = s["idx"] >= 0
    w = score.gather(1, s["idx"].clamp(min=0).long()) * on
    if case["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return {"dlogits": torch.autograd.grad((w * s["dw"].double()).sum(), l)[0]}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gate":
        return _exact_gate(s)
    if op == "gate_grad":
        return _exact_gate_grad(s)
    if op == "norm":
        out, z = {}, s["x"].double()
        if case["residual"]:
            z = z + s["residual"].double()
            out["z"] = z
            z = z.to(s["x"].dtype).double()                  # the norm is of the stored sum
        out["rstd"] = 1 / torch.sqrt(z.square().mean(1) + EPS)
        y = z * out["rstd"][:, None] * s["weight"].double()
        if case["y"]:
            out["y"] = y
        if case["sf"]:
            out["codes"], out["sf"] = _exact_fp8(y, case["sf"])
        return out
    if op == "norm_grad":
        z, r = s["z"].double(), s["rstd"].double()[:, None]
        dy, w = s["dy"].double(), s["weight"].double()
        dx = r * dy * w - r ** 3 * z * (dy * w * z).mean(1, keepdim=True)
        return {"dx": dx if s["dz"] is None else dx + s["dz"].double(), "dw": (dy * z * r).sum(0)}
    if op in ("swiglu", "swiglu_grad"):
        used = int(s["offsets"][-1])
        at = torch.nonzero(s["row_src"][:used] >= 0)[:, 0]
        I = case["inner"]
        if op == "swiglu":
            gu = s["gu"][at].double()
            h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
            out = {}
            if case["h"]:
                out["h"] = s["h"].double()
                out["h"][at] = h
            for name, v in (("h", h),) * bool(case["sf"]) + (("gu", gu),) * case["keep"]:
                codes, sf = _exact_fp8(v, case["sf"])
                out[name + "_codes"], out[name + "_sf"] = (t.double() for t in _stands_for(
                    s[name + "_codes"], s[name + "_sf"]))
                out[name + "_codes"][at], out[name + "_sf"][at] = codes, sf
            return out
        gu = s["gu"][at].double() if "gu" in s else _exact_read(s["gu_codes"][at], s["gu_sf"][at])
        g, u = gu[:, :I], gu[:, I:]
        dh, sg = s["dh"][at].double(), torch.sigmoid(g)
        dgu = s["dgu"].double()
        dgu[at, :I] = dh * u * (sg + g * sg * torch.sigmoid(-g))
        dgu[at, I:] = dh * g * sg
        return {"dgu": dgu}
    E = case["experts"]
    x = _exact_read(s["x"], s["x_sf"]).to(s["dy"].dtype)     # rounded once, where the type holds fewer bits
    dw = torch.zeros(E, case["n"], case["k"], dtype=torch.float64, device="cuda")
    for e in range(E):
        first, n = (0, x.shape[0]) if E == 1 else (int(s["offsets"][e]), int(s["counts"][e]))
        if n:
            dw[e] = s["dy"][first:first + n].double().t() @ x[first:first + n].double()
    return {"dw": dw if E > 1 else dw[0]}
