"""Measured cases of the row operators around the expert products: tokens put
into expert order and back (with their gradients), microscaled 4-bit
quantisation, and the product of two microscaled 4-bit matrices, dense and
over the experts' row segments.

`run` computes a case with the library's entry points when `own` is true and
in elementary torch operations otherwise.

Formats: e2m1 codes, two per byte, the even element in the low nibble; one
UE8M0 code c per 32 elements of a row, standing for 2^(c - 127).  Routing
lists are those of the library's planner: expert e's rows are offsets[e] ..
offsets[e] + counts[e] - 1 of the pool, in ascending slot order, row_src[r]
is the slot f = t * top_k + j of pool row r (-1: padding), src_row[f] the pool
row of slot f (-1: masked).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# the most elements a drawn case of each kind handles: those of the largest listed one
MOST_ROWS = 8192 * 6 * 7168
MOST_QUANT = 65536 * 4096
MOST_FLOP = 2 * 8192 * 8192 * 7168
MOST_WEIGHTS = 32 * 4096 * 4096


def listed():
    return [
        # One token of the pro shape enters the experts: latency alone.
        dict(name="permute 1 token", op="permute", dtype="bf16", tokens=1, top_k=6, width=7168,
             experts=384, align=16, masked=0.0),
        # The pro layer's prompt batch, segments aligned to 128-row tiles.
        dict(name="permute prompt", op="permute", dtype="bf16", tokens=8192, top_k=6, width=7168,
             experts=384, align=128, masked=0.0),
        # Gradient of the gather in a float32 training step, top-8 of 256 with
        # slots dropped by a capacity limit.
        dict(name="permute gradient", op="permute_grad", dtype="f32", tokens=4096, top_k=8,
             width=4096, experts=256, align=1, masked=0.1),
        # A decode batch's expert outputs back to its tokens, in half precision.
        dict(name="combine decode", op="combine", dtype="f16", tokens=128, top_k=6, width=4096,
             experts=256, align=16, masked=0.0),
        # The pro layer's prompt batch back to token order.
        dict(name="combine prompt", op="combine", dtype="bf16", tokens=8192, top_k=6, width=7168,
             experts=384, align=128, masked=0.0),
        # Training: gradients of the expert outputs and of the router weights.
        dict(name="combine gradient", op="combine_grad", dtype="bf16", tokens=4096, top_k=8,
             width=4096, experts=256, align=16, masked=0.1),
        # A few rows of odd width in float32: a small batch's activations.
        dict(name="quantise few rows", op="quantise", dtype="f32", rows=37, cols=2080),
        # The gate and up weights of 16 flash experts, quantised once at loading.
        dict(name="quantise weights", op="quantise", dtype="bf16", rows=65536, cols=4096),
        # One token through one 4-bit matrix: the decode step of a dense layer.
        dict(name="product 1 token", op="product", out="bf16", experts=1, rows=1, n=4096, k=7168,
             align=1),
        # One GPU's 32 resident experts of the flash layer at a decode batch:
        # 768 routed rows, about 24 an expert.
        dict(name="product decode", op="product", out="bf16", experts=32, rows=768, n=4096,
             k=4096, align=1),
        # The same experts on a prompt batch.
        dict(name="product prompt", op="product", out="bf16", experts=32, rows=12288, n=4096,
             k=4096, align=1),
        # A large dense product, the prompt of a dense or shared-expert layer.
        dict(name="product dense", op="product", out="bf16", experts=1, rows=8192, n=8192, k=7168,
             align=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["permute", "permute_grad", "combine", "combine_grad", "quantise", "product",
                     "product", "product"])
    if op == "quantise":
        rows, cols = _log(rng, 1, 65536), 32 * _log(rng, 1, 256)
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]),
                    rows=max(1, min(rows, MOST_QUANT // 2 // cols)), cols=cols)
    if op == "product":
        experts = rng.choice([1, 1, _log(rng, 2, 64)])
        n, k = _log(rng, 16, 8192), 32 * _log(rng, 1, 256)
        if rng.random() < 0.5:
            n = max(16, n // 16 * 16)
        experts = max(1, min(experts, MOST_WEIGHTS // (n * k)))
        rows = min(_log(rng, 1, 12288), MOST_FLOP // (2 * n * k))
        return dict(op=op, out=rng.choice(["bf16", "f16", "f32"]), experts=experts,
                    rows=max(1, rows), n=n, k=k, align=rng.choice([1, 16, 128]))
    top_k = rng.randint(1, 8)
    width = _log(rng, 16, 8192)
    if rng.random() < 0.6:
        width = max(16, width // 8 * 8)
    tokens = max(1, min(_log(rng, 1, 8192), MOST_ROWS // 2 // (top_k * width)))
    return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), tokens=tokens, top_k=top_k,
                width=width, experts=_log(rng, 8, 384), align=rng.choice([1, 16, 64, 128]),
                masked=rng.choice([0.0, 0.0, 0.1, 0.5]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _pool_rows(case):
    """Capacity of the pool: every slot and each expert's padding."""
    slots = case["tokens"] * case["top_k"] if "tokens" in case else case["rows"]
    return slots + case["experts"] * (case["align"] - 1)


def _route(idx, experts, align, pool):
    """The planner's lists for expert ids idx [T, K] (-1: masked)."""
    f = idx.reshape(-1).to(torch.int64)
    n = f.numel()
    key = torch.where(f < 0, experts, f)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    counts.scatter_add_(0, key, torch.ones_like(key))
    seg = (counts[:experts] + align - 1) // align * align
    ends = torch.cumsum(seg, 0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    order = torch.argsort(key, stable=True)
    first = torch.cumsum(counts, 0) - counts       # of each expert in sorted order
    e = key[order]
    routed = e < experts
    rank = torch.arange(n, device="cuda") - first[e]
    at = torch.where(routed, offsets[e.clamp(max=experts - 1)] + rank, pool)
    row_src = torch.full((pool + 1,), -1, dtype=torch.int64, device="cuda")
    row_src[at] = order
    src_row = torch.empty(n, dtype=torch.int64, device="cuda")
    src_row[order] = torch.where(routed, at, -1)
    return {"counts": counts[:experts].int().contiguous(), "offsets": offsets.int(),
            "row_src": row_src[:pool].int().contiguous(), "src_row": src_row.int()}


def _router(g, tokens, experts, top_k, masked):
    """Top-k expert ids and softmax weights of a skewed router, some slots dropped."""
    logits = _randn(g, tokens, experts) + 0.5 * _randn(g, 1, experts)
    top, idx = torch.topk(logits, top_k, dim=1)
    if masked:
        idx = idx.masked_fill(torch.rand(idx.shape, generator=g, device="cuda") < masked, -1)
    return idx, torch.softmax(top, 1).contiguous()


def _quantised(v):
    """Packed e2m1 codes and UE8M0 codes of the rows of v (float32)."""
    q, sf = _round_mx(v)
    mag = q.abs()
    code = torch.where(mag < 2, 2 * mag, torch.where(mag < 4, 2 + mag, 4 + mag / 2))
    code = code.to(torch.uint8) | ((q < 0).to(torch.uint8) << 3)
    m, e = torch.frexp(sf)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 126).to(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "quantise":
        # activations and weights: Gaussian, with a few columns of larger values
        x = _randn(g, case["rows"], case["cols"])
        x = x * (1 + 15 * (torch.rand(1, case["cols"], generator=g, device="cuda") < 0.01).float())
        return {"case": case, "x": x.to(DTYPES[case["dtype"]])}
    if case["op"] == "product":
        E, rows, n, k = case["experts"], case["rows"], case["n"], case["k"]
        pool = _pool_rows(case)
        s = {"case": case}
        if E > 1:
            idx = _router(g, rows, E, 1, 0.0)[0]
            r = _route(idx, E, case["align"], pool)
            s.update(counts=r["counts"], offsets=r["offsets"],
                     most=int(r["counts"].max()))
        else:
            pool = rows
        a = _randn(g, pool, k) * (1 + 15 * (torch.rand(1, k, generator=g, device="cuda") < 0.01).float())
        s["a"], s["a_sf"] = _quantised(a)
        s["b"] = torch.empty(E, n, k // 2, dtype=torch.uint8, device="cuda")
        s["b_sf"] = torch.empty(E, n, k // 32, dtype=torch.uint8, device="cuda")
        for e in range(E):
            s["b"][e], s["b_sf"][e] = _quantised(_randn(g, n, k) / math.sqrt(k))
        s["y"] = torch.zeros(pool, n, dtype=DTYPES[case["out"]], device="cuda")
        return s
    T, K, W = case["tokens"], case["top_k"], case["width"]
    dt = DTYPES[case["dtype"]]
    pool = _pool_rows(case)
    idx, w = _router(g, T, case["experts"], K, case["masked"])
    s = {"case": case, "w": w, **_route(idx, case["experts"], case["align"], pool)}
    if case["op"] == "permute":
        s["x"] = _randn(g, T, W).to(dt)
        s["xp"] = torch.zeros(pool, W, dtype=dt, device="cuda")
    elif case["op"] == "permute_grad":
        s["dxp"] = _randn(g, pool, W).to(dt)
    else:
        s["yp"] = _randn(g, pool, W).to(dt)
        if case["op"] == "combine_grad":
            s["dy"] = _randn(g, T, W).to(dt)
            s["dyp"] = torch.zeros(pool, W, dtype=dt, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms

def _round_mx(v):
    """The e2m1 values (in units of their block's scale) and the blocks' scales of float32 rows:
    the scale is the smallest power of two >= max(amax, 1e-10) / 6, rounding is to nearest even."""
    blk = v.reshape(v.shape[0], -1, 32)
    amax = blk.abs().amax(-1).clamp(min=1e-10)
    m, e = torch.frexp(amax)                       # amax = m 2^e, 0.5 <= m < 1; 6 = 0.75 * 2^3
    sf = torch.ldexp(torch.ones_like(m), torch.where(m > 0.75, e - 2, e - 3))
    q = blk / sf[..., None]
    mag = q.abs()
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0))
    q = torch.copysign(torch.round(mag / step) * step, q)
    return q.reshape(v.shape), sf


def _values(codes, sf):
    """float32 values of packed e2m1 codes [..., K / 2] with UE8M0 codes [..., K / 32]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    mag = (c & 7).float()
    mag = torch.where(mag < 4, 0.5 * mag, torch.where(mag < 6, mag - 2, 2 * mag - 8))
    v = torch.where(c > 7, -mag, mag)
    s = torch.ldexp(torch.ones((), device=codes.device), sf.to(torch.int32) - 127)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _slots(s, rows):
    """float32 rows [pool, W] of every slot, [T, K, W]; a masked slot's are zero."""
    T, K = s["case"]["tokens"], s["case"]["top_k"]
    at = s["src_row"].view(T, K)
    return torch.where((at >= 0)[..., None], rows[at.clamp(min=0).long()].float(), 0.0)


def _to_pool(s, rows, into):
    """rows(t, f) of every routed pool row, zeros in padding; rows past the last segment as in `into`."""
    live = torch.arange(into.shape[0], device="cuda") < s["offsets"][-1]
    f = s["row_src"]
    out = torch.where((f >= 0)[:, None], rows(f.clamp(min=0).long()), 0.0)
    return torch.where(live[:, None], out.to(into.dtype), into)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantise":
        q, sf = _round_mx(s["x"].float())
        v = (q.unflatten(-1, (-1, 32)) * sf[..., None]).flatten(-2)
        return {"values": v.to(s["x"].dtype), "scales": sf}
    if op == "product":
        a, b = _values(s["a"], s["a_sf"]), _values(s["b"], s["b_sf"])
        if case["experts"] == 1:
            return {"y": torch.matmul(a, b[0].t()).to(s["y"].dtype)}
        at = torch.arange(s["most"], device="cuda") + s["offsets"][:-1, None]
        rows = a[at.clamp(max=a.shape[0] - 1).long()]
        y = torch.matmul(rows, b.transpose(1, 2))                  # [E, most, n]
        r = torch.arange(a.shape[0], device="cuda", dtype=torch.int32)
        e = torch.searchsorted(s["offsets"][1:].contiguous(), r, right=True).clamp(max=case["experts"] - 1)
        rank = r - s["offsets"][e]
        live = rank < s["counts"][e]
        y = y[e, rank.clamp(max=s["most"] - 1).long()].to(s["y"].dtype)
        return {"y": torch.where(live[:, None], y, s["y"])}
    if op == "permute":
        return {"xp": _to_pool(s, lambda f: s["x"][f // case["top_k"]], s["xp"])}
    if op == "permute_grad":
        return {"dx": _slots(s, s["dxp"]).sum(1).to(s["dxp"].dtype)}
    if op == "combine":
        return {"y": (_slots(s, s["yp"]) * s["w"][..., None]).sum(1).to(s["yp"].dtype)}
    dy, w = s["dy"].float(), s["w"].reshape(-1)
    dyp = _to_pool(s, lambda f: dy[f // case["top_k"]] * w[f][:, None], s["dyp"])
    return {"dyp": dyp, "dw": (_slots(s, s["yp"]) * dy[:, None, :]).sum(-1)}


# ---------------------------------------------------------------- one pass

def run(s):
    if not own:
        return _plain(s)
    import fp8_grouped_gemm_amd as moe
    case = s["case"]
    op = case["op"]
    if op == "quantise":
        codes, sf = moe.moe_quantize_mxfp4(s["x"])
        return {"values": moe.moe_dequantize_mxfp4(codes, sf, s["x"].dtype),
                "scales": sf.view(torch.float8_e8m0fnu).float()}
    if op == "product":
        if case["experts"] == 1:
            return {"y": moe.moe_gemm_mxfp4(s["a"], s["a_sf"], s["b"][0], s["b_sf"][0], out=s["y"])}
        return {"y": moe.moe_gemm_mxfp4(s["a"], s["a_sf"], s["b"], s["b_sf"], offsets=s["offsets"],
                                        counts=s["counts"], out=s["y"])}
    if op == "permute":
        return {"xp": moe.moe_permute(s["x"], s["row_src"], s["src_row"], s["offsets"], out=s["xp"])}
    if op == "permute_grad":
        return {"dx": moe.moe_permute_bwd(s["dxp"], s["src_row"], case["tokens"])}
    if op == "combine":
        return {"y": moe.moe_unpermute(s["yp"], s["src_row"], case["tokens"], s["w"])}
    dyp, dw = moe.moe_unpermute_bwd(s["dy"], s["yp"], s["row_src"], s["src_row"], s["offsets"],
                                    s["w"], dyp=s["dyp"])
    return {"dyp": dyp, "dw": dw}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "quantise":
        n = case["rows"] * case["cols"]
        # x read, codes and scales written and read again, values written
        return {"bytes": n * (2 * SIZE[case["dtype"]] + 2 * (0.5 + 1 / 32)), "flops": 4 * n}
    if op == "product":
        m, n, k, E = case["rows"], case["n"], case["k"], case["experts"]
        touched = E * (1 - (1 - 1 / E) ** m)           # experts with a row, routed uniformly
        return {"bytes": (m + touched * n) * (k / 2 + k / 32) + m * n * SIZE[case["out"]],
                "flops": 2 * m * n * k}
    slots = case["tokens"] * case["top_k"] * (1 - case["masked"])
    token, slot = case["tokens"] * case["width"], slots * case["width"]
    size, index = SIZE[case["dtype"]], 4 * case["tokens"] * case["top_k"]
    if op == "permute":
        return {"bytes": (token + slot) * size + 2 * index, "flops": 0}
    if op == "permute_grad":
        return {"bytes": (token + slot) * size + index, "flops": slot}
    if op == "combine":
        return {"bytes": (token + slot) * size + 2 * index, "flops": 2 * slot}
    return {"bytes": (token + 2 * slot) * size + 4 * index, "flops": 3 * slot}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_values(codes, sf):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    v = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device="cuda")
    v[:, 0::2] = table[(codes % 16).long()]
    v[:, 1::2] = table[(codes // 16).long()]
    return v * torch.exp2(sf.double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        x = s["x"].double()
        values, scales = torch.empty_like(x), torch.empty(x.shape[0], x.shape[1] // 32, dtype=torch.float64, device="cuda")
        table = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        for at in range(0, x.shape[0], 4096):
            blk = x[at:at + 4096].unflatten(1, (-1, 32))
            least = blk.abs().amax(-1).clamp(min=1e-10) / 6
            # a value within 1e-12 of a power of two is one: float32 quotients by 6 are no nearer
            sf = torch.exp2(torch.ceil(torch.log2(least) - 1e-12))
            mag = (blk / sf[..., None]).abs()
            best = torch.zeros_like(mag)
            off = torch.full_like(mag, math.inf)
            for c in (0, 2, 4, 6, 1, 3, 5, 7):             # the even code wins a tie
                nearer = (mag - table[c]).abs() < off
                best = torch.where(nearer, table[c], best)
                off = torch.where(nearer, (mag - table[c]).abs(), off)
            values[at:at + 4096] = (torch.sign(blk) * best * sf[..., None]).flatten(1)
            scales[at:at + 4096] = sf
        return {"values": values, "scales": scales}
    if op == "product":
        y = s["y"].double()
        for e in range(case["experts"]):
            first, n = (0, y.shape[0]) if case["experts"] == 1 else (int(s["offsets"][e]), int(s["counts"][e]))
            if n:
                y[first:first + n] = _exact_values(s["a"][first:first + n], s["a_sf"][first:first + n]) @ \
                    _exact_values(s["b"][e], s["b_sf"][e]).t()
        return {"y": y}
    T, K, W = case["tokens"], case["top_k"], case["width"]
    at = s["src_row"].view(T, K).long()
    used = int(s["offsets"][-1])
    zeros = lambda n: torch.zeros(n, W, dtype=torch.float64, device="cuda")
    if op == "permute":
        xp = s["xp"].double()
        xp[:used] = 0
        for j in range(K):
            t = torch.nonzero(at[:, j] >= 0)[:, 0]
            xp[at[t, j]] = s["x"][t].double()
        return {"xp": xp}
    if op in ("permute_grad", "combine"):
        rows, w = (s["dxp"], torch.ones_like(s["w"])) if op == "permute_grad" else (s["yp"], s["w"])
        out = zeros(T)
        for j in range(K):
            t = torch.nonzero(at[:, j] >= 0)[:, 0]
            out[t] += w[t, j].double()[:, None] * rows[at[t, j]].double()
        return {"dx" if op == "permute_grad" else "y": out}
    dyp, dw = s["dyp"].double(), torch.zeros(T, K, dtype=torch.float64, device="cuda")
    dyp[:used] = 0
    for j in range(K):
        t = torch.nonzero(at[:, j] >= 0)[:, 0]
        dyp[at[t, j]] = s["w"][t, j].double()[:, None] * s["dy"][t].double()
        dw[t, j] = (s["dy"][t].double() * s["yp"][at[t, j]].double()).sum(1)
    return {"dyp": dyp, "dw": dw}
