"""Plain 64-bit forms of the operators around the experts' products, and of the
8-bit rows they write (no code of the library)."""
import numpy as np
import torch

import ops_util as ou

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = {0: 128, 1: 32}                                       # MOE_SF_F32_128, MOE_SF_UE8M0_32
U32 = ou.U32

_c = np.arange(256)
_e, _m = (_c >> 3) & 15, _c & 7
E4M3 = np.where(_e > 0, (8 + _m) * np.exp2(_e - 10.0), _m * 2.0 ** -9) * np.where(_c > 127, -1, 1)
E4M3[[127, 255]] = np.nan


def f64(t):
    return t.double().cpu().numpy()


def within(got, want, bound):
    """got (numpy or tensor) within bound of want, both NaN or infinite in the same places."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (got.shape, want.shape)
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True)
    off = np.where(odd, 0, abs(got - np.where(odd, 0, want)))
    bound = np.broadcast_to(bound, off.shape)
    assert np.all(off <= bound), (float(off.max()), float((off / np.maximum(bound, 1e-300))[~odd].max()))


def overflowed(v, dtype):
    """Values beyond the type's range (its largest and half a step) as the infinities they round to."""
    top = torch.finfo(dtype).max
    return np.where(abs(v) >= top * (1 + torch.finfo(dtype).eps / 4), np.copysign(np.inf, v), v)


def rounded_bound(value, inner, dtype):
    """Of a value off by `inner` that is rounded once to dtype."""
    return inner + ou.half_step(dtype) * (abs(value) + inner) + ou.least(dtype)


# --- 8-bit rows ------------------------------------------------------------------

def scales(sf):
    """float64 scales of a scale tensor (uint8: powers of two, 0xFF NaN)."""
    v = f64(sf)
    return v if sf.dtype == torch.float32 else np.where(v == 255, np.nan, np.exp2(v - 127))


def read(codes, sf):
    s = scales(sf)
    return E4M3[codes.cpu().numpy()] * np.repeat(s, codes.shape[1] // s.shape[1], 1)


def quantised(v, fmt):
    """(codes, sf) of float32 rows by moe_quantize_act's rule: float32 quotients, rounded to nearest even."""
    v = v.detach().float().cpu()
    blk = v.view(v.shape[0], v.shape[1] // BLOCK[fmt], BLOCK[fmt])
    s = blk.abs().amax(-1).clamp(min=1e-10) / 448.0
    if fmt == 1:
        m, e = torch.frexp(s)
        code = torch.where(m == 0.5, e - 1, e) + 127
        s, sf = torch.ldexp(torch.ones_like(m), code - 127), code.to(torch.uint8)
    else:
        sf = s
    q = (blk / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(v.shape), sf


def same_codes(codes, sf, v, fmt):
    """codes and sf are those of the float32 rows v, bit for bit."""
    c, s = quantised(v, fmt)
    assert torch.equal(codes.cpu(), c) and torch.equal(sf.cpu(), s)


def near_codes(codes, sf, want, rel, fmt):
    """codes and sf stand for float64 rows `want` whose float32 form may be off by `rel` of each value."""
    s = scales(sf)
    amax = np.maximum(abs(want).reshape(want.shape[0], want.shape[1] // BLOCK[fmt], BLOCK[fmt]).max(-1), float(np.float32(1e-10))) / 448
    if fmt == 1:                                              # a power of two: the least that covers it
        assert np.all(s >= amax * (1 - rel - 2 * U32)) and np.all(s < 2 * amax * (1 + rel + 2 * U32))
    else:
        within(s, amax, (rel + 2 * U32) * amax)
    wide = np.repeat(s, BLOCK[fmt], 1)
    v = abs(want) * (1 + rel)
    # half a step of e4m3 (2^-4 of the value, 2^-10 of the scale below its normals), and the quotient's rounding
    within(read(codes, sf), want, rel * abs(want) + np.maximum(2.0 ** -4 * v, 2.0 ** -10 * wide) * (1 + 4 * U32))


# --- the router ------------------------------------------------------------------

def gate_scores(l, sigmoid):
    with np.errstate(all="ignore"):
        if sigmoid:
            return 1 / (1 + np.exp(-l))
        p = np.exp(l - l.max(1, keepdims=True))
        return p / p.sum(1, keepdims=True)


def gate(l, K, bias, mask, sigmoid, groups, top_groups, group_top, renorm, scale):
    """(idx, w, rounding steps of w) of float64 logits [T, E]."""
    T, E = l.shape
    s = gate_scores(l, sigmoid)
    idx, w = np.full((T, K), -1), np.zeros((T, K))
    first = lambda key, ids: sorted(ids, key=lambda i: (-np.inf if np.isnan(key[i]) else -key[i], i))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        b = np.zeros(E) if bias is None else bias
        on = [e for e in range(E) if l[t, e] != -np.inf and b[e] != -np.inf]
        key = l[t] if bias is None else s[t] + b
        if groups > 1:
            size = E // groups
            by = s[t] if bias is None and group_top > 1 else key
            score = np.full(groups, -np.inf)
            for g in range(groups):
                members = first(by, [e for e in on if e // size == g])[:group_top]
                if members:
                    score[g] = sum(by[e] for e in members)
            # (a group with nothing to offer cannot matter)
            kept = first(score, range(groups))[:top_groups]
            on = [e for e in on if e // size in kept]
        best = first(key, on)[:K]
        idx[t, :len(best)] = best
        v = s[t, best]
        if renorm and len(best):
            v = v / (v.sum() + 1e-20)
        w[t, :len(best)] = scale * v
    return idx, w


def spread(l):
    """The largest |l - max| of each token's finite logits: what exp(l - max) loses roundings by."""
    fin = np.isfinite(l)
    d = np.where(fin, l, -np.inf).max(1) - np.where(fin, l, np.inf).min(1)
    return np.maximum(d, 0)[:, None]


def gate_steps(l, E):
    """float32 roundings of one score: exp (2, and |l - max| of its argument's), the sum's run and
    tree over the row with its terms' own, the quotient."""
    return 2 * spread(l) + E / 64 + 14


def gate_grad(l, idx, dw, sigmoid, renorm, scale):
    """(dlogits, sum of the magnitudes it is made of)."""
    T, E = l.shape
    s = gate_scores(l, sigmoid)
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        on = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
        if not on:
            continue
        p, g = s[t, idx[t, on]], scale * dw[t, on]
        dp, mdp, q, mq = g.copy(), abs(g), (g * p).sum(), (abs(g) * p).sum()
        if renorm:
            D = p.sum() + 1e-20
            dp = ((g[:, None] - g[None]) * p[None]).sum(1) / D / D + 1e-20 * g / D / D
            mdp = (abs(g[:, None] - g[None]) * p[None]).sum(1) / D / D + 1e-20 * abs(g) / D / D
            q, mq = 1e-20 * q / D / D, 1e-20 * mq / D / D
        d, m = np.zeros(E), np.zeros(E)
        np.add.at(d, idx[t, on], dp)
        np.add.at(m, idx[t, on], mdp)
        if sigmoid:
            e = np.exp(-abs(l[t]))
            out[t], mag[t] = d * e / (1 + e) ** 2, m * e / (1 + e) ** 2
        else:
            out[t], mag[t] = s[t] * (d - q), s[t] * (m + mq)
    return out, mag


# --- norm and activation ---------------------------------------------------------

def norm(z, weight, eps):
    rstd = 1 / np.sqrt((z * z).mean(1) + eps)
    return rstd, z * rstd[:, None] * weight


def norm_steps(W):
    """float32 roundings of rstd and y: a thread's run of the sum (16, or W / 1024 and its last step),
    the tree of a wave and of 16 waves, halved by the root; mean, eps, root, quotient; two products."""
    return (max(16, W / 1024 + 8) + 6 + 16) / 2 + 4 + 2


def norm_grads(dy, z, rstd, weight, dz):
    """(dx, its magnitudes, dw, its magnitudes)."""
    xh, g = z * rstd[:, None], dy * weight
    c, mc = (g * xh).mean(1, keepdims=True), abs(g * xh).mean(1, keepdims=True)
    r = rstd[:, None]
    dx, mag = r * (g - xh * c) + dz, r * (abs(g) + abs(xh) * mc) + abs(dz)
    return dx, mag, (dy * xh).sum(0), abs(dy * xh).sum(0)


def sigmoid(g):
    with np.errstate(all="ignore"):
        return 1 / (1 + np.exp(-g))


def swiglu(gu, clamp=0.0):
    g, u = np.split(gu, 2, 1)
    if clamp > 0:
        g, u = np.clip(g, -clamp, clamp), np.clip(u, -clamp, clamp)
    return g * sigmoid(g) * u


def swiglu_grads(dh, gu, clamp=0.0):
    """(dgu, its magnitudes)."""
    g, u = np.split(gu, 2, 1)
    og, ou_ = (abs(g) > clamp, abs(u) > clamp) if clamp > 0 else (np.zeros(g.shape, bool),) * 2
    if clamp > 0:
        g, u = np.clip(g, -clamp, clamp), np.clip(u, -clamp, clamp)
    s, r = sigmoid(g), sigmoid(-g)
    dg, mg = dh * u * s * (1 + g * r), abs(dh * u * s) * (1 + abs(g) * r)
    du = dh * g * s
    return (np.concatenate([np.where(og, 0, dg), np.where(ou_, 0, du)], 1),
            np.concatenate([np.where(og, 0, mg), np.where(ou_, 0, abs(du))], 1))
