"""Plain 64-bit forms of the row operators, routing lists for their tests and
the error bounds the tests hold them to (no code of the library)."""
import math

import numpy as np
import torch

U32 = 2.0 ** -24  # a float32 rounding is off by at most this part of the value
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half the spacing of the type's subnormals: the error of rounding near zero."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def route(idx, experts, align):
    """The planner's lists for expert ids idx [T, K] (numpy, -1: masked)."""
    T, K = idx.shape
    flat = idx.reshape(-1)
    pool = T * K + experts * (align - 1)
    row_src = np.full(pool, -1, np.int32)
    src_row = np.full(T * K, -1, np.int32)
    offsets, counts, at = [0], [], 0
    for e in range(experts):
        f = np.nonzero(flat == e)[0]
        row_src[at:at + f.size] = f
        src_row[f] = at + np.arange(f.size)
        counts.append(f.size)
        at += -(-f.size // align) * align
        offsets.append(at)
    return {"row_src": row_src, "src_row": src_row, "offsets": np.array(offsets, np.int32),
            "counts": np.array(counts, np.int32), "pool": pool}


def draw_idx(rng, T, K, E, masked):
    idx = np.stack([rng.permutation(E)[:K] for _ in range(T)]) if T else np.zeros((0, K), np.int64)
    idx = idx.astype(np.int64)
    idx[rng.random(idx.shape) < masked] = -1
    return idx


def dev(lists):
    return {k: torch.from_numpy(v).cuda() for k, v in lists.items() if isinstance(v, np.ndarray)}


# --- plain forms: float64 numpy in, float64 out --------------------------------

def permute(x, lists, before):
    out, used, K = before.copy(), lists["offsets"][-1], lists["src_row"].size // max(1, len(x))
    for r in range(used):
        f = lists["row_src"][r]
        out[r] = x[f // K] if f >= 0 else 0
    return out


def token_sums(rows, lists, T, w=None):
    """(sums, sums of magnitudes) of each token's slots."""
    K = lists["src_row"].size // max(1, T)
    s, m = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(K):
            r = lists["src_row"][t * K + j]
            if r >= 0:
                v = rows[r] * (1.0 if w is None else w[t, j])
                s[t] += v
                m[t] += abs(v)
    return s, m


def unpermute_grads(dy, yp, lists, w, before):
    T = len(dy)
    K = lists["src_row"].size // max(1, T)
    dyp, dw, mag = before.copy(), np.zeros((T, K)), np.zeros((T, K))
    for r in range(lists["offsets"][-1]):
        f = lists["row_src"][r]
        dyp[r] = dy[f // K] * w[f // K, f % K] if f >= 0 else 0
    for f, r in enumerate(lists["src_row"]):
        if r >= 0:
            dw[f // K, f % K] = dy[f // K] @ yp[r]
            mag[f // K, f % K] = abs(dy[f // K]) @ abs(yp[r])
    return dyp, dw, mag


def quantised(x):
    """(values in units of the block scale, scale exponents) of float64 rows by the definition:
    the smallest power of two >= max(amax, 1e-10) / 6, nearest e2m1 value, ties to the even code."""
    blk = x.reshape(x.shape[0], x.shape[1] // 32, 32)
    # 1e-10 as the float32 the rule uses; amax <= 6 * 2^e compared exactly
    amax = np.maximum(abs(blk).max(-1), float(np.float32(1e-10)))
    e = np.floor(np.log2(amax)).astype(np.int64) - 4
    for _ in range(4):
        e = np.where(amax > 6 * np.exp2(e.astype(float)), e + 1, e)
    mag = abs(blk) / np.exp2(e.astype(float))[..., None]
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])             # even codes first: they win ties
    best = order[np.argmin(abs(mag[..., None] - E2M1[order]), -1)]
    q = np.where(np.signbit(blk), -1.0, 1.0) * E2M1[best]
    return q.reshape(x.shape), e


def values(codes, sf):
    """float64 values of packed codes [..., K/2] and scale codes [..., K/32] (0xFF: NaN)."""
    c = codes.astype(np.int64)
    v = np.stack([E2M1[c & 15], E2M1[c >> 4]], -1).reshape(*c.shape[:-1], -1)
    s = np.where(sf == 255, np.nan, np.exp2(sf.astype(float) - 127))
    return v * np.repeat(s, 32, -1)


def rounded(v, dtype):
    """float64 -> dtype -> float64 by one rounding to nearest even."""
    if dtype == torch.float32:
        return v.astype(np.float32).astype(np.float64)
    info = torch.finfo(dtype)
    digits = -int(math.log2(info.eps)) + 1                 # of the significand
    lowest = int(math.log2(info.smallest_normal)) - digits + 1
    m, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - digits, lowest))
    r = np.rint(v / step) * step
    return np.where(abs(r) > info.max, np.copysign(np.inf, r), r)
