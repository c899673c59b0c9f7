// The router's choice of experts and its gradient (include/moe_ops.h: moe_gate,
// moe_gate_bwd).
//   s = softmax(l) or sigmoid(l),  c = s + bias (without a bias: the order of l)
//   the K largest c, of the best groups' experts;  w_j = scale s_j / (S + 1e-20), S = sum s_j
// and with D = S + 1e-20, g = scale dw
//   dp_j = (sum_i p_i (g_j - g_i) + 1e-20 g_j) / D^2,  q = sum_j dp_j p_j = 1e-20 sum g p / D^2
//   softmax dl_e = s_e (dp_e - q),  sigmoid dl_e = dp_e s_e (1 - s_e)
// (dp as a sum of differences: g_j - sum g p / D loses everything where one slot
// holds all the weight; without renorm dp_j = g_j, q = sum g p).
//
// One wave per token, each lane a run of N adjacent experts of a group in registers, a group's
// runs in 1 to 32 lanes (a power of two), so that the lowest lane holding a maximum also holds
// the lowest id and a group's best are a few lane exchanges away.  Values are compared as
// integers in the order of the values (NaN on top, 0 for experts that cannot be
// chosen), whose maximum over a wave is a handful of instructions.  c and the groups' sums
// are formed in f32 first: where neighbours of the choice are further apart than f32
// can be off (all but a few tokens of ordinary logits), the choice is that of the formula;
// elsewhere the token's c are formed in 64 bits.
//
// Instructions bound it: 8192 tokens of 256 experts, sigmoid and bias, 4 of 8 groups, top-8
// take 11.1 us of which 10 are the call, 32768 tokens 30.3 (27.8 if the kernel had no 64-bit part, which one
// token in a thousand needs), where the logits take 7 to read.  The gradient moves 52 MB of
// 32768 x 384 bf16 in 13.5 us, 3.7 TB/s; waves that walk the tokens and load the next one
// early take 16.0.  Runs of at most eight experts make most calls; 32768 tokens of 512 experts,
// 8 groups, top-8: 47 - 50 us, of 1024 with runs of 16 92, of 1000 in 10 groups with runs of 25 (in
// instances for 32) 410 - 480: a run's sort grows with its square.
#include "../../include/moe_ops.h"
#include "ops_internal.h"
#include "rows_device.h"

#include <type_traits>

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr float kTiny = 1e-20f;  // added to the chosen scores' sum

__device__ __forceinline__ uint32_t lane_of(uint32_t v, int lane)
{
    return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

__device__ __forceinline__ float lane_of(float v, int lane)
{
    return __uint_as_float(lane_of(__float_as_uint(v), lane));
}

// v from another lane of the 16-lane row, in a form that the compiler folds into the
// instruction that takes it.
template <int CTRL>
__device__ __forceinline__ uint32_t swap(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

template <int CTRL>
__device__ __forceinline__ float swap(float v)
{
    return __uint_as_float(swap<CTRL>(__float_as_uint(v)));
}

template <int CTRL>
__device__ __forceinline__ uint64_t swap(uint64_t v)
{
    return (uint64_t)swap<CTRL>((uint32_t)(v >> 32)) << 32 | swap<CTRL>((uint32_t)v);
}

__device__ __forceinline__ uint64_t lane_of(uint64_t v, int lane)
{
    return (uint64_t)lane_of((uint32_t)(v >> 32), lane) << 32 | lane_of((uint32_t)v, lane);
}

constexpr int kNext = 0xB1, kPairs = 0x4E, kHalves = 0x141, kRow = 0x140;  // neighbours, pairs, mirrored halves and rows

// The maximum over the wave, in every lane (a scalar).
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = max(v, swap<kNext>(v));
    v = max(v, swap<kPairs>(v));
    v = max(v, swap<kHalves>(v));
    v = max(v, swap<kRow>(v));
    return max(max(lane_of(v, 0), lane_of(v, 16)), max(lane_of(v, 32), lane_of(v, 48)));
}

__device__ __forceinline__ float row_sum(float v)
{
    v += swap<kNext>(v);
    v += swap<kPairs>(v);
    v += swap<kHalves>(v);
    v += swap<kRow>(v);
    return v;
}

__device__ __forceinline__ float wave_sum(float v)
{
    v = row_sum(v);
    return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

// The sum over the first n lanes, the others' values being 0.
__device__ __forceinline__ float slots_sum(float v, int n)
{
    return n <= 16 ? lane_of(row_sum(v), 0) : wave_sum(v);
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int x = 1; x < 64; x *= 2)
        v += __shfl_xor(v, x);
    return v;
}

// Integers in the order of the values: -0 counts as 0, NaN as the largest, and
// 0 is below every value's (-infinity is no choice and never asked for).
__device__ __forceinline__ uint32_t order32(float v)
{
    const uint32_t u = __float_as_uint(v + 0.f);
    return v != v ? 0xFFFFFFFFu : u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float from_order32(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ uint64_t order64(double v)
{
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return v != v ? ~UINT64_C(0) : u ^ ((uint64_t)((int64_t)u >> 63) | UINT64_C(1) << 63);
}

__device__ __forceinline__ double from_order64(uint64_t k)
{
    return __longlong_as_double((long long)(k >> 63 ? k ^ UINT64_C(1) << 63 : ~k));
}

// A lane's N experts of a row of n, from e0 on; -infinity past the row.
template <class E, int N>
__device__ __forceinline__ void load_run(const char* row, int e0, int n, float* f)
{
    alignas(16) char raw[N * E::SIZE];
    if (e0 + N <= n) {
        __builtin_memcpy(raw, row + (int64_t)e0 * E::SIZE, N * E::SIZE);
#pragma unroll
        for (int i = 0; i < N; ++i)
            f[i] = E::load(raw + i * E::SIZE);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            f[i] = e0 + i < n ? E::load(row + (int64_t)(e0 + i) * E::SIZE) : -INFINITY;
    }
}

template <class E, int N>
__device__ __forceinline__ void store_run(char* row, int e0, int n, const float* f)
{
    if (e0 + N <= n) {
        alignas(16) char raw[N * E::SIZE];
#pragma unroll
        for (int i = 0; i < N; ++i)
            E::store(raw + i * E::SIZE, f[i]);
        __builtin_memcpy(row + (int64_t)e0 * E::SIZE, raw, N * E::SIZE);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (e0 + i < n)
                E::store(row + (int64_t)(e0 + i) * E::SIZE, f[i]);
    }
}

// exp by the hardware's 2^x: off by 1.25 |x| + 2 roundings (the product's, and a quarter of log2 e),
// zero below 2^-126.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// The same for x <= 0 with what the product lost as a factor: off by 4 roundings whatever x is (2
// of 2^x, 1 of the last sum, less than 1 of what is left out); zero from -104 on, as
// -infinity has no lost part.
__device__ __forceinline__ float near_exp(float x)
{
    constexpr float kLog2e = 1.44269504f, kRest = 1.92596303e-8f;  // (their sum: log2 e to 2^-50)
    const float p = x * kLog2e, lost = __builtin_fmaf(x, kRest, __builtin_fmaf(x, kLog2e, -p));
    const float e = __builtin_amdgcn_exp2f(p);
    return x < -104.f ? 0.f : __builtin_fmaf(e * lost, 0.693147181f, e);
}

// m, the terms exp(l - m) and their sum over the row (m passes NaN over, the sum does not).
// NEAR: the terms are results.
template <bool NEAR, int N>
__device__ __forceinline__ float softmax_sum(const float* l, float& m, float* e)
{
    m = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i)
        m = fmaxf(m, l[i]);
    m = from_order32(wave_max(order32(m)));
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        z += e[i] = NEAR ? near_exp(l[i] - m) : fast_exp(l[i] - m);
    return wave_sum(z);
}

// The hardware's reciprocal, here and below: a Newton step behind each left the weights of 2^18 tokens
// as they are (softmax, renormalised) or a little further off (mean 0.61 roundings for 0.54, sigmoid).
__device__ __forceinline__ float sigmoid(float l) { return __builtin_amdgcn_rcpf(1.f + expf(-l)); }

// Whether two f32 values of c, above >= below, are too near for their order to be sure; in
// roundings u = 2^-24, with `off` for what two scores can be off by:
//   sigmoid: 1 + exp and its reciprocal 3, exp's own (1.5 |x| + 2) s (1 - s) below 1: 8 of two
//   softmax: s <= 1 / z; e^-x: (2.5 |x| + 2) e^-x below 3; z: the mean of 2.5 |x| over the terms
//            below 2.5 log E, 2, and 22 of its sum; 2 of 1 / z: 94 / z of two
// and one of |c| each for the bias' sum.
__device__ __forceinline__ float off_by(bool softmax, float rz) { return softmax ? 128.f * rz : 16.f; }

__device__ __forceinline__ bool near(float above, float below, float off)
{
    return !(above - below > 0x1p-24f * (off + 4.f * fabsf(above)));
}

// Whether f32 may have ranked a group that is `in` above one that is not and ought to be: `sum` is
// that of the lane's group, `any` whether it has one.  Every group has its own error, as what is
// left of large terms that cancel is wrong by their size, and one that is far off may stand
// anywhere in the ranking.  In u, of n terms whose magnitudes come to `size`: off / 2 of each
// score, n roundings of |c|, n - 1 of partial sums, one of the bound formed here.
__device__ __forceinline__ bool near_sums(bool any, bool in, float sum, float off, int n, float size)
{
    const float err = 0x1p-24f * (float)n * (0.5f * off + 3.f * size), least = sum - err, most = sum + err;
    // (a bound that is NaN outdoes all others, comes back as NaN and compares as near)
    const uint32_t worst = wave_max(any && in ? (least != least ? 0xFFFFFFFFu : ~order32(least)) : 0u);
    const uint32_t best = wave_max(any && !in ? order32(most) : 0u);
    return worst != 0 && best != 0 && !(from_order32(~worst) > from_order32(best));
}

// The largest key of the wave: its lane (the lowest of equals); 0 if all keys are 0.
template <bool WIDE>
__device__ __forceinline__ uint32_t wave_best(uint32_t hi, uint32_t lo, int& lane)
{
    const uint32_t top = wave_max(hi);
    uint64_t who = __ballot(hi == top);
    if (WIDE && (who & (who - 1))) {
        const uint32_t low = wave_max(hi == top ? lo : 0u);
        who = __ballot(hi == top && lo == low);
    }
    lane = __builtin_ctzll(who);
    return top;
}

__device__ __forceinline__ double from_key(uint64_t k) { return from_order64(k); }
__device__ __forceinline__ float from_key(uint32_t k) { return from_order32(k); }
__device__ __forceinline__ uint64_t to_key(double v) { return order64(v); }
__device__ __forceinline__ uint32_t to_key(float v) { return order32(v); }

// Where the experts lie: a group's in 1 << shift lanes, its first N in the first of them.
struct Layout {
    int shift, group_size;
};

// Takes the experts of other than the best groups out (their keys become 0).  `sums`: the
// groups' sums are of values that may be `off`; true then if another choice of groups may be the
// formula's.  WIDE: keys of 64 bits.
template <int N, bool WIDE>
__device__ __forceinline__ bool keep_groups(const GateArgs& a, int shift, int lane, bool sums, float off, uint32_t* hi,
                                            uint32_t* lo)
{
    using Key = std::conditional_t<WIDE, uint64_t, uint32_t>;
    const int lanes = 1 << shift;
    const auto high = [](Key x, Key y) { return x > y ? x : y; };
    const auto low = [](Key x, Key y) { return x > y ? y : x; };
    const auto key = [&](int i) { return WIDE ? (Key)((uint64_t)hi[i] << 32 | lo[i]) : (Key)hi[i]; };
    const auto far = [](Key x) { return (Key)__shfl_xor((unsigned long long)x, 16); };
    Key group = 0;
    float size = 0.f;  // magnitudes of the group's sum
    if (a.group_top <= 2) {
        Key one = key(0), two = 0;
#pragma unroll
        for (int i = 1; i < N; ++i) {
            two = high(two, low(one, key(i)));
            one = high(one, key(i));
        }
        const auto merge = [&](Key b1, Key b2) {
            two = high(high(two, b2), low(one, b1));
            one = high(one, b1);
        };
        if (lanes > 1)
            merge(swap<kNext>(one), swap<kNext>(two));
        if (lanes > 2)
            merge(swap<kPairs>(one), swap<kPairs>(two));
        if (lanes > 4)
            merge(swap<kHalves>(one), swap<kHalves>(two));
        if (lanes > 8)
            merge(swap<kRow>(one), swap<kRow>(two));
        if (lanes > 16) {
            const Key b1 = far(one), b2 = far(two);
            merge(b1, b2);
        }
        group = one;
        if (a.group_top == 2 && two != 0) {
            const auto first = from_key(one), second = from_key(two);
            group = to_key(first + second);
            size = fabsf((float)first) + fabsf((float)second);
        } else if (one != 0) {
            size = fabsf((float)from_key(one));
        }
    } else {
        // the largest of what is left, as often as asked for; the lowest lane that holds it gives it up
        Key left[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            left[i] = key(i);
        std::conditional_t<WIDE, double, float> sum = 0;
        bool any = false;
        for (int p = 0; p < a.group_top; ++p) {
            Key own = left[0];
#pragma unroll
            for (int i = 1; i < N; ++i)
                own = high(own, left[i]);
            Key top = own;
            if (lanes > 1)
                top = high(top, swap<kNext>(top));
            if (lanes > 2)
                top = high(top, swap<kPairs>(top));
            if (lanes > 4)
                top = high(top, swap<kHalves>(top));
            if (lanes > 8)
                top = high(top, swap<kRow>(top));
            if (lanes > 16) {
                const Key other = far(top);
                top = high(top, other);
            }
            const uint64_t who = __ballot(own == top) >> (lane & ~(lanes - 1));
            bool gives = __builtin_ctzll(who) == (lane & (lanes - 1));
            if (top != 0) {
                const auto v = from_key(top);
                sum += v;
                size += fabsf((float)v);
                any = true;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const bool this_one = gives && left[i] == top;
                left[i] = this_one ? 0 : left[i];
                gives = gives && !this_one;
            }
        }
        group = any ? to_key(sum) : 0;
    }
    bool close = false;
    const int own = lane >> shift;
    if (a.groups <= 16) {
        // a group's rank: how many are above it
        int rank = own < a.groups ? 0 : 64;
        for (int g = 0; g < a.groups; ++g) {
            const Key other = lane_of(group, g << shift);
            rank += other > group || (other == group && g < own);
        }
        if (!WIDE && sums)
            close = near_sums(group != 0, rank < a.top_groups, from_order32((uint32_t)group), off, a.group_top, size);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (rank >= a.top_groups)
                hi[i] = lo[i] = 0;
        return close;
    }
    // (one lane stands for a group)
    Key left = (lane & (lanes - 1)) != 0 ? (Key)0 : group;
    uint64_t kept = 0;
    for (int p = 0; p < a.top_groups; ++p) {
        int from;
        const uint32_t top = WIDE ? wave_best<true>((uint32_t)((uint64_t)left >> 32), (uint32_t)left, from)
                                  : wave_best<false>((uint32_t)left, 0u, from);
        if (top == 0)
            break;
        kept |= UINT64_C(1) << (from >> shift);
        if (lane == from)
            left = 0;
    }
    if (!WIDE && sums)
        close = near_sums(group != 0, kept >> own & 1, from_order32((uint32_t)group), off, a.group_top, size);
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (!(kept >> own & 1))
            hi[i] = lo[i] = 0;
    return close;
}

// The K largest keys, the j-th's expert in lane j (-1: there is none).  Each lane sorts its
// own, equal ones by id, and shifts them down as they are taken.  `sums`: true if two
// that follow one another, the last one in and the first one out among them, are too near.
template <int N, bool WIDE>
__device__ __forceinline__ bool pick(int K, int lane, int e0, bool sums, float off, uint32_t* hi, uint32_t* lo, int& mine)
{
    int id[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        id[i] = e0 + i;
#pragma unroll
    for (int phase = 0; phase < N; ++phase)
#pragma unroll
        for (int i = phase & 1; i + 1 < N; i += 2) {
            const bool above = hi[i + 1] > hi[i] || (WIDE && hi[i + 1] == hi[i] && lo[i + 1] > lo[i]);
            const int one = id[i], two = id[i + 1];
            id[i] = above ? two : one;
            id[i + 1] = above ? one : two;
            const uint32_t h1 = hi[i], h2 = hi[i + 1], l1 = lo[i], l2 = lo[i + 1];
            hi[i] = above ? h2 : h1;
            hi[i + 1] = above ? h1 : h2;
            if (WIDE) {
                lo[i] = above ? l2 : l1;
                lo[i + 1] = above ? l1 : l2;
            }
        }
    mine = -1;
    int top_of = 0, n = 0;  // lane j: the j-th key
    uint32_t out = 0;       // the first one that is not taken
    for (; n <= K; ++n) {
        int from;
        out = wave_best<WIDE>(hi[0], lo[0], from);
        if (out == 0 || n == K)
            break;
        const int taken = (int)lane_of((uint32_t)id[0], from);
        mine = lane == n ? taken : mine;
        top_of = lane == n ? (int)out : top_of;
        if (lane == from) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                hi[i] = i + 1 < N ? hi[i + 1] : 0u;
                lo[i] = WIDE && i + 1 < N ? lo[i + 1] : 0u;
                id[i] = i + 1 < N ? id[i + 1] : 0;
            }
        }
    }
    if (!sums)
        return false;
    const uint32_t next = (uint32_t)__shfl_down(top_of, 1);  // (by itself: every lane has to take part)
    const uint32_t below = lane == n - 1 ? out : next;
    return __ballot(lane < n && below != 0 && near(from_order32((uint32_t)top_of), from_order32(below), off)) != 0;
}

}  // namespace

// SUMS: the choice, or the groups', goes by sums that f32 rounds (a bias, or more than
// one expert standing for a group).
template <class E, int N, bool SUMS>
__global__ __launch_bounds__(kThreads) void gate_choose(GateArgs a, Layout p)
{
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)workgroup() * kWaves + wave;
    if (t >= a.T)
        return;
    int32_t* const idx = a.idx + t * a.K;
    float* const w = a.w + t * a.K;
    if (a.mask && !a.mask[t]) {
        if (lane < a.K) {
            idx[lane] = -1;
            w[lane] = 0.f;
        }
        return;
    }
    const char* const row = a.logits + t * a.ld;
    const int group = lane >> p.shift, first = group * p.group_size;
    const int e0 = first + (lane & ((1 << p.shift) - 1)) * N;
    const int end = group < a.groups ? first + p.group_size : 0;
    float l[N], e[N], b[N];
    load_run<E, N>(row, e0, end, l);
#pragma unroll
    for (int i = 0; i < N; ++i)
        b[i] = 0.f;
    if (SUMS && a.bias) {
        load_run<F32, N>(reinterpret_cast<const char*>(a.bias), e0, end, b);
    }
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    float m = 0.f, z = 1.f;
    if (softmax)
        z = softmax_sum<false, N>(l, m, e);  // (z is off by the mean of |l - m| over its terms only)

    uint32_t hi[N], lo[N];
    bool close = false;
    float off = 0.f;
    if constexpr (SUMS) {
        // c in f32; what is not finite is left to 64 bits
        if (!softmax)
#pragma unroll
            for (int i = 0; i < N; ++i)
                e[i] = __builtin_amdgcn_rcpf(1.f + fast_exp(-l[i]));
        const float rz = softmax ? __builtin_amdgcn_rcpf(z) : 1.f;
        off = off_by(softmax, rz);
        float odd = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool on = l[i] != -INFINITY && b[i] != -INFINITY;
            const float c = __builtin_fmaf(e[i], rz, b[i]);
            odd += on ? c - c : 0.f;  // (0, or NaN of an infinity or a NaN)
            hi[i] = on ? order32(c) : 0u;
            lo[i] = 0;
        }
        close = __ballot(odd != 0.f) != 0;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            hi[i] = l[i] == -INFINITY ? 0u : order32(l[i]);
            lo[i] = 0;
        }
    }
    // without a bias the experts' order is the logits', once the groups are chosen
    const auto by_logits = [&] {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (hi[i] | lo[i]) {
                hi[i] = order32(l[i]);
                lo[i] = 0;
            }
    };
    int mine = -1;
    if (a.groups > 1 && !close)
        close = keep_groups<N, false>(a, p.shift, lane, SUMS, off, hi, lo);
    if (SUMS && !a.bias)
        by_logits();
    if (!close)
        close = pick<N, false>(a.K, lane, e0, SUMS && a.bias, off, hi, lo, mine);
    if (SUMS && close) {
        double c[N], zd = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            c[i] = exp(softmax ? (double)l[i] - (double)m : -(double)l[i]);
        if (softmax) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                zd += c[i];
            zd = wave_sum(zd);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const double s = softmax ? c[i] / zd : 1.0 / (1.0 + c[i]);
            const bool on = l[i] != -INFINITY && b[i] != -INFINITY;
            const uint64_t k = on ? order64(s + (double)b[i]) : 0;
            hi[i] = (uint32_t)(k >> 32);
            lo[i] = (uint32_t)k;
        }
        if (a.groups > 1)
            keep_groups<N, true>(a, p.shift, lane, false, 0.f, hi, lo);
        if (!a.bias)
            by_logits();
        pick<N, true>(a.K, lane, e0, false, 0.f, hi, lo, mine);
    }

    // lane j the weight of slot j
    float s = 0.f;
    if (mine >= 0) {
        const float v = E::load(row + (int64_t)mine * E::SIZE);
        s = softmax ? expf(v - m) * __builtin_amdgcn_rcpf(z) : sigmoid(v);
    }
    if (a.renorm)
        s *= __builtin_amdgcn_rcpf(slots_sum(s, a.K) + kTiny);
    if (lane < a.K) {
        idx[lane] = mine;
        w[lane] = mine >= 0 ? a.scale * s : 0.f;
    }
}

template <class E, int N>
__global__ __launch_bounds__(kThreads) void gate_grad(GateArgs a)
{
    __shared__ __attribute__((aligned(16))) float slot_table[kWaves * 64 * N];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)workgroup() * kWaves + wave;
    if (t >= a.T)
        return;
    char* const out = a.dlogits + t * a.dlogits_ld;
    const int e0 = lane * N;
    const char* const row = a.logits + t * a.ld;
    float l[N], given = 0.f;
    int mine = -1;
    if (lane < a.K) {
        mine = a.idx[t * a.K + lane];
        given = a.w[t * a.K + lane];
    }
    load_run<E, N>(row, e0, a.E, l);
    if (mine >= a.E)
        mine = -1;
    float d[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        d[i] = 0.f;
    const uint64_t slots = __ballot(mine >= 0);
    if (slots != 0) {
        const bool softmax = a.score == MOE_SCORE_SOFTMAX;
        float e[N], m = 0.f, z = 1.f, v = 0.f, g = 0.f;
        float* const table = slot_table + wave * (64 * N);
        // the slots' logits by way of LDS (a second, dependent load: 14.4 us for 13.5 at 32768
        // x 384 bf16; the row after its slots, too: 15.0)
#pragma unroll
        for (int i = 0; i < N; ++i)
            table[e0 + i] = l[i];
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        if (mine >= 0) {
            v = table[mine];
            g = a.scale * given;
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        if (softmax)
            z = softmax_sum<E::SIZE == 4, N>(l, m, e);  // (14.8 us for 14.2 at 32768 x 256 f32; 16 bits round more away)
        const float rz = __builtin_amdgcn_rcpf(z);
        const float p = mine < 0 ? 0.f : softmax ? expf(v - m) * rz : sigmoid(v);
        float dp = g, q = 0.f;
        if (softmax || a.renorm)
            q = slots_sum(g * p, a.K);
        if (a.renorm) {
            // (each factor 1 / D at once: g p and 1e-20 g p may be below what f32 holds)
            const float one = __builtin_amdgcn_rcpf(slots_sum(p, a.K) + kTiny), tiny = kTiny * one, share = p * one;
            dp = tiny * g;
            for (uint64_t left = slots; left; left &= left - 1) {
                const int i = __builtin_ctzll(left);
                dp = __builtin_fmaf(lane_of(share, i), g - lane_of(g, i), dp);
            }
            dp = dp * one;
            q = tiny * (q * one);
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            d[i] = softmax ? -q : 0.f;
        // the slots' dp to their experts' lanes by way of LDS, unless an expert is named twice
#pragma unroll
        for (int i = 0; i < N; ++i)
            table[e0 + i] = 0.f;
        const int named = lane + 1;
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        if (mine >= 0)
            table[mine] = __int_as_float(named);
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        const bool twice = mine >= 0 && __float_as_int(table[mine]) != named;
        if (__ballot(twice) == 0) {
            if (mine >= 0)
                table[mine] = dp;
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
#pragma unroll
            for (int i = 0; i < N; ++i)
                d[i] += table[e0 + i];
        } else {
            for (uint64_t left = slots; left; left &= left - 1) {
                const int j = __builtin_ctzll(left);
                const int at = (int)lane_of((uint32_t)mine, j) - e0;
                const float add = lane_of(dp, j);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    d[i] += at == i ? add : 0.f;
            }
        }
        if (softmax) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                d[i] *= e[i] * rz;
        } else {  // s (1 - s) without 1 - s, which loses the small ones
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float x = expf(-fabsf(l[i])), r = __builtin_amdgcn_rcpf(1.f + x);
                d[i] *= x * r * r;
            }
        }
    }
    store_run<E, N>(out, e0, a.E, d);
}

// ------------------------------------------------------------ launchers

namespace {

template <class E, int N>
hipError_t launch(const GateArgs& a, const Layout* p, hipStream_t s)
{
    const dim3 grid = grid_of(((int64_t)a.T + kWaves - 1) / kWaves), block(kThreads);
    if (!p) {
        if constexpr (N <= 16) {  // (1024 experts over the wave)
            hipLaunchKernelGGL((gate_grad<E, N>), grid, block, 0, s, a);
            return hipGetLastError();
        }
        return hipErrorInvalidValue;
    }
    const bool sums = a.bias || (a.groups > 1 && a.group_top > 1);
    const auto kernel = sums ? gate_choose<E, N, true> : gate_choose<E, N, false>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, *p);
    return hipGetLastError();
}

// n: experts a lane takes; p: the choice's layout, null for the gradient.
template <class E>
hipError_t launch_run(const GateArgs& a, int n, const Layout* p, hipStream_t s)
{
    if (n <= 1)
        return launch<E, 1>(a, p, s);
    if (n <= 2)
        return launch<E, 2>(a, p, s);
    if (n <= 4)
        return launch<E, 4>(a, p, s);
    if (n <= 6)
        return launch<E, 6>(a, p, s);
    if (n <= 8)
        return launch<E, 8>(a, p, s);
    if (n <= 16)
        return launch<E, 16>(a, p, s);
    // (many experts in a number of groups that leaves lanes without any: at most 31 of them)
    return launch<E, 32>(a, p, s);
}

hipError_t launch_type(const GateArgs& a, int n, const Layout* p, hipStream_t s)
{
    switch (a.dtype) {
    case MOE_DTYPE_BF16: return launch_run<Bf16>(a, n, p, s);
    case MOE_DTYPE_F16: return launch_run<F16>(a, n, p, s);
    case MOE_DTYPE_F32: return launch_run<F32>(a, n, p, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_gate(const GateArgs& a, hipStream_t s)
{
    Layout p{6, a.E / a.groups};
    while (a.groups << p.shift > 64)
        --p.shift;
    return launch_type(a, (p.group_size + (1 << p.shift) - 1) >> p.shift, &p, s);
}

hipError_t launch_gate_bwd(const GateArgs& a, hipStream_t s) { return launch_type(a, (a.E + 63) / 64, nullptr, s); }

}  // namespace moe
