// Token rows into expert order and back (include/moe_ops.h: moe_permute,
// moe_permute_bwd, moe_unpermute, moe_unpermute_bwd), over the lists of the
// routing planner: src_row[f] the pool row of slot f = t*K + j, row_src[r] the
// slot of pool row r.
//   permute        xp[src_row[f]] = x[f / K]
//   its gradient   dx[t] = sum_j dxp[src_row[tK + j]]
//   unpermute      y[t] = sum_j w[tK + j] yp[src_row[tK + j]]
//   its gradients  dyp[src_row[f]] = w[f] dy[f / K],  dw[f] = dy[f / K] . yp[src_row[f]]
//
// All four move bytes and compute next to nothing, so HBM bounds them (4.9 to
// 6.0 TB/s at 8192 x 6 x 7168 and 4096 x 8 x 4096; a large copy reaches 5.2).  They
// walk the token side, not the pool: a token's row is read once (or its
// sums stay in registers) and its K pool rows are written or read whole,
// where walking the pool would read every token row K times.  Nothing is
// summed by atomics: a token's sum runs over its slots in ascending j.
//
// Every list entry is range-checked before it forms an address.
#include "../../include/moe_ops.h"
#include "ops_internal.h"
#include "rows_device.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kPadRows = 4;  // pool rows each wave looks over for padding

// Zeros the padding rows (row_src outside [0, TK)) among pool rows
// [r0, r0 + kPadRows) below `used`, by one wave.
template <bool NT>
__device__ __forceinline__ void clear_padding(const RowsArgs& a, int r0, int row_bytes, int lane)
{
    const int used = a.used ? min(*a.used, a.R) : a.R;
    const int end = min(r0 + kPadRows, used);
    const rows_u32x4 zero = {0, 0, 0, 0};
    for (int r = r0; r < end; ++r) {
        const int f = a.row_src[r];
        if (f >= 0 && f < a.T * a.K)
            continue;
        char* p = a.pool_out + (int64_t)r * a.pool_out_ld;
        int at = lane * 16;
        for (; at + 16 <= row_bytes; at += 64 * 16)
            store16<NT>(p + at, zero);
        for (; at < row_bytes; ++at)  // the one lane (if any) holding the ragged end
            p[at] = 0;
    }
}

// Whether a call's pool rows stream past the caches (nontemporal accesses):
// whole aligned 16-byte pieces, and more of them than the eight L2s hold
// twice over.  Measured cached and streamed, us, other inputs in every call:
// permute 8192 x 6 x 7168 bf16 174 and 173 (146 where the last-level cache still holds
// the token rows; 260 and 259, 229, with the padding of 128-row segments), its
// gradient 4096 x 8 x 4096 f32 119 and 99, unpermute 8192 x 6 x 7168 172 and 160, its
// gradient 4096 x 8 x 4096 128 and 123; rows of 4097 bf16 (unaligned) 52 and 57.
// Around the limit, top-8 of 4096 bf16:
//   pool   permute    gradient   unpermute's   permute +    permute +
//                                gradient      unpermute    quantise
//    32 MB  9.0  8.4  12.8 12.5  19.5 18.4     18.4 19.7    18.4 18.5
//    64 MB 16.1 14.7  17.1 16.9  33.8 31.7     28.6 31.2    30.1 33.6
//   128 MB 30   27    32   31    79   68       60   57      53   62
//   192 MB 45   40    46   44    90   87       78   82      81   92
//   402 MB 94   81    97   87   184  178      210  165     174  187
// Streaming is the faster by itself, but the call that reads the pool next pays for it
// while the last-level cache could hold the pool; small pools, which are read
// soon, stay cached.  The token rows stay cached too: several workgroups
// read them (permute 145, 176 streamed, the same inputs in every call).
bool streams(const RowsArgs& a, const void* pool, int64_t pool_ld, int size)
{
    const int64_t row = (int64_t)a.width * size;
    const uintptr_t tok = reinterpret_cast<uintptr_t>(a.tok ? a.tok : a.tok_out);
    return (int64_t)a.T * a.K * row > (INT64_C(64) << 20) &&
           (row | pool_ld | a.tok_ld | (int64_t)reinterpret_cast<uintptr_t>(pool) | (int64_t)tok) % 16 == 0;
}

// Workgroups of one launch: token_wgs over tokens, then those that look for
// padding.
unsigned pad_wgs(const RowsArgs& a)
{
    const int per_wg = kPadRows * kThreads / 64;
    return a.row_src ? (unsigned)((a.R + per_wg - 1) / per_wg) : 0u;
}

// Threads along a row: the smallest power of two that covers its n vectors,
// 16 to 256 (narrow rows share a workgroup).
int row_threads(int64_t n)
{
    int t = 16;
    while (t < kThreads && t < n)
        t *= 2;
    return t;
}

}  // namespace

// x row -> its K pool rows, one 16-byte piece per thread.  A row's last piece
// reaches back to stay whole (it writes bytes the previous piece also
// writes, with the same values); rows under 16 bytes go byte by byte.
template <bool NT>
__global__ __launch_bounds__(kThreads) void permute_rows(RowsArgs a, int row_bytes, int tpr,
                                                         int pieces, unsigned token_wgs)
{
    const unsigned wg = workgroup();
    if (wg >= token_wgs) {
        const int wave = (wg - token_wgs) * (kThreads / 64) + (threadIdx.x >> 6);
        clear_padding<NT>(a, wave * kPadRows, row_bytes, threadIdx.x & 63);
        return;
    }
    const unsigned g = wg / pieces;
    const int t = g * (kThreads / tpr) + threadIdx.x / tpr;
    int at = ((wg - g * pieces) * tpr + threadIdx.x % tpr) * 16;
    if (t >= a.T || at >= row_bytes)
        return;
    const char* src = a.tok + (int64_t)t * a.tok_ld;
    const int32_t* slot = a.src_row + (int64_t)t * a.K;
    if (row_bytes < 16) {
        for (int j = 0; j < a.K; ++j) {
            const int r = slot[j];
            if (r >= 0 && r < a.R)
                for (int i = 0; i < row_bytes; ++i)
                    a.pool_out[(int64_t)r * a.pool_out_ld + i] = src[i];
        }
        return;
    }
    at = min(at, row_bytes - 16);
    const rows_u32x4 v = load16(src + at);
    for (int j = 0; j < a.K; ++j) {
        const int r = slot[j];
        if (r >= 0 && r < a.R)
            store16<NT>(a.pool_out + (int64_t)r * a.pool_out_ld + at, v);
    }
}

// out[t] = sum_j w[tK + j] pool[src_row[tK + j]], j ascending, one vector of the row
// per thread; four slots' loads are in flight at a time (eight: 213 us for 161 at
// 8192 x 6 x 7168, their registers halve the waves; two: 162).
template <class E, bool W, bool NT>
__global__ __launch_bounds__(kThreads) void token_sums(RowsArgs a, int tpr, int pieces)
{
    const unsigned wg = workgroup(), g = wg / pieces;
    const int t = g * (kThreads / tpr) + threadIdx.x / tpr;
    const int c = ((wg - g * pieces) * tpr + threadIdx.x % tpr) * E::VEC;
    if (t >= a.T || c >= a.width)
        return;
    const int n = a.width - c;
    const int32_t* slot = a.src_row + (int64_t)t * a.K;
    const float* w = W ? a.w + (int64_t)t * a.K : nullptr;
    float acc[E::VEC];
#pragma unroll
    for (int i = 0; i < E::VEC; ++i)
        acc[i] = 0.f;
    constexpr int U = 4;
    for (int j0 = 0; j0 < a.K; j0 += U) {
        float v[U][E::VEC], wt[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = j0 + u < a.K ? slot[j0 + u] : -1;
            on[u] = r >= 0 && r < a.R;
            wt[u] = 1.f;
            if (on[u]) {
                if (W)
                    wt[u] = w[j0 + u];
                load_vec<E, NT>(a.pool + (int64_t)r * a.pool_ld + (int64_t)c * E::SIZE, n, v[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (on[u])
#pragma unroll
                for (int i = 0; i < E::VEC; ++i)
                    acc[i] = W ? __builtin_fmaf(wt[u], v[u][i], acc[i]) : acc[i] + v[u][i];
    }
    store_vec<E, NT>(a.tok_out + (int64_t)t * a.tok_ld + (int64_t)c * E::SIZE, n, acc);
}

// dyp row and dw of one slot per wave: the lanes stride over the row, write
// w dy and sum dy yp, and the wave's 64 sums meet in a butterfly (a fixed
// order).  Consecutive waves take consecutive slots, so the K waves of a
// token read its dy row together.
template <class E, bool DYP, bool DW, bool NT>
__global__ __launch_bounds__(kThreads) void unpermute_grad(RowsArgs a, unsigned token_wgs)
{
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const unsigned wg = workgroup();
    if (wg >= token_wgs) {
        clear_padding<NT>(a, ((wg - token_wgs) * (kThreads / 64) + wave) * kPadRows,
                      a.width * E::SIZE, lane);
        return;
    }
    const int f = wg * (kThreads / 64) + wave;
    if (f >= a.T * a.K)
        return;
    const int r = a.src_row[f];
    if (r < 0 || r >= a.R) {
        if (DW && lane == 0)
            a.dw[f] = 0.f;
        return;
    }
    const char* dy = a.tok + (int64_t)(f / a.K) * a.tok_ld;
    const char* yp = DW ? a.pool + (int64_t)r * a.pool_ld : nullptr;
    char* dyp = DYP ? a.pool_out + (int64_t)r * a.pool_out_ld : nullptr;
    const float w = a.w ? a.w[f] : 1.f;
    float sum = 0.f;
#pragma unroll 2
    for (int c = lane * E::VEC; c < a.width; c += 64 * E::VEC) {
        const int n = a.width - c;
        float d[E::VEC], y[E::VEC];
        load_vec<E>(dy + (int64_t)c * E::SIZE, n, d);
        if (DW) {
            load_vec<E, NT>(yp + (int64_t)c * E::SIZE, n, y);
#pragma unroll
            for (int i = 0; i < E::VEC; ++i)
                sum = __builtin_fmaf(d[i], y[i], sum);
        }
        if (DYP) {
#pragma unroll
            for (int i = 0; i < E::VEC; ++i)
                d[i] *= w;
            store_vec<E, NT>(dyp + (int64_t)c * E::SIZE, n, d);
        }
    }
    if (DW) {
#pragma unroll
        for (int x = 32; x >= 1; x >>= 1)
            sum += __shfl_xor(sum, x);
        if (lane == 0)
            a.dw[f] = sum;
    }
}

// ------------------------------------------------------------ launchers

hipError_t launch_permute(const RowsArgs& a, hipStream_t s)
{
    const int size = a.dtype == MOE_DTYPE_F32 ? 4 : a.dtype == MOE_DTYPE_U8 ? 1 : 2;
    const int row_bytes = a.width * size;
    const int64_t n = (row_bytes + 15) / 16;
    const int tpr = row_threads(n), per = kThreads / tpr;
    const int pieces = (int)((n + tpr - 1) / tpr);
    const int64_t wgs = (int64_t)((a.T + per - 1) / per) * pieces;
    const unsigned pad = pad_wgs(a);
    if (wgs + pad >= (INT64_C(1) << 31))
        return hipErrorInvalidValue;
    if (wgs + pad == 0)
        return hipSuccess;
    const auto kernel = streams(a, a.pool_out, a.pool_out_ld, size) ? permute_rows<true> : permute_rows<false>;
    hipLaunchKernelGGL(kernel, grid_of(wgs + pad), dim3(kThreads), 0, s, a, row_bytes, tpr, pieces,
                       (unsigned)wgs);
    return hipGetLastError();
}

template <class E>
static hipError_t launch_token_sums(const RowsArgs& a, hipStream_t s)
{
    const int64_t n = (a.width + E::VEC - 1) / E::VEC;
    const int tpr = row_threads(n), per = kThreads / tpr;
    const int pieces = (int)((n + tpr - 1) / tpr);
    const int64_t wgs = (int64_t)((a.T + per - 1) / per) * pieces;
    if (wgs >= (INT64_C(1) << 31))
        return hipErrorInvalidValue;
    const bool nt = streams(a, a.pool, a.pool_ld, E::SIZE);
    const auto kernel = a.w ? (nt ? token_sums<E, true, true> : token_sums<E, true, false>)
                            : (nt ? token_sums<E, false, true> : token_sums<E, false, false>);
    hipLaunchKernelGGL(kernel, grid_of(wgs), dim3(kThreads), 0, s, a, tpr, pieces);
    return hipGetLastError();
}

hipError_t launch_unpermute(const RowsArgs& a, hipStream_t s)
{
    switch (a.dtype) {
    case MOE_DTYPE_BF16: return launch_token_sums<Bf16>(a, s);
    case MOE_DTYPE_F16: return launch_token_sums<F16>(a, s);
    case MOE_DTYPE_F32: return launch_token_sums<F32>(a, s);
    default: return hipErrorInvalidValue;
    }
}

template <class E>
static hipError_t launch_grad(const RowsArgs& a, hipStream_t s)
{
    const unsigned wgs = (unsigned)(((int64_t)a.T * a.K + kThreads / 64 - 1) / (kThreads / 64));
    const unsigned pad = a.pool_out ? pad_wgs(a) : 0u;
    const dim3 grid = grid_of((int64_t)wgs + pad), block(kThreads);
    if (wgs + pad == 0)
        return hipSuccess;
    bool nt = true;
    if (a.dw)
        nt = nt && streams(a, a.pool, a.pool_ld, E::SIZE);
    if (a.pool_out)
        nt = nt && streams(a, a.pool_out, a.pool_out_ld, E::SIZE);
    auto kernel = nt ? unpermute_grad<E, true, true, true> : unpermute_grad<E, true, true, false>;
    if (!a.dw)
        kernel = nt ? unpermute_grad<E, true, false, true> : unpermute_grad<E, true, false, false>;
    else if (!a.pool_out)
        kernel = nt ? unpermute_grad<E, false, true, true> : unpermute_grad<E, false, true, false>;
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, wgs);
    return hipGetLastError();
}

hipError_t launch_unpermute_bwd(const RowsArgs& a, hipStream_t s)
{
    switch (a.dtype) {
    case MOE_DTYPE_BF16: return launch_grad<Bf16>(a, s);
    case MOE_DTYPE_F16: return launch_grad<F16>(a, s);
    case MOE_DTYPE_F32: return launch_grad<F32>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace moe
