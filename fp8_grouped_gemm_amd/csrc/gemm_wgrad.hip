// Weight gradients of the experts from rows kept in 8 bits (include/moe_ops.h:
// moe_gemm_wgrad):
//   dw[e, i, k] = sum over the rows r of expert e of dy[r, i] x[r, k],  x = code * scale
//
// A product whose contraction runs over the rows, so that both operands lie the
// wrong way round in memory for the matrix instruction (v_mfma_f32_32x32x16, whose
// lanes take 8 adjacent r of one column).  A stage of kStage rows is brought into
// LDS as it lies, dy's columns and x's side by side, x decoded to dy's type on the
// way; the transposing LDS read (ds_read_b64_tr_b16: 16 lanes read four rows of 16
// columns and get four rows of one column each) turns it.  Its half wave reads four
// rows of 64 bytes, whose 64-byte slots are exchanged by the row (slot ^ row), so
// that they lie in different banks.
//
// The stages are double-buffered: a stage's loads are under way in registers while
// the one before is multiplied.  Rows past the segment and columns past the
// matrix enter as zeros.  Where few tiles and many rows leave compute units idle, the
// rows are split over workgroups whose f32 sums meet in the workspace and are added in
// a fixed order by a second kernel.
#include "../../include/moe_ops.h"
#include "ops_internal.h"
#include "rows_device.h"

namespace moe {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kStage = 32;      // rows of a stage
constexpr int kMostSplit = 16;

struct Frag {
    v4s lo, hi;
};

__device__ __forceinline__ v16f mfma(Bf16, const Frag& a, const Frag& b, const v16f& c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

__device__ __forceinline__ v16f mfma(F16, const Frag& a, const Frag& b, const v16f& c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Byte of element (row, col) of a stage's matrix of COLS 16-bit columns.
template <int COLS>
__device__ __forceinline__ int lds_at(int row, int col)
{
    constexpr int kSlots = COLS / 32 < 8 ? COLS / 32 : 8;
    return row * COLS * 2 + ((col * 2) ^ ((row & (kSlots - 1)) << 6));
}

// The 8 rows of column c0 + lane % 32 that the lane gives the matrix instruction:
// r0 + 4 (lane / 32) .. + 3 and the same 8 rows on (the same set for both operands,
// whose order the sum does not know).
template <int COLS>
__device__ __forceinline__ Frag read_frag(char* lds, int r0, int c0, int lane)
{
    const int row = r0 + 4 * (lane >> 5) + ((lane & 15) >> 2);
    const int col = c0 + (lane & 16) + 4 * (lane & 3);
    Frag f;
    f.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(lds + lds_at<COLS>(row, col)));
    f.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(lds + lds_at<COLS>(row + 8, col)));
    return f;
}

// 16 codes times their scale, rounded to E: two pieces of eight values.
template <class E>
__device__ __forceinline__ void decode16(rows_u32x4 q, float scale, rows_u32x4* out)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    float f[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], true);
        f[4 * i] = a[0] * scale;
        f[4 * i + 1] = a[1] * scale;
        f[4 * i + 2] = b[0] * scale;
        f[4 * i + 3] = b[1] * scale;
    }
    out[0] = E::pack(f);
    out[1] = E::pack(f + 8);
}

// First row and number of rows of a group's share `s` of S (whole stages but the last).
__device__ __forceinline__ void share(const WgradArgs& a, int e, int s, int64_t& first, int& rows)
{
    int64_t lo = 0, hi = a.R;
    if (a.offsets) {
        lo = max(a.offsets[e], 0);
        hi = a.counts ? lo + max(a.counts[e], 0) : (int64_t)a.offsets[e + 1];
        hi = min(hi, (int64_t)a.R);
    }
    const int64_t all = max(hi - lo, INT64_C(0));
    const int64_t per = ((all + a.split - 1) / a.split + kStage - 1) / kStage * kStage;
    const int64_t at = min(per * s, all);
    first = lo + at;
    rows = (int)min(per, all - at);
}

// One value to dw (type OUT), added to what is there with `add`.
template <class OUT>
__device__ __forceinline__ void put(char* p, float v, bool add)
{
    if (add)
        v += OUT::load(p);
    OUT::store(p, v);
}

}  // namespace

// A workgroup computes BM rows (dy's columns) by BN columns (x's) of one expert's dw
// over one share of its rows; its waves WM by WN each.
template <class E, bool MX, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void wgrad_tile(WgradArgs a, int tiles_m, int tiles_n)
{
    constexpr int kThreads = (BM / WM) * (BN / WN) * 64;
    constexpr int kBytes = kStage * (BM + BN) * 2;  // of a stage in LDS
    constexpr int kDy = kStage * BM / 8 / kThreads, kX = kStage * BN / 16 / kThreads;  // pieces a thread loads
    static_assert(kDy >= 1 && kX >= 1 && kStage * BN / 16 % kThreads == 0, "whole pieces");
    __shared__ __attribute__((aligned(16))) char lds[2][kBytes];

    unsigned wg = workgroup();
    const unsigned tiles = tiles_m * tiles_n;
    const unsigned unit = wg / tiles;  // share of an expert
    if (unit >= (unsigned)(a.E * a.split))
        return;
    wg -= unit * tiles;
    const int e = unit / a.split, s = unit - e * a.split;
    const int m0 = (int)(wg / tiles_n) * BM, n0 = (int)(wg % tiles_n) * BN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / (BN / WN) * WM, wn = wave % (BN / WN) * WN;

    int64_t first;
    int rows;
    share(a, e, s, first, rows);
    const int stages = (rows + kStage - 1) / kStage;
    const char* const dy = a.dy + first * a.dy_ld;
    const uint8_t* const x = a.x + first * a.K;
    const char* const sf = a.x_sf + first * (MX ? a.K / 32 : a.K / 128 * 4);

    rows_u32x4 dreg[kDy], xreg[kX];
    float xs[kX];
    const auto load = [&](int stage) {
        const int r0 = stage * kStage;
#pragma unroll
        for (int p = 0; p < kDy; ++p) {
            const int piece = p * kThreads + threadIdx.x;
            const int r = r0 + piece / (BM / 8), c = m0 + piece % (BM / 8) * 8;
            dreg[p] = {0, 0, 0, 0};
            if (r < rows && c < a.N) {
                const char* const at = dy + (int64_t)r * a.dy_ld + (int64_t)c * 2;
                if (c + 8 <= a.N) {
                    dreg[p] = load16(at);
                } else {
                    uint16_t v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = c + i < a.N ? reinterpret_cast<const uint16_t*>(at)[i] : 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dreg[p][i] = v[2 * i] | (uint32_t)v[2 * i + 1] << 16;
                }
            }
        }
#pragma unroll
        for (int p = 0; p < kX; ++p) {
            const int piece = p * kThreads + threadIdx.x;
            const int r = r0 + piece / (BN / 16), c = n0 + piece % (BN / 16) * 16;
            xreg[p] = {0, 0, 0, 0};
            xs[p] = 0.f;
            if (r < rows && c < a.K) {
                xreg[p] = *reinterpret_cast<const rows_u32x4*>(x + (int64_t)r * a.K + c);
                if constexpr (MX) {
                    const uint32_t b = (uint8_t)sf[(int64_t)r * (a.K / 32) + c / 32];
                    xs[p] = __uint_as_float(b == 0 ? 0x400000u : b == 0xFFu ? 0x7FC00000u : b << 23);
                } else {
                    xs[p] = reinterpret_cast<const float*>(sf)[(int64_t)r * (a.K / 128) + c / 128];
                }
            }
        }
    };
    const auto store = [&](char* to) {
#pragma unroll
        for (int p = 0; p < kDy; ++p) {
            const int piece = p * kThreads + threadIdx.x;
            *reinterpret_cast<rows_u32x4*>(to + lds_at<BM>(piece / (BM / 8), piece % (BM / 8) * 8)) = dreg[p];
        }
        char* const xt = to + kStage * BM * 2;
#pragma unroll
        for (int p = 0; p < kX; ++p) {
            const int piece = p * kThreads + threadIdx.x;
            const int r = piece / (BN / 16), c = piece % (BN / 16) * 16;
            rows_u32x4 v[2];
            decode16<E>(xreg[p], xs[p], v);
            *reinterpret_cast<rows_u32x4*>(xt + lds_at<BN>(r, c)) = v[0];
            *reinterpret_cast<rows_u32x4*>(xt + lds_at<BN>(r, c + 8)) = v[1];
        }
    };

    v16f acc[WM / 32][WN / 32];
#pragma unroll
    for (int i = 0; i < WM / 32; ++i)
#pragma unroll
        for (int j = 0; j < WN / 32; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k)
                acc[i][j][k] = 0.f;

    if (stages > 0) {
        load(0);
        store(lds[0]);
    }
    __syncthreads();
    for (int t = 0; t < stages; ++t) {
        if (t + 1 < stages)
            load(t + 1);
        char* const dt = lds[t & 1];
        char* const xt = dt + kStage * BM * 2;
#pragma unroll
        for (int r = 0; r < kStage; r += 16) {
            Frag fa[WM / 32], fb[WN / 32];
#pragma unroll
            for (int i = 0; i < WM / 32; ++i)
                fa[i] = read_frag<BM>(dt, r, wm + i * 32, lane);
#pragma unroll
            for (int j = 0; j < WN / 32; ++j)
                fb[j] = read_frag<BN>(xt, r, wn + j * 32, lane);
#pragma unroll
            for (int i = 0; i < WM / 32; ++i)
#pragma unroll
                for (int j = 0; j < WN / 32; ++j)
                    acc[i][j] = mfma(E{}, fa[i], fb[j], acc[i][j]);
        }
        if (t + 1 < stages)
            store(lds[(t + 1) & 1]);
        __syncthreads();
    }

    if (a.split == 1 && a.accumulate && rows == 0)
        return;
    // lane l holds column l % 32 and rows 8 (k / 4) + 4 (l / 32) + k % 4 of a block
    const int64_t plane = (int64_t)a.N * a.K;
    float* const part = a.split > 1 ? a.partial + ((int64_t)s * a.E + e) * plane : nullptr;
    char* const dw = a.dw + e * plane * (a.dw_dtype == MOE_DTYPE_F32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < WM / 32; ++i)
#pragma unroll
        for (int j = 0; j < WN / 32; ++j) {
            const int col = n0 + wn + j * 32 + (lane & 31);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int row = m0 + wm + i * 32 + 8 * (k / 4) + 4 * (lane >> 5) + k % 4;
                if (row >= a.N || col >= a.K)
                    continue;
                const int64_t at = (int64_t)row * a.K + col;
                const float v = acc[i][j][k];
                if (part)
                    part[at] = v;
                else if (a.dw_dtype == MOE_DTYPE_F32)
                    put<F32>(dw + at * 4, v, a.accumulate);
                else if (a.dw_dtype == MOE_DTYPE_BF16)
                    put<Bf16>(dw + at * 2, v, a.accumulate);
                else
                    put<F16>(dw + at * 2, v, a.accumulate);
            }
        }
}

// dw = the shares' sums, added in ascending order, four columns a thread.
template <class OUT>
__global__ __launch_bounds__(256) void wgrad_join(WgradArgs a)
{
    const int64_t n = (int64_t)a.E * a.N * a.K, at = ((int64_t)workgroup() * 256 + threadIdx.x) * 4;
    if (at >= n)
        return;
    if (a.accumulate) {
        int64_t first;
        int rows;
        share(a, (int)(at / ((int64_t)a.N * a.K)), 0, first, rows);
        if (rows == 0)
            return;
    }
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < a.split; ++s) {
        float p[4];
        F32::unpack(load16(reinterpret_cast<const char*>(a.partial + s * n + at)), p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] += p[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        put<OUT>(a.dw + (at + i) * OUT::SIZE, v[i], a.accumulate);
}

// ------------------------------------------------------------ launchers

namespace {

int64_t tiles_of(int n, int k) { return (int64_t)((n + 127) / 128) * ((k + 127) / 128); }

template <class E, bool MX>
hipError_t launch(const WgradArgs& a, hipStream_t s)
{
    constexpr int BM = 128, BN = 128;
    const int tm = (a.N + BM - 1) / BM, tn = (a.K + BN - 1) / BN;
    const int64_t wgs = (int64_t)a.E * a.split * tm * tn;
    if (wgs >= (INT64_C(1) << 31))
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((wgrad_tile<E, MX, BM, BN, 64, 64>), grid_of(wgs), dim3(256), 0, s, a, tm, tn);
    return hipGetLastError();
}

}  // namespace

int wgrad_split(int groups, int rows, int n, int k)
{
    const int64_t tiles = groups * tiles_of(n, k);
    int split = 1;
    while (split < kMostSplit && tiles * split < 256 && (int64_t)rows / groups >= (int64_t)split * 2 * 256)
        split *= 2;
    return split;
}

hipError_t launch_gemm_wgrad(const WgradArgs& a, hipStream_t s)
{
    const bool mx = a.sf_format == MOE_SF_UE8M0_32;
    hipError_t e;
    if (a.dtype == MOE_DTYPE_BF16)
        e = mx ? launch<Bf16, true>(a, s) : launch<Bf16, false>(a, s);
    else
        e = mx ? launch<F16, true>(a, s) : launch<F16, false>(a, s);
    if (e != hipSuccess || a.split == 1)
        return e;
    const int64_t n = (int64_t)a.E * a.N * a.K;
    const auto kernel = a.dw_dtype == MOE_DTYPE_F32    ? wgrad_join<F32>
                        : a.dw_dtype == MOE_DTYPE_BF16 ? wgrad_join<Bf16> : wgrad_join<F16>;
    hipLaunchKernelGGL(kernel, grid_of((n / 4 + 255) / 256), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
