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

constexpr int kMostSplit = 16;
constexpr int kStrip = 8;
constexpr int kShareRows = 64;  // shares are whole multiples of it

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

// A buffer of `bytes` bytes, past whose end loads give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, unsigned bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
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
    const int64_t per = ((all + a.split - 1) / a.split + kShareRows - 1) / kShareRows * kShareRows;
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

// The neighbour lane's value.
__device__ __forceinline__ uint32_t neighbour(uint32_t v) { return row_perm_u<0xB1>(v); }

// A wave's blocks of dw: lane l holds column l % 32 and rows 8 (k / 4) + 4 (l / 32) + k % 4
// of each.  16-bit types: neighbouring lanes first exchange one of two rows' values, so
// that each has two adjacent columns of one row, then of two blocks' one, so that a store
// writes whole lines of 128 bytes, as one of f32 does (64-byte runs: 2.6 TB/s for 5.4).
template <class OUT, int MB, int NB>
__device__ __forceinline__ void put_blocks(char* dw, const v16f (&acc)[MB][NB], int row0, int col0, int N, int K,
                                           int lane, bool add)
{
    const bool odd = lane & 1;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
            const int row = row0 + i * 32 + 8 * (k / 4) + 4 * (lane >> 5) + k % 4;
#pragma unroll
            for (int j = 0; j < NB; j += 2) {
                if constexpr (OUT::SIZE == 4) {
                    const int col = col0 + j * 32 + (lane & 31);
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        if (row + h / 2 < N && col + h % 2 * 32 < K)
                            put<OUT>(dw + ((int64_t)(row + h / 2) * K + col + h % 2 * 32) * 4, acc[i][j + h % 2][k + h / 2], add);
                } else {
                    // the lane's columns: two of block j (even lanes) or j + 1, of row and row + 1
                    const int col = col0 + (j + odd) * 32 + (lane & 30);
                    float v[2][2];  // [block][row], columns col % 32 and the next
                    uint32_t two[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float lo = acc[i][j + b][k], hi = acc[i][j + b][k + 1];
                        const float got = row_perm<0xB1>(odd ? lo : hi);
                        v[b][0] = odd ? got : lo;
                        v[b][1] = odd ? hi : got;
                    }
                    if (add) {  // block b of the lane's row is at its own place now
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const int r = row + odd, c = col0 + (j + b) * 32 + (lane & 30);
                            if (r < N && c < K) {
                                const char* const at = dw + ((int64_t)r * K + c) * 2;
                                v[b][0] += OUT::load(at);
                                v[b][1] += OUT::load(at + 2);
                            }
                        }
                    }
                    two[0] = OUT::pack2(v[0][0], v[0][1]);
                    two[1] = OUT::pack2(v[1][0], v[1][1]);
                    const uint32_t got = neighbour(odd ? two[0] : two[1]);
                    const uint32_t at_row = odd ? got : two[0], at_next = odd ? two[1] : got;
                    typedef unsigned int bytes4 __attribute__((aligned(1)));
                    char* const at = dw + ((int64_t)row * K + col) * 2;
                    if (row < N && col < K)
                        *reinterpret_cast<bytes4*>(at) = at_row;
                    if (row + 1 < N && col < K)
                        *reinterpret_cast<bytes4*>(at + (int64_t)K * 2) = at_next;
                }
            }
        }
}

}  // namespace

// A workgroup computes BM rows (dy's columns) by BN columns (x's) of one expert's dw
// over one share of its rows; its waves WM by WN each.
template <class E, bool MX, int BM, int BN, int WM, int WN, int kStage>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, 2) void wgrad_tile(WgradArgs a, int tiles_m, int tiles_n)
{
    constexpr int kThreads = (BM / WM) * (BN / WN) * 64;
    constexpr int kBytes = kStage * (BM + BN) * 2;  // of a stage in LDS
    constexpr int kDy = kStage * BM / 8 / kThreads, kX = kStage * BN / 16 / kThreads;  // pieces a thread loads
    static_assert(kDy >= 1 && kX >= 1 && kStage * BN / 16 % kThreads == 0, "whole pieces");
    __shared__ __attribute__((aligned(16))) char lds[2][kBytes];

    // Workgroups go to the 8 dies in turn: each die takes a run of a unit's (a share of an
    // expert's) tiles, counted down strips of kStrip rows, so that it reads a compact block.
    const unsigned wg = workgroup(), tiles = tiles_m * tiles_n, run = (tiles + 7) / 8;
    const unsigned unit = wg / (run * 8), in = wg - unit * run * 8;
    const unsigned tile = (in & 7) * run + in / 8;
    if (unit >= (unsigned)(a.E * a.split) || tile >= tiles)
        return;
    const int e = unit / a.split, s = unit - e * a.split;
    const int strip = tile / (kStrip * tiles_n), left = tile - strip * kStrip * tiles_n;
    const int high = min(kStrip, tiles_m - strip * kStrip);
    const int m0 = (strip * kStrip + left % high) * BM, n0 = left / high * BN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / (BN / WN) * WM, wn = wave % (BN / WN) * WN;

    int64_t first;
    int rows;
    share(a, e, s, first, rows);
    const int stages = (rows + kStage - 1) / kStage;
    const char* const dy = a.dy + first * a.dy_ld;
    const uint8_t* const x = a.x + first * a.K;
    const char* const sf = a.x_sf + first * (MX ? a.K / 32 : a.K / 128 * 4);

    // The thread's pieces: offsets from a stage's first row, kOut for columns past the
    // matrix.  A buffer ends with the share's last row, so that rows past it (and kOut) read as
    // zeros; only a piece that holds a row's last columns and more is loaded one by one.
    constexpr unsigned kOut = 0x80000000u;
    unsigned d_at[kDy], x_at[kX], sf_at[kX];
    int ragged = 0;  // columns of such a piece (the thread's pieces lie in the same columns)
    const int sf_row = MX ? a.K / 32 : a.K / 128 * 4;
    static_assert(kThreads % (BM / 8) == 0, "a thread's pieces lie in the same columns");
#pragma unroll
    for (int p = 0; p < kDy; ++p) {
        const int piece = p * kThreads + threadIdx.x, c = m0 + piece % (BM / 8) * 8;
        d_at[p] = c < a.N ? piece / (BM / 8) * (unsigned)a.dy_ld + c * 2u : kOut;
        ragged = c < a.N && c + 8 > a.N ? a.N - c : 0;
    }
#pragma unroll
    for (int p = 0; p < kX; ++p) {
        const int piece = p * kThreads + threadIdx.x, r = piece / (BN / 16), c = n0 + piece % (BN / 16) * 16;
        x_at[p] = c < a.K ? r * (unsigned)a.K + c : kOut;
        sf_at[p] = c < a.K ? r * (unsigned)sf_row + (MX ? c / 32 : c / 128 * 4) : kOut;
    }
    const bool odd_edge = a.N % 8 != 0 && m0 + BM > a.N;
    const auto bytes_left = [&](int r0, int64_t ld, int64_t width) {
        const int64_t n = (rows - r0 - 1) * ld + width;
        return (unsigned)min(n, INT64_C(0x7FFFFFFF));
    };

    rows_u32x4 dreg[kDy], xreg[kX];
    uint32_t xs[kX];
    const auto load = [&](int stage) {
        const int r0 = stage * kStage;
        const auto db = buffer(dy + r0 * a.dy_ld, bytes_left(r0, a.dy_ld, a.N * 2));
        const auto xb = buffer(x + (int64_t)r0 * a.K, bytes_left(r0, a.K, a.K));
        const auto sb = buffer(sf + (int64_t)r0 * sf_row, bytes_left(r0, sf_row, sf_row));
        if (odd_edge && ragged) {
#pragma unroll
            for (int p = 0; p < kDy; ++p) {
                const int r = r0 + (p * kThreads + (int)threadIdx.x) / (BM / 8);
                uint16_t v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = i < ragged && r < rows
                               ? reinterpret_cast<const uint16_t*>(dy + r0 * a.dy_ld + d_at[p])[i] : 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dreg[p][i] = v[2 * i] | (uint32_t)v[2 * i + 1] << 16;
            }
        } else {
#pragma unroll
            for (int p = 0; p < kDy; ++p)
                dreg[p] = __builtin_bit_cast(rows_u32x4, __builtin_amdgcn_raw_buffer_load_b128(db, d_at[p], 0, 0));
        }
#pragma unroll
        for (int p = 0; p < kX; ++p) {
            xreg[p] = __builtin_bit_cast(rows_u32x4, __builtin_amdgcn_raw_buffer_load_b128(xb, x_at[p], 0, 0));
            if constexpr (MX)
                xs[p] = __builtin_amdgcn_raw_buffer_load_b8(sb, sf_at[p], 0, 0);
            else
                xs[p] = __builtin_amdgcn_raw_buffer_load_b32(sb, sf_at[p], 0, 0);
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
            // code 0 is the subnormal 2^-127, 0xFF NaN
            const uint32_t b = xs[p];
            const uint32_t scale = !MX ? b : b == 0 ? 0x400000u : b == 0xFFu ? 0x7FC00000u : b << 23;
            decode16<E>(xreg[p], __uint_as_float(scale), v);
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
    const int64_t plane = (int64_t)a.N * a.K;
    char* const dw = a.dw + e * plane * (a.dw_dtype == MOE_DTYPE_F32 ? 4 : 2);
    if (a.split > 1)
        put_blocks<F32>(reinterpret_cast<char*>(a.partial + ((int64_t)s * a.E + e) * plane), acc, m0 + wm, n0 + wn, a.N,
                        a.K, lane, false);
    else if (a.dw_dtype == MOE_DTYPE_F32)
        put_blocks<F32>(dw, acc, m0 + wm, n0 + wn, a.N, a.K, lane, a.accumulate);
    else if (a.dw_dtype == MOE_DTYPE_BF16)
        put_blocks<Bf16>(dw, acc, m0 + wm, n0 + wn, a.N, a.K, lane, a.accumulate);
    else
        put_blocks<F16>(dw, acc, m0 + wm, n0 + wn, a.N, a.K, lane, a.accumulate);
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
#ifndef CFG
#define CFG 128, 128, 64, 64, 32
#endif
    constexpr int cfg[] = {CFG};
    constexpr int BM = cfg[0], BN = cfg[1], TH = cfg[0]/cfg[2]*cfg[1]/cfg[3]*64;
    const int tm = (a.N + BM - 1) / BM, tn = (a.K + BN - 1) / BN;
    const int64_t wgs = (int64_t)a.E * a.split * (((int64_t)tm * tn + 7) / 8 * 8);
    if (wgs >= (INT64_C(1) << 31))
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((wgrad_tile<E, MX, CFG>), grid_of(wgs), dim3(TH), 0, s, a, tm, tn);
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
