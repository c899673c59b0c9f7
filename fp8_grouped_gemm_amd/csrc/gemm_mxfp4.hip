// Product of two microscaled 4-bit matrices (include/moe_ops.h:
// moe_gemm_mxfp4), dense or over the row segments of experts:
//   y[r, n] = sum over 32-blocks b of 2^(ca[r,b] - 127 + cb[n,b] - 127)
//             sum over k in b of a[r, k] b[n, k]
// gfx950's block-scaled MFMA does the inner line for 64 (32x32x64) or 128
// (16x16x128) K values at a time, scales included, and accumulates in f32:
// products and sums of e2m1 values are exact in it up to the f32 rounding of
// the running sum (measured error at most 1.3e-7 of the sum of magnitudes
// per instruction, whatever the scales).
//
// Operand layout of both instructions (checked on the GPU against exact
// arithmetic): lane l holds 32 consecutive K values -- 16 bytes, one scale
// block -- of row l % 16 (l % 32), block l / 16 (l / 32) of the
// instruction's 4 (2), and that block's UE8M0 code in the byte of its scale
// register that the instruction selects.
#include <algorithm>
#include <type_traits>

#include "../../include/moe_ops.h"
#include "moe_lds.h"
#include "ops_internal.h"
#include "rows_device.h"

namespace moe {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

// The part of a segment one tile covers.
struct RowTile {
    int e, row0, rows;  // expert, first row, live rows; rows 0: no such tile
};

// Segment e, cut to the matrix: first row and row count.
__device__ __forceinline__ void segment(const MxGemmArgs& a, int e, int& first, int& n)
{
    first = a.offsets[e];
    n = a.counts ? a.counts[e] : a.offsets[e + 1] - first;
    if (first < 0 || first >= a.R)
        n = 0;
    n = max(0, min(n, a.R - first));
}

// Row tiles of BM rows over all segments, in expert order: how many there
// are, and (by find_tile) which one is number `want`.  A wave looks at 64
// experts at a time; every wave of a workgroup does so for itself.
template <int BM>
__device__ __forceinline__ int count_tiles(const MxGemmArgs& a, int lane)
{
    int total = 0;
    for (int e = lane; e < a.E; e += 64) {
        int first, n;
        segment(a, e, first, n);
        total += (n + BM - 1) / BM;
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        total += __shfl_xor(total, d);
    return __builtin_amdgcn_readfirstlane(total);
}

template <int BM>
__device__ __forceinline__ RowTile find_tile(const MxGemmArgs& a, int want, int lane)
{
    int before = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int e = e0 + lane;
        int first = 0, n = 0;
        if (e < a.E)
            segment(a, e, first, n);
        const int tiles = (n + BM - 1) / BM;
        int incl = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(incl, d);
            if (lane >= d)
                incl += v;
        }
        const uint64_t past = __ballot(before + incl > want);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int skip = (want - before - __shfl(incl - tiles, l)) * BM;
            RowTile t;
            t.e = e0 + l;
            t.row0 = __builtin_amdgcn_readfirstlane(__shfl(first, l) + skip);
            t.rows = __builtin_amdgcn_readfirstlane(min(BM, __shfl(n, l) - skip));
            return t;
        }
        before += __shfl(incl, 63);
    }
    return {0, 0, 0};
}

// Row tile and column tile of workgroup `wg`.  Workgroups go to the 8 XCDs
// round-robin, each XCD takes a contiguous share of the tiles, and tiles run
// in bands of up to 8 row tiles, column by column, so that the tiles an XCD
// works on at one time share rows of a and of b in its L2.
template <int BM>
__device__ __forceinline__ RowTile pick_tile(const MxGemmArgs& a, int col_tiles, int lane, int& ct)
{
    constexpr int kBand = 8;
    const int row_tiles = a.offsets ? count_tiles<BM>(a, lane) : (a.R + BM - 1) / BM;
    const int total = row_tiles * col_tiles;
    const int share = (total + 7) / 8;
    const int i = blockIdx.x / 8, at = (blockIdx.x % 8) * share + i;
    if (i >= share || at >= total)
        return {0, 0, 0};
    const int band = at / (kBand * col_tiles), in = at - band * kBand * col_tiles;
    const int tall = min(kBand, row_tiles - band * kBand);
    ct = in / tall;
    const int rt = band * kBand + in - ct * tall;
    if (a.offsets)
        return find_tile<BM>(a, rt, lane);
    return {0, rt * BM, min(BM, a.R - rt * BM)};
}

template <class T>
__device__ __forceinline__ void store_y(const MxGemmArgs& a, int row, int col, float v)
{
    T::store(a.y + (int64_t)row * a.y_ld + (int64_t)col * T::SIZE, v);
}

}  // namespace

// ---------------------------------------------------------------- few rows
//
// 16 MT rows x 16 NT columns per workgroup of WV waves that split K: wave w
// takes the 256-wide K steps w, w + WV, ... (so the workgroup reads WV * 128
// consecutive bytes of each weight row at a time), straight from memory into
// MFMA operands, and the waves' sums meet in LDS in wave order.  A step is
// two MFMAs per subtile pair: lane group g supplies K blocks 2g and 2g + 1
// of the step's 8, so its two 16-byte loads are adjacent and the four groups
// read one whole 128-byte line of each row.
template <int MT, int NT>
struct Step {
    uint4 a[MT][2], b[NT][2];
    int sa[MT], sb[NT];  // codes of the two blocks in bytes 0 and 1
};

template <class T, int MT, int NT, int WV>
__global__ __launch_bounds__(64 * WV) void mxfp4_rows(MxGemmArgs a, int col_tiles)
{
    constexpr int BM = 16 * MT, BN = 16 * NT;
    __shared__ float part[WV][BM][BN + 4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int ct = 0;
    const RowTile t = pick_tile<BM>(a, col_tiles, lane, ct);
    if (t.rows <= 0)
        return;
    const int lr = lane & 15, lg = lane >> 4;
    const int nb = a.K / 32;  // K blocks
    const int col0 = ct * BN;
    // Rows and columns past the tile's repeat its last one (never stored).
    const uint8_t *pa[MT], *pb[NT], *psa[MT], *psb[NT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int64_t r = t.row0 + min(16 * m + lr, t.rows - 1);
        pa[m] = a.a + r * (a.K / 2);
        psa[m] = a.a_sf + r * nb;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int64_t c = (int64_t)t.e * a.N + min(col0 + 16 * n + lr, a.N - 1);
        pb[n] = a.b + c * (a.K / 2);
        psb[n] = a.b_sf + c * nb;
    }
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto fetch = [&](Step<MT, NT>& s, int step) {
        const int blk = step * 8 + 2 * lg;
        if (step * 8 + 8 <= nb) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                s.b[n][0] = *reinterpret_cast<const uint4*>(pb[n] + blk * 16);
                s.b[n][1] = *reinterpret_cast<const uint4*>(pb[n] + blk * 16 + 16);
                s.sb[n] = psb[n][blk] | (psb[n][blk + 1] << 8);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                s.a[m][0] = *reinterpret_cast<const uint4*>(pa[m] + blk * 16);
                s.a[m][1] = *reinterpret_cast<const uint4*>(pa[m] + blk * 16 + 16);
                s.sa[m] = psa[m][blk] | (psa[m][blk + 1] << 8);
            }
        } else {  // the step K ends in: blocks past it are zeros with scale 1
            const bool in0 = blk < nb, in1 = blk + 1 < nb;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                s.b[n][0] = in0 ? *reinterpret_cast<const uint4*>(pb[n] + blk * 16) : zero;
                s.b[n][1] = in1 ? *reinterpret_cast<const uint4*>(pb[n] + blk * 16 + 16) : zero;
                s.sb[n] = (in0 ? psb[n][blk] : 127) | ((in1 ? psb[n][blk + 1] : 127) << 8);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                s.a[m][0] = in0 ? *reinterpret_cast<const uint4*>(pa[m] + blk * 16) : zero;
                s.a[m][1] = in1 ? *reinterpret_cast<const uint4*>(pa[m] + blk * 16 + 16) : zero;
                s.sa[m] = (in0 ? psa[m][blk] : 127) | ((in1 ? psa[m][blk + 1] : 127) << 8);
            }
        }
    };
    v4f acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
            acc[m][n] = v4f{0.f, 0.f, 0.f, 0.f};
    auto mul = [&](const Step<MT, NT>& s) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    e2m1_operand(s.a[m][0]), e2m1_operand(s.b[n][0]), acc[m][n], 4, 4, 0, s.sa[m], 0, s.sb[n]);
                acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    e2m1_operand(s.a[m][1]), e2m1_operand(s.b[n][1]), acc[m][n], 4, 4, 1, s.sa[m], 1, s.sb[n]);
            }
    };
    const int steps = (nb + 7) / 8;
    {
        Step<MT, NT> s0, s1;
        int i = wave;
        if (i < steps)
            fetch(s0, i);
        while (i < steps) {
            if (i + WV < steps)
                fetch(s1, i + WV);
            mul(s0);
            i += WV;
            if (i >= steps)
                break;
            if (i + WV < steps)
                fetch(s0, i + WV);
            mul(s1);
            i += WV;
        }
    }
    // lane l holds column l % 16, rows 4 (l / 16) + i of each subtile
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[wave][16 * m + 4 * lg + i][16 * n + lr] = acc[m][n][i];
    __syncthreads();
    for (int c = threadIdx.x; c < BM * BN; c += 64 * WV) {
        const int m = c / BN, n = c % BN;
        if (m >= t.rows || col0 + n >= a.N)
            continue;
        float v = part[0][m][n];
#pragma unroll
        for (int w = 1; w < WV; ++w)
            v += part[w][m][n];
        store_y<T>(a, t.row0 + m, col0 + n, v);
    }
}

// ---------------------------------------------------------------- tiles
//
// BM x BN tile per workgroup of WM x WN waves, each MI x NI subtiles of
// 32 x 32; K in stages of 256 (128 bytes of each row), staged in LDS by
// asynchronous copies into one of two buffers while the other is multiplied.
// One copy instruction of a wave brings 8 rows x 128 bytes -- whole lines
// from memory, 1 KiB in a row of LDS -- and a row's eight 16-byte chunks sit
// in LDS at position chunk ^ key(row), key = (row & 7) ^ (row >> 3 & 1): any 8
// (16) consecutive rows then hold a given chunk in different banks, so the
// fragment reads run without conflicts.  Scales pass through registers: each
// thread loads the 8 codes of a row one stage ahead and leaves them in LDS,
// and one byte permute of a row's 8 codes gives the MFMA's scale register
// for all four 64-wide K steps of the stage (lane group g takes the codes
// 2s + g).  Blocks past the end of K are copied from 16 zero bytes, scale 1.
__device__ __constant__ const uint4 kZeroBlock = {0, 0, 0, 0};

template <class T, int WM, int WN, int MI, int NI>
__global__ __launch_bounds__(64 * WM * WN) void mxfp4_tile(MxGemmArgs a, int col_tiles)
{
    constexpr int BM = WM * MI * 32, BN = WN * NI * 32;
    constexpr int W = WM * WN, TH = 64 * W;
    constexpr int ROWS = BM + BN;              // of both operands, a's first
    constexpr int STAGE = ROWS * 128;
    constexpr int COPIES = ROWS / 8 / W;       // per wave and stage
    constexpr int SCALES = (ROWS + TH - 1) / TH;
    static_assert(ROWS % (8 * W) == 0, "whole copies per wave");
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    uint8_t* const sc = smem + 2 * STAGE;      // [2][ROWS][8]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int ct = 0;
    const RowTile t = pick_tile<BM>(a, col_tiles, lane, ct);
    if (t.rows <= 0)
        return;
    const int col0 = ct * BN, cols = min(BN, a.N - col0);
    const int nb = a.K / 32, stages = (nb + 7) / 8;
    const uint8_t* const abase = a.a + (int64_t)t.row0 * (a.K / 2);
    const uint8_t* const bbase = a.b + ((int64_t)t.e * a.N + col0) * (a.K / 2);
    const uint8_t* const asf = a.a_sf + (int64_t)t.row0 * nb;
    const uint8_t* const bsf = a.b_sf + ((int64_t)t.e * a.N + col0) * nb;

    // Copies: instruction q of this wave brings LDS rows 8 (q W + wave) ..
    // + 7, lane l the chunk at position l % 8 of row l / 8.
    uint32_t off[COPIES];
#pragma unroll
    for (int q = 0; q < COPIES; ++q) {
        const int r8 = q * W + wave;
        const int row = 8 * r8 + (lane >> 3);
        const int key = ((lane >> 3) ^ (r8 & 1)) & 7;
        const int c = (lane & 7) ^ key;
        const int live = row < BM ? min(row, t.rows - 1) : min(row - BM, cols - 1);
        off[q] = (uint32_t)live * (uint32_t)(a.K / 2) + c * 16;
    }
    const uint32_t lds0 = lds_addr(smem);
    auto copy = [&](int stage, int buf) {
        const bool ragged = stage * 8 + 8 > nb;
#pragma unroll
        for (int q = 0; q < COPIES; ++q) {
            const int r8 = q * W + wave;
            const uint8_t* base = (8 * r8 < BM ? abase : bbase) + (int64_t)stage * 128;
            const uint32_t dst = lds0 + buf * STAGE + r8 * 1024;
            if (!ragged) {
                dma16_off(base, off[q], dst);
            } else {
                const int c = (lane & 7) ^ (((lane >> 3) ^ (r8 & 1)) & 7);
                const void* src = stage * 8 + c < nb ? (const void*)(base + off[q]) : (const void*)&kZeroBlock;
                dma16(src, dst);
            }
        }
    };
    // Scales: thread i takes row i (and i + TH ...) of the ROWS.
    uint2 codes[SCALES];
    auto fetch_scales = [&](int stage) {
#pragma unroll
        for (int q = 0; q < SCALES; ++q) {
            const int row = q * TH + threadIdx.x;
            codes[q] = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
            if (row >= ROWS)
                continue;
            const uint8_t* p = (row < BM ? asf + (int64_t)min(row, t.rows - 1) * nb
                                         : bsf + (int64_t)min(row - BM, cols - 1) * nb) + stage * 8;
            if (stage * 8 + 8 <= nb) {
                struct __attribute__((packed, aligned(1))) U2 { uint32_t x, y; };
                const U2 u = *reinterpret_cast<const U2*>(p);
                codes[q] = make_uint2(u.x, u.y);
            } else {
                uint32_t w[2] = {0x7F7F7F7Fu, 0x7F7F7F7Fu};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (stage * 8 + i < nb)
                        w[i / 4] = (w[i / 4] & ~(0xFFu << (8 * (i % 4)))) | ((uint32_t)p[i] << (8 * (i % 4)));
                codes[q] = make_uint2(w[0], w[1]);
            }
        }
    };
    auto leave_scales = [&](int buf) {
#pragma unroll
        for (int q = 0; q < SCALES; ++q) {
            const int row = q * TH + threadIdx.x;
            if (row < ROWS)
                *reinterpret_cast<uint2*>(sc + (buf * ROWS + row) * 8) = codes[q];
        }
    };

    const int wm = wave / WN, wn = wave % WN;
    const int lr = lane & 31, lg = lane >> 5;
    const int key = (lr & 7) ^ ((lr >> 3) & 1);
    const uint32_t pick = lg ? 0x07050301u : 0x06040200u;  // codes 1,3,5,7 or 0,2,4,6
    v16f acc[MI][NI];
#pragma unroll
    for (int m = 0; m < MI; ++m)
#pragma unroll
        for (int n = 0; n < NI; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[m][n][i] = 0.f;

    fetch_scales(0);
    copy(0, 0);
    leave_scales(0);
    MOE_WAIT_VMCNT(0);
    __syncthreads();
    for (int st = 0; st < stages; ++st) {
        const int buf = st & 1;
        if (st + 1 < stages) {
            fetch_scales(st + 1);
            copy(st + 1, buf ^ 1);
        }
        const uint8_t* const la = smem + buf * STAGE + (wm * MI * 32 + lr) * 128;
        const uint8_t* const lb = smem + buf * STAGE + (BM + wn * NI * 32 + lr) * 128;
        const uint8_t* const sa0 = sc + (buf * ROWS + wm * MI * 32 + lr) * 8;
        const uint8_t* const sb0 = sc + (buf * ROWS + BM + wn * NI * 32 + lr) * 8;
        int sa[MI], sb[NI];
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            const uint2 u = *reinterpret_cast<const uint2*>(sa0 + m * 256);
            sa[m] = (int)__builtin_amdgcn_perm(u.y, u.x, pick);
        }
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const uint2 u = *reinterpret_cast<const uint2*>(sb0 + n * 256);
            sb[n] = (int)__builtin_amdgcn_perm(u.y, u.x, pick);
        }
        auto step = [&](auto S) {
            constexpr int s = decltype(S)::value;
            const int at = ((2 * s + lg) ^ key) * 16;
            uint4 fa[MI], fb[NI];
#pragma unroll
            for (int m = 0; m < MI; ++m)
                fa[m] = *reinterpret_cast<const uint4*>(la + m * 4096 + at);
#pragma unroll
            for (int n = 0; n < NI; ++n)
                fb[n] = *reinterpret_cast<const uint4*>(lb + n * 4096 + at);
#pragma unroll
            for (int m = 0; m < MI; ++m)
#pragma unroll
                for (int n = 0; n < NI; ++n)
                    acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        e2m1_operand(fa[m]), e2m1_operand(fb[n]), acc[m][n], 4, 4, s, sa[m], s, sb[n]);
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
        if (st + 1 < stages)
            leave_scales(buf ^ 1);
        // the next stage's copies have landed, and no wave still reads this one
        MOE_WAIT_VMCNT(0);
        __syncthreads();
    }
    // lane l holds column l % 32, rows 8 (i / 4) + 4 (l / 32) + i % 4
#pragma unroll
    for (int m = 0; m < MI; ++m)
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const int c = col0 + (wn * NI + n) * 32 + lr;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = (wm * MI + m) * 32 + 8 * (i / 4) + 4 * lg + i % 4;
                if (r < t.rows && c < a.N)
                    store_y<T>(a, t.row0 + r, c, acc[m][n][i]);
            }
        }
}

// ------------------------------------------------------------ launchers

namespace {

// Workgroups that cover every tile: row tiles (grouped: at most one partial
// tile per segment beyond the full ones, and no more than rows) times column
// tiles, rounded so that every XCD's share is whole.  0 if it does not fit.
unsigned tile_grid(const MxGemmArgs& a, int bm, int col_tiles)
{
    int64_t rt = (a.R + bm - 1) / bm;
    if (a.offsets)
        rt = std::min<int64_t>(a.R, a.R / bm + a.E);
    const int64_t g = (rt * col_tiles + 7) / 8 * 8;
    return g < (INT64_C(1) << 31) ? (unsigned)g : 0u;
}

template <class T, int MT, int NT, int WV>
hipError_t launch_few(const MxGemmArgs& a, hipStream_t s)
{
    const int ct = (a.N + 16 * NT - 1) / (16 * NT);
    const unsigned grid = tile_grid(a, 16 * MT, ct);
    if (!grid)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((mxfp4_rows<T, MT, NT, WV>), dim3(grid), dim3(64 * WV), 0, s, a, ct);
    return hipGetLastError();
}

template <class T, int WM, int WN, int MI, int NI>
hipError_t launch_tile(const MxGemmArgs& a, hipStream_t s)
{
    constexpr int BM = WM * MI * 32, BN = WN * NI * 32;
    constexpr int smem = 2 * (BM + BN) * (128 + 8);
    static_assert(smem <= 160 * 1024, "LDS");
    const int ct = (a.N + BN - 1) / BN;
    const unsigned grid = tile_grid(a, BM, ct);
    if (!grid)
        return hipErrorInvalidValue;
    auto kernel = mxfp4_tile<T, WM, WN, MI, NI>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * WM * WN), smem, s, a, ct);
    return hipGetLastError();
}

template <class T>
hipError_t launch(const MxGemmArgs& a, hipStream_t s)
{
    const double mean = (double)a.R / a.E;
    if (mean <= 16)
        return launch_few<T, 1, 1, 8>(a, s);
    if (mean <= 48)
        return launch_few<T, 2, 2, 8>(a, s);
    if (mean <= 512)
        return launch_tile<T, 2, 4, 2, 1>(a, s);
    return launch_tile<T, 2, 4, 4, 2>(a, s);
}

}  // namespace

hipError_t launch_gemm_mxfp4(const MxGemmArgs& a, hipStream_t s)
{
    switch (a.dtype) {
    case MOE_DTYPE_BF16: return launch<Bf16>(a, s);
    case MOE_DTYPE_F16: return launch<F16>(a, s);
    case MOE_DTYPE_F32: return launch<F32>(a, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace moe
