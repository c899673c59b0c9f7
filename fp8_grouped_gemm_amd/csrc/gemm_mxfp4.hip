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
// 32 x 32; K in stages of 256 (one 128-byte line of each row, four MFMA
// steps), copied asynchronously into a ring of NBUF LDS buffers.
//
// Pipeline: a wave reads the fragments of step s + 1 while it multiplies
// step s, and the stage's one barrier stands before its last products, so the
// matrix cores run through it.  At the barrier every wave has read its last
// fragments of the stage, whose buffer is then free, and its copies of the
// next stage have landed; the copies into the freed buffer go out right
// behind it, one by one between products (issued together they fill the
// memory pipeline and hold the products back).
//
// One copy instruction of a wave brings 8 rows x 128 bytes, whole lines from
// memory and 1 KiB in a row of LDS (16 rows x 64 bytes took 1.6 times as
// long per byte from L2).  A row's eight 16-byte chunks sit at position
// chunk ^ key(row), key = (row & 7) ^ (row >> 3 & 1): any 8 (16) consecutive
// rows then hold a given chunk in different banks of 32 (64), and the
// fragment reads run without conflicts.  Blocks past the end of K are copied
// from outside the buffer resource, which reads as zeros.
//
// Scale codes pass through registers into LDS, 32 (4 stages) of a row at a
// time; a byte permute of a row's 8 codes of one stage gives the MFMAs' scale
// register for its four steps (lane group g takes codes 2 s + g, step s byte
// s).  Codes past the end of K are 127, scale 1.
typedef int v4i __attribute__((ext_vector_type(4)));
constexpr int kCodeStages = 4;  // stages per load of scale codes

template <class T, int WM, int WN, int MI, int NI, int NBUF>
struct TileCfg {
    static constexpr int BM = WM * MI * 32, BN = WN * NI * 32, ROWS = BM + BN;
    static constexpr int W = WM * WN, TH = 64 * W;
    static constexpr int STAGE = ROWS * 128;
    static constexpr int COPIES = ROWS / 8 / W;         // per wave and stage
    static constexpr int CODES = (ROWS + TH - 1) / TH;  // rows of scale codes per thread
    static constexpr int SC = kCodeStages * ROWS * 8;   // one load of codes in LDS
    static constexpr int SMEM = NBUF * STAGE + 2 * SC;
    // the result leaves through LDS, 32 rows of a wave at a time
    static constexpr int OUT_LD = NI * 32 * T::SIZE + 16;
    static_assert(BM % (8 * W) == 0 && BN % (8 * W) == 0, "whole copies per wave and operand");
    static_assert(W % 2 == 0, "a wave's copies share the parity of row / 8");
    static_assert(SMEM <= 160 * 1024 && W * 32 * OUT_LD <= SMEM, "LDS");
};

// A buffer resource of `bytes` bytes at p (both wave-uniform); what lies past
// them reads as zeros.
__device__ __forceinline__ v4i byte_rsrc(const uint8_t* p, uint32_t bytes)
{
    const uint64_t b = reinterpret_cast<uint64_t>(p);
    v4i r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32) & 0xFFFF);
    r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
    r[3] = 0x00020000;
    return r;
}

// 16 bytes per lane from byte `off` of the resource to LDS at lds + 16 * lane.
__device__ __forceinline__ void dma16_rsrc(const v4i& r, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(r),
                 "s"(__builtin_amdgcn_readfirstlane(lds))
                 : "memory", "m0");
}

template <class T, int WM, int WN, int MI, int NI, int NBUF>
__global__ __launch_bounds__(64 * WM * WN) void mxfp4_tile(MxGemmArgs a, int col_tiles)
{
    using C = TileCfg<T, WM, WN, MI, NI, NBUF>;
    constexpr int BM = C::BM, BN = C::BN, ROWS = C::ROWS, W = C::W, TH = C::TH;
    extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
    uint8_t* const sc = smem + NBUF * C::STAGE;  // [2][kCodeStages][ROWS][8]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int ct = 0;
    const RowTile t = pick_tile<BM>(a, col_tiles, lane, ct);
    if (t.rows <= 0)
        return;
    const int col0 = ct * BN, cols = min(BN, a.N - col0);
    const int nb = a.K / 32, stages = (nb + 7) / 8;
    const uint32_t pitch = a.K / 2;
    const v4i ra = byte_rsrc(a.a + (int64_t)t.row0 * pitch, t.rows * pitch);
    const v4i rb = byte_rsrc(a.b + ((int64_t)t.e * a.N + col0) * pitch, cols * pitch);
    const uint8_t* const asf = a.a_sf + (int64_t)t.row0 * nb;
    const uint8_t* const bsf = a.b_sf + ((int64_t)t.e * a.N + col0) * nb;

    // Copy q of this wave brings LDS rows 8 (q W + wave) .. + 7, lane l the
    // chunk at position l % 8 of row l / 8; rows past the tile lie outside the
    // resource (zeros).  off0: the lane's place in stage 0 of copy 0.
    const int chunk = (lane & 7) ^ (lane >> 3) ^ (wave & 1);
    const uint32_t off0 = (8 * wave + (lane >> 3)) * pitch + chunk * 16;
    const uint32_t lds0 = lds_addr(smem) + wave * 1024;
    auto copy = [&](int st, int buf, int q) {
        constexpr int QA = BM / 8 / W;  // copies of a's rows
        const uint32_t at = off0 + (q < QA ? q : q - QA) * (8 * W) * pitch + st * 128;
        dma16_rsrc(q < QA ? ra : rb, st * 8 + chunk < nb ? at : 0x80000000u,
                   lds0 + buf * C::STAGE + q * W * 1024);
    };
    // Scale codes: thread i takes rows i, i + TH, ... of the ROWS.
    auto code_row = [&](int row) {  // rows past the tile repeat its last
        return row < BM ? asf + min(row, t.rows - 1) * nb : bsf + min(row - BM, cols - 1) * nb;
    };
    uint32_t codes[C::CODES][2 * kCodeStages];
    auto fetch_codes = [&](int g) {
        struct __attribute__((packed, aligned(1))) U4 { uint32_t v[4]; };
#pragma unroll
        for (int q = 0; q < C::CODES; ++q) {
            const int row = q * TH + threadIdx.x;
            const uint8_t* p = code_row(row) + g * 8 * kCodeStages;
            if ((g + 1) * 8 * kCodeStages <= nb) {
#pragma unroll
                for (int i = 0; i < kCodeStages / 2; ++i) {
                    const U4 u = *reinterpret_cast<const U4*>(p + 16 * i);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        codes[q][4 * i + j] = u.v[j];
                }
            } else {  // the group K ends in, byte by byte
                const int last = nb - 1 - g * 8 * kCodeStages;
#pragma unroll
                for (int i = 0; i < 2 * kCodeStages; ++i) {
                    uint32_t w = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t c = p[max(0, min(4 * i + j, last))];
                        w |= (4 * i + j <= last ? c : 127u) << (8 * j);
                    }
                    codes[q][i] = w;
                }
            }
        }
    };
    auto leave_codes = [&](int g) {
#pragma unroll
        for (int q = 0; q < C::CODES; ++q) {
            const int row = q * TH + threadIdx.x;
            if (ROWS % TH == 0 || row < ROWS)
#pragma unroll
                for (int i = 0; i < kCodeStages; ++i)
                    *reinterpret_cast<uint2*>(sc + (g & 1) * C::SC + (i * ROWS + row) * 8) =
                        make_uint2(codes[q][2 * i], codes[q][2 * i + 1]);
        }
    };

    const int wm = wave / WN, wn = wave % WN;
    const int lr = lane & 31, lg = lane >> 5;
    const int key = (lr & 7) ^ ((lr >> 3) & 1);
    const uint32_t la = (wm * MI * 32 + lr) * 128, lb = (BM + wn * NI * 32 + lr) * 128;
    const uint32_t ca = (wm * MI * 32 + lr) * 8, cb = (BM + wn * NI * 32 + lr) * 8;
    const uint32_t pick = lg ? 0x07050301u : 0x06040200u;  // codes 1,3,5,7 or 0,2,4,6
    v16f acc[MI][NI];
#pragma unroll
    for (int m = 0; m < MI; ++m)
#pragma unroll
        for (int n = 0; n < NI; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[m][n][i] = 0.f;
    uint4 fa[2][MI], fb[2][NI];  // fragments of even and odd steps
    uint2 ua[MI], ub[NI];        // codes of the next stage as read
    int sa[MI], sb[NI];          // scale registers of the current one
    auto read = [&](int buf, int s) {
        const uint8_t* const p = smem + buf * C::STAGE + (((2 * s + lg) ^ key) * 16);
#pragma unroll
        for (int m = 0; m < MI; ++m)
            fa[s & 1][m] = *reinterpret_cast<const uint4*>(p + la + m * 4096);
#pragma unroll
        for (int n = 0; n < NI; ++n)
            fb[s & 1][n] = *reinterpret_cast<const uint4*>(p + lb + n * 4096);
    };
    auto read_codes = [&](int st) {
        const uint8_t* const p = sc + ((st / kCodeStages) & 1) * C::SC + (st % kCodeStages) * ROWS * 8;
#pragma unroll
        for (int m = 0; m < MI; ++m)
            ua[m] = *reinterpret_cast<const uint2*>(p + ca + m * 256);
#pragma unroll
        for (int n = 0; n < NI; ++n)
            ub[n] = *reinterpret_cast<const uint2*>(p + cb + n * 256);
    };
    // step S's products; `between(m)` runs after those of row subtile m
    auto mul = [&](auto S, auto between) {
        constexpr int s = decltype(S)::value;
#pragma unroll
        for (int m = 0; m < MI; ++m) {
#pragma unroll
            for (int n = 0; n < NI; ++n)
                acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    e2m1_operand(fa[s & 1][m]), e2m1_operand(fb[s & 1][n]), acc[m][n], 4, 4, s, sa[m], s, sb[n]);
            __builtin_amdgcn_sched_barrier(0);
            between(m);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto nothing = [](int) {};
    constexpr int HALF = C::COPIES / 2;

    // prologue: the first codes, stages 0 .. NBUF - 2 and half of the next
    fetch_codes(0);
    leave_codes(0);
#pragma unroll
    for (int st = 0; st < NBUF - 1; ++st)
#pragma unroll
        for (int q = 0; q < C::COPIES; ++q)
            copy(st, st, q);
    MOE_WAIT_VMCNT((NBUF - 2) * C::COPIES);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < HALF; ++q)
        copy(NBUF - 1, NBUF - 1, q);
    read(0, 0);
    read_codes(0);
    int buf = 0;  // of the current stage
    // One stage, as one basic block: past a branch the compiler sinks
    // products to where their sums are used.  (So the copies of stages past
    // the last are issued too, and read zeros without a memory access.)
    auto stage = [&](int st, auto LAST) {
        constexpr bool last = decltype(LAST)::value;  // of its code group
        const int next = buf + 1 == NBUF ? 0 : buf + 1, prev = buf == 0 ? NBUF - 1 : buf - 1;
#pragma unroll
        for (int m = 0; m < MI; ++m)
            sa[m] = (int)__builtin_amdgcn_perm(ua[m].y, ua[m].x, pick);
#pragma unroll
        for (int n = 0; n < NI; ++n)
            sb[n] = (int)__builtin_amdgcn_perm(ub[n].y, ub[n].x, pick);
        read(buf, 1);
        __builtin_amdgcn_sched_barrier(0);
        mul(std::integral_constant<int, 0>{}, [&](int m) {
#pragma unroll
            for (int q = HALF + m; q < C::COPIES; q += MI)
                copy(st + NBUF - 1, prev, q);
        });
        read(buf, 2);
        __builtin_amdgcn_sched_barrier(0);
        mul(std::integral_constant<int, 1>{}, nothing);
        read(buf, 3);
        __builtin_amdgcn_sched_barrier(0);
        mul(std::integral_constant<int, 2>{}, nothing);
        // stage st + 1 landed, NBUF - 2 newer ones may be in flight (the
        // compiler's wait for the code loads takes in those too)
        if constexpr (last)
            leave_codes(st / kCodeStages + 1);
        MOE_WAIT_VMCNT((NBUF - 2) * C::COPIES);
        __syncthreads();
        read(next, 0);  // (past the last stage: read, not used)
        read_codes(st + 1);
        __builtin_amdgcn_sched_barrier(0);
        mul(std::integral_constant<int, 3>{}, [&](int m) {
#pragma unroll
            for (int q = m; q < HALF; q += MI)
                copy(st + NBUF, buf, q);
        });
        buf = next;
    };
    for (int g = 0; g * kCodeStages < stages; ++g) {
        if ((g + 1) * kCodeStages < stages)
            fetch_codes(g + 1);
        const int end = min(stages, (g + 1) * kCodeStages);
        for (int st = g * kCodeStages; st < end - 1; ++st)
            stage(st, std::false_type{});
        stage(end - 1, std::true_type{});
    }
    MOE_WAIT_VMCNT(0);
    __syncthreads();  // every wave is done with the stages' LDS
    // lane l holds column l % 32, rows 8 (i / 4) + 4 (l / 32) + i % 4 of a
    // subtile: 32 rows at a time go through LDS and leave as 16-byte stores
    uint8_t* const out = smem + wave * 32 * C::OUT_LD;
    constexpr int PIECES = NI * 32 / T::VEC;  // 16-byte pieces of a row
    constexpr int PER = 64 / PIECES;          // rows per store instruction
    const int c = col0 + wn * NI * 32 + (lane % PIECES) * T::VEC;
#pragma unroll
    for (int m = 0; m < MI; ++m) {
#pragma unroll
        for (int n = 0; n < NI; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                T::store(reinterpret_cast<char*>(out) + (8 * (i / 4) + 4 * lg + i % 4) * C::OUT_LD +
                             (n * 32 + lr) * T::SIZE, acc[m][n][i]);
        // (a wave reads only what it wrote and LDS serves a wave in order;
        // the compiler must not move the accesses, of other types, past here)
        asm volatile("" ::: "memory");
#pragma unroll
        for (int q = 0; q < 32 / PER; ++q) {
            const int lrow = q * PER + lane / PIECES;
            const int r = (wm * MI + m) * 32 + lrow;
            const char* src = reinterpret_cast<const char*>(out) + lrow * C::OUT_LD + (lane % PIECES) * 16;
            if (r < t.rows && c < a.N) {
                char* dst = a.y + (int64_t)(t.row0 + r) * a.y_ld + (int64_t)c * T::SIZE;
                if (c + T::VEC <= a.N) {
                    store16(dst, *reinterpret_cast<const rows_u32x4*>(src));
                } else {
                    for (int i = 0; i < a.N - c; ++i)
                        T::store(dst + i * T::SIZE, T::load(src + i * T::SIZE));
                }
            }
        }
        asm volatile("" ::: "memory");
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

template <class T, int WM, int WN, int MI, int NI, int NBUF>
hipError_t launch_tile(const MxGemmArgs& a, hipStream_t s)
{
    using C = TileCfg<T, WM, WN, MI, NI, NBUF>;
    const int ct = (a.N + C::BN - 1) / C::BN;
    const unsigned grid = tile_grid(a, C::BM, ct);
    if (!grid)
        return hipErrorInvalidValue;
    auto kernel = mxfp4_tile<T, WM, WN, MI, NI, NBUF>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(C::TH), C::SMEM, s, a, ct);
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
        return launch_tile<T, 2, 4, 2, 1, 2>(a, s);
    return launch_tile<T, 2, 4, 4, 2, 2>(a, s);
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
