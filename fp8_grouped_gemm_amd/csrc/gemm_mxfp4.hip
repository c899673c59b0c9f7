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
#include <cmath>
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

// Inclusive sum over the lanes below and including this one.
__device__ __forceinline__ int lane_sums(int v, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d);
        if (lane >= d)
            v += u;
    }
    return v;
}

// Row tile and column tile of this workgroup.  Row tiles of BM rows are
// numbered over all segments in expert order; a wave looks at 64 experts at
// a time, and every wave does so for itself.  Workgroups go to the 8 XCDs
// round-robin, each XCD takes a contiguous share of the tiles, and tiles run
// in bands of up to 8 row tiles, column by column, so that the tiles an XCD
// works on at one time share rows of a and of b in its L2.
template <int BM>
__device__ __forceinline__ RowTile pick_tile(const MxGemmArgs& a, int col_tiles, int lane, int& ct)
{
    constexpr int kBand = 8;
    const bool grouped = a.offsets != nullptr;
    int first = 0, n = 0, tiles = 0, upto = 0;  // of the lane's expert in the last 64 looked at
    int row_tiles = (a.R + BM - 1) / BM;
    if (grouped) {
        row_tiles = 0;
        for (int e0 = 0; e0 < a.E; e0 += 64) {
            n = 0;
            if (e0 + lane < a.E)
                segment(a, e0 + lane, first, n);
            tiles = (n + BM - 1) / BM;
            upto = lane_sums(tiles, lane);
            // (at most 2^30 in 64 segments; the cap, which segments that do not
            // overlap keep below, holds every sum of them inside 32 bits)
            row_tiles = min(row_tiles + __builtin_amdgcn_readlane(upto, 63), a.R / BM + a.E);
        }
    }
    const int total = row_tiles * col_tiles;
    const int share = (total + 7) / 8;
    const int wg = workgroup();
    const int i = wg / 8, at = (wg % 8) * share + i;
    if (i >= share || at >= total)
        return {0, 0, 0};
    const int band = at / (kBand * col_tiles), in = at - band * kBand * col_tiles;
    const int tall = min(kBand, row_tiles - band * kBand);
    ct = in / tall;
    const int rt = band * kBand + in - ct * tall;
    if (!grouped)
        return {0, rt * BM, min(BM, a.R - rt * BM)};
    int before = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        if (a.E > 64) {  // (up to 64 experts: still in the registers)
            n = 0;
            if (e0 + lane < a.E)
                segment(a, e0 + lane, first, n);
            tiles = (n + BM - 1) / BM;
            upto = lane_sums(tiles, lane);
        }
        const uint64_t past = __ballot(before + upto > rt);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int skip = (rt - before - __builtin_amdgcn_readlane(upto - tiles, l)) * BM;
            return {e0 + l, __builtin_amdgcn_readlane(first, l) + skip,
                    min(BM, __builtin_amdgcn_readlane(n, l) - skip)};
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return {0, 0, 0};
}

// A buffer resource of `bytes` bytes at p (both wave-uniform); what lies past
// them reads as zeros, an offset of kOutside among it.
constexpr uint32_t kOutside = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t byte_rsrc(const uint8_t* p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), (short)0, (int)bytes, 0x00020000);
}

}  // namespace

// ---------------------------------------------------------------- few rows
//
// 16 MT rows x 16 NT columns per workgroup of WV waves that split K: wave w
// takes the 256-wide K steps w, w + WV, ... (so the workgroup reads WV * 128
// consecutive bytes of each weight row at a time), straight from memory into
// MFMA operands, D steps of each wave in flight, and the waves' sums meet in
// LDS in wave order.  (One row by 4096 x 7168: 6.4 us on the device, 2.4 TB/s,
// bound by the latency of a call that is over in a few loads; the host needs 7.)
// A step is two MFMAs per subtile pair: lane group g
// supplies K blocks 2 g and 2 g + 1 of the step's 8, so its two 16-byte loads
// are adjacent and the four groups read one whole 128-byte line of each row.
// Steps past the end are loads from outside the buffer resource: zeros.
template <int MT, int NT>
struct Step {
    uint4 a[MT][2], b[NT][2];
    int sa[MT], sb[NT];  // codes of the two blocks in bytes 0 and 1
};

template <class T, int MT, int NT, int WV, int D>
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
    const int nb = a.K / 32, full = nb / 8;  // K blocks, whole steps
    const uint32_t pitch = a.K / 2;
    const int col0 = ct * BN, cols = min(BN, a.N - col0);
    const int64_t b0 = (int64_t)t.e * a.N + col0;
    const auto ra = byte_rsrc(a.a + (int64_t)t.row0 * pitch, t.rows * pitch);
    const auto rb = byte_rsrc(a.b + b0 * pitch, cols * pitch);
    const auto rsa = byte_rsrc(a.a_sf + (int64_t)t.row0 * nb, t.rows * nb);
    const auto rsb = byte_rsrc(a.b_sf + b0 * nb, cols * nb);
    // (rows and columns past the tile lie outside the resources)
    auto load = [](__amdgpu_buffer_rsrc_t r, uint32_t off) {
        typedef unsigned int u4 __attribute__((ext_vector_type(4)));
        const u4 v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
        return make_uint4(v.x, v.y, v.z, v.w);
    };
    auto fetch = [&](Step<MT, NT>& s, int step) {
        const uint32_t blk = step * 8 + 2 * lg;
        const bool in = step < full;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint32_t r = 16 * n + lr, off = in ? r * pitch + blk * 16 : kOutside;
            s.b[n][0] = load(rb, off);
            s.b[n][1] = load(rb, off + 16);
            s.sb[n] = __builtin_amdgcn_raw_buffer_load_b16(rsb, (int)(in ? r * nb + blk : kOutside), 0, 0);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint32_t r = 16 * m + lr, off = in ? r * pitch + blk * 16 : kOutside;
            s.a[m][0] = load(ra, off);
            s.a[m][1] = load(ra, off + 16);
            s.sa[m] = __builtin_amdgcn_raw_buffer_load_b16(rsa, (int)(in ? r * nb + blk : kOutside), 0, 0);
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
    Step<MT, NT> s[D];
#pragma unroll
    for (int d = 0; d < D; ++d)
        fetch(s[d], wave + d * WV);
    for (int i = wave; i < full; i += D * WV) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            mul(s[d]);
            fetch(s[d], i + (D + d) * WV);
        }
    }
    if (nb % 8 != 0 && wave == full % WV) {  // the step K ends in: code by code
        const uint32_t blk = full * 8 + 2 * lg;
        const bool in0 = (int)blk < nb, in1 = (int)blk + 1 < nb;
        auto code2 = [&](__amdgpu_buffer_rsrc_t r, uint32_t off) {
            const int lo = __builtin_amdgcn_raw_buffer_load_b8(r, (int)(in0 ? off : kOutside), 0, 0);
            const int hi = __builtin_amdgcn_raw_buffer_load_b8(r, (int)(in1 ? off + 1 : kOutside), 0, 0);
            return lo | (hi << 8);
        };
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint32_t r = 16 * n + lr, off = r * pitch + blk * 16;
            s[0].b[n][0] = load(rb, in0 ? off : kOutside);
            s[0].b[n][1] = load(rb, in1 ? off + 16 : kOutside);
            s[0].sb[n] = code2(rsb, r * nb + blk);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint32_t r = 16 * m + lr, off = r * pitch + blk * 16;
            s[0].a[m][0] = load(ra, in0 ? off : kOutside);
            s[0].a[m][1] = load(ra, in1 ? off + 16 : kOutside);
            s[0].sa[m] = code2(rsa, r * nb + blk);
        }
        mul(s[0]);
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
        if (m >= t.rows || n >= cols)
            continue;
        float v = part[0][m][n];
#pragma unroll
        for (int w = 1; w < WV; ++w)
            v += part[w][m][n];
        T::store(a.y + (int64_t)(t.row0 + m) * a.y_ld + (int64_t)(col0 + n) * T::SIZE, v);
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
//
// 256 x 256 tiles at 8192 x 8192 x 7168: 233 us on Gaussian rows, 236 on uniform
// codes (4.1 PFLOP/s), 172 on zeros, the same inputs in every call.  Two things
// bound them.  The pipeline: 403 thousand cycles whatever the data, of which the
// matrix cores work 229 (57 %; other inputs in every call: 460 thousand, 50 %; LDS is
// active 31 %; what the rest waits for has not been told apart).  And power, which sets the
// clock: 2.24 GHz on zeros, 1.72 and 1.63 on the others.  (The matrix cores alone,
// never idle, sustain 6.2 PFLOP/s on random codes, 155 us, and 9.2 on zeros, 105 us.)
// Measured and not kept, us, uniform codes, when the form kept took 276 to 284: four
// waves of 128 x 128 297, 64 x 128 per wave 285, copies spread over three steps 290,
// raised wave priority 291, workgroups that walk tiles and copy the next one's
// first stages early 288.  Tiles between the ones kept, as then: 192 x 256 317 here and
// 203 for 196 at 12288 rows over 32 experts of 4096 x 4096 (112 for 118 at 6144), 128 x 256
// 395 and 241 (24.3 for 26.0 at 2048 x 4096 x 4096).
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

// 16 bytes per lane from byte `off` of the resource to LDS at lds + 16 * lane
// (NT: nontemporal).
template <bool NT>
__device__ __forceinline__ void dma16_rsrc(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t lds)
{
    const uint32_t at = __builtin_amdgcn_readfirstlane(lds);
    if constexpr (NT)
        asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dwordx4 %0, %1, 0 offen nt lds" ::"v"(off), "s"(r), "s"(at)
                     : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(r), "s"(at)
                     : "memory", "m0");
}

// ONCE: b is large and (nearly) read once, so it streams past the caches
// (streams_b).
template <class T, int WM, int WN, int MI, int NI, int NBUF, bool ONCE>
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
    const auto ra = byte_rsrc(a.a + (int64_t)t.row0 * pitch, t.rows * pitch);
    const auto rb = byte_rsrc(a.b + ((int64_t)t.e * a.N + col0) * pitch, cols * pitch);
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
        const uint32_t src = st * 8 + chunk < nb ? at : kOutside, dst = lds0 + buf * C::STAGE + q * W * 1024;
        if (q < QA)
            dma16_rsrc<false>(ra, src, dst);
        else
            dma16_rsrc<ONCE>(rb, src, dst);
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
            } else {  // the group K ends in: n codes, whole words and a last part
                struct __attribute__((packed, aligned(1))) U1 { uint32_t v; };
                const int n = nb - g * 8 * kCodeStages, part = n % 4;
                uint32_t end = 0;
                if (part && nb >= 4) {  // the row's last four codes, those before the part shifted out
                    end = reinterpret_cast<const U1*>(p + n - 4)->v >> (8 * (4 - part));
                } else {
                    for (int j = 0; j < part; ++j)
                        end |= (uint32_t)p[n - part + j] << (8 * j);
                }
                end |= 0x7F7F7F7Fu << (8 * part);
#pragma unroll
                for (int i = 0; i < 2 * kCodeStages; ++i)
                    codes[q][i] = 4 * i + 4 <= n ? reinterpret_cast<const U1*>(p + 4 * i)->v
                                                 : i == n / 4 ? end : 0x7F7F7F7Fu;
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
#pragma unroll
    for (int st = 0; st < NBUF - 1; ++st)
#pragma unroll
        for (int q = 0; q < C::COPIES; ++q)
            copy(st, st, q);
    fetch_codes(0);
    leave_codes(0);
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
    // whole aligned pieces bypass the caches: y is not read here, and what a
    // tile shares in its L2 stays (2048 x 4096 x 4096: 26.6 us cached, 25.1;
    // 8192 x 8192 x 7168, uniform codes, then: 278, 273; unaligned ones would be split)
    const bool nt = (reinterpret_cast<uintptr_t>(a.y) | a.y_ld) % 16 == 0;
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
                const rows_u32x4 v = *reinterpret_cast<const rows_u32x4*>(src);
                if (c + T::VEC <= a.N) {
                    if (nt)
                        store16<true>(dst, v);
                    else
                        store16(dst, v);
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
        rt = std::min<int64_t>(a.slots, a.slots / bm + a.E);
    const int64_t g = (rt * col_tiles + 7) / 8 * 8;
    return g < (INT64_C(1) << 31) ? (unsigned)g : 0u;
}

template <class T, int MT, int NT, int WV, int D>
hipError_t launch_few(const MxGemmArgs& a, hipStream_t s)
{
    const int ct = (a.N + 16 * NT - 1) / (16 * NT);
    const unsigned grid = tile_grid(a, 16 * MT, ct);
    if (!grid)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((mxfp4_rows<T, MT, NT, WV, D>), grid_of(grid), dim3(64 * WV), 0, s, a, ct);
    return hipGetLastError();
}

template <class T, int WM, int WN, int MI, int NI, int NBUF, bool ONCE = false>
hipError_t launch_tile(const MxGemmArgs& a, hipStream_t s)
{
    using C = TileCfg<T, WM, WN, MI, NI, NBUF>;
    const int ct = (a.N + C::BN - 1) / C::BN;
    const unsigned grid = tile_grid(a, C::BM, ct);
    if (!grid)
        return hipErrorInvalidValue;
    auto kernel = mxfp4_tile<T, WM, WN, MI, NI, NBUF, ONCE>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(kernel, grid_of(grid), dim3(C::TH), C::SMEM, s, a, ct);
    return hipGetLastError();
}

// The kernel a call takes: the one whose estimated time is least.  A kernel's
// workgroups run `per_cu` to a compute unit, each fix + step * (256-wide K
// steps) microseconds at that occupancy and fix1 + step1 * steps alone on its
// unit, in whole rounds over the 256 units.  The figures are fits to a sweep
// of 34 shapes (rows 1 to 12288, n and k 512 to 8192, 1 to 64 experts); over it
// the choice is 2 % from the best of all (geometric mean), 12 % at worst, where
// a call is host time.  Some of its points, us per call (7 of them the host's):
//   rows x n x k (experts)   16x16  32x16  32x64  32x128  64x128  128^2  256^2
//   1 x 4096 x 7168            7.8    7.7   11.0    16.5    13.0   20.6   37.2
//   32 x 512 x 8192            9.1   10.6   11.2    14.2    13.8   18.9   40.9
//   128 x 4096 x 7168         44.1   34.2   12.2    18.7    15.5   24.5   39.4
//   300 x 8192 x 1024         43.7   38.0   11.2     7.5     8.6    7.9   11.5
//   512 x 4096 x 4096          101   76.5   18.7    14.3    11.7   16.1   26.7
//   2048 x 4096 x 4096         400    301   66.4    48.1    40.0   26.4   30.8
//   4096 x 4096 x 4096         798    599    126    90.5    79.0   51.1   40.5
//   6144 x 4096 x 4096 (32)   1261   1053    276     193     176    119    118
//   12288 x 4096 x 4096 (32)  2469   2028    492     326     317    204    170
// A call that reads b once, and more of it than the L2s hold twice over
// (streams_b), takes its tile from the last three kernels, whose copies of b
// are nontemporal (32 x 128 with two and three buffers, 128^2), and of the
// others the few-rows ones; us:
//   rows x n x k (experts)   cached 32x128   128^2   nt 32x128, 2   3   128^2
//   32 x 4096 x 4096 (32)             31.3    46.0         29.3   35.5   45.1
//   256 x 4096 x 4096 (32)            63.6    61.1         57.9   49.3   57.3
//   768 x 4096 x 4096 (32)            63.4    64.1         61.4   64.2   59.6
//   1536 x 4096 x 4096 (32)           85.8    76.6         94.1   95.0   70.5
//   2048 x 4096 x 4096 (dense)        48.1    26.4         69.4   68.9   28.7
// The two sides of streams_b's limits, the choice among either set, over 32
// experts of 4096 columns with ROWS each, weights that no cache holds, us:
//   b, ROWS          1       12       24       48       96      128      192      256
//    40 MB    9.8 10.7  22 17    18 19    24 23    31 31    39 37    42 45    44 55
//    66 MB   12.5 14.5  35 30    27 31    29 33    51 44    52 46    55 58    58 71
//   128 MB   16.5 14.6  39 28.5  34 34    38 38    49 49    66 52    66 65    71 81
//   256 MB   34   30    62 50    63 57    76 63    87 85    93 92   117 128  122 155
// (the same 66 MB in every call, which the last-level cache then keeps: 24 rows 22 and
// 29).  Between 32 and 128 rows an expert the two differ by the tile they lead to.
// A dense call that streams has few tiles, and of the smaller cached ones a
// whole round may run where the nontemporal ones leave half the units idle, so
// those stay in the choice while they fit one round.  us, without and with
// them: 16384 columns x 9216, 1 row 24.7 and 20.5, 32 rows 26.8 and 20.8, 96 rows 40.3
// and 28.0; 12288 x 16384, 96 rows 66.2 and 42.7; 32768 x 8192, 64 rows 39.9 and 35.2.
// Past one round they lose: 131072 x 2048, 1 row 25.6 and 32.4.  Over 105 such
// calls (8192 to 151936 columns, 1 to 128 rows) the choice is 2 % from the best of all
// kernels (geometric mean; 12 % without them), 21 % at worst.
struct Choice {
    int bm, bn, per_cu;
    double fix, step, fix1, step1;
};
constexpr Choice kChoices[] = {
    {16, 16, 2, 2.0, 0.22, 2.0, 0.12},   {32, 16, 2, 2.0, 0.31, 2.0, 0.16},
    {32, 64, 2, 1.5, 0.40, 1.5, 0.28},   {32, 128, 3, 3.0, 0.95, 2.0, 0.40},
    {64, 128, 1, 2.5, 0.47, 2.5, 0.36},  {128, 128, 2, 5.0, 1.30, 4.0, 0.75},
    {256, 256, 1, 6.0, 2.10, 6.0, 2.10}, {32, 128, 3, 3.0, 1.60, 2.0, 0.40},
    {32, 128, 2, 3.0, 1.25, 2.0, 0.35},  {128, 128, 2, 5.0, 1.45, 4.0, 0.75},
};
constexpr int kNumChoices = sizeof(kChoices) / sizeof(kChoices[0]);

bool streams_b(int E, int R, int N, int K)
{
    return (int64_t)E * N * (K / 2) > (INT64_C(64) << 20) && R <= (int64_t)E * 128;
}

// Row tiles of bm rows: exact for a dense product; over segments, whose
// lengths only the device knows, the routed experts at least and half a tile
// for each beyond the full ones.
double row_tiles(int E, int R, bool grouped, int bm)
{
    if (!grouped)
        return (R + bm - 1) / bm;
    const double routed = E * (1.0 - std::exp(-(double)R / E));
    return std::max(routed, (double)R / bm + 0.5 * routed);
}

int choose(int E, int R, int N, int K, bool grouped)
{
    constexpr int kUnits = 256;
    const double steps = (K + 255) / 256;
    const bool once = streams_b(E, R, N, K);
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < kNumChoices; ++i) {
        const Choice& c = kChoices[i];
        const double tiles = row_tiles(E, R, grouped, c.bm) * ((N + c.bn - 1) / c.bn);
        const bool one_round = !grouped && (i == 2 || i == 4) && tiles <= kUnits;
        if (i >= 2 && (i >= 7) != once && !(once && one_round))
            continue;
        const double us = tiles <= kUnits ? c.fix1 + c.step1 * steps
                                          : std::ceil(tiles / (kUnits * c.per_cu)) * (c.fix + c.step * steps);
        if (i == 0 || us < least) {
            best = i;
            least = us;
        }
    }
    return best;
}

template <class T>
hipError_t launch(const MxGemmArgs& a, hipStream_t s)
{
    const int choice = choose(a.E, a.slots, a.N, a.K, a.offsets != nullptr);
    switch (choice) {
    case 0: return launch_few<T, 1, 1, 8, 2>(a, s);
    case 1: return launch_few<T, 2, 1, 8, 2>(a, s);
    case 2: return launch_tile<T, 1, 2, 1, 1, 4>(a, s);
    case 3: return launch_tile<T, 1, 4, 1, 1, 2>(a, s);
    case 4: return launch_tile<T, 2, 4, 1, 1, 3>(a, s);
    case 5: return launch_tile<T, 2, 2, 2, 2, 2>(a, s);
    case 6: return launch_tile<T, 2, 4, 4, 2, 2>(a, s);
    case 7: return launch_tile<T, 1, 4, 1, 1, 2, true>(a, s);
    case 8: return launch_tile<T, 1, 4, 1, 1, 3, true>(a, s);
    default: return launch_tile<T, 2, 2, 2, 2, 2, true>(a, s);
    }
}

}  // namespace

void gemm_mxfp4_tile(int E, int R, int N, int K, bool grouped, int& bm, int& bn)
{
    const Choice& c = kChoices[choose(E, R, N, K, grouped)];
    bm = c.bm;
    bn = c.bn;
}

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
