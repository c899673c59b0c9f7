// Weight gradients of the experts from rows kept in 8 bits (include/moe_ops.h:
// moe_gemm_wgrad):
//   dw[e, i, k] = sum over the rows r of expert e of dy[r, i] x[r, k],  x = code * scale
//
// A product whose contraction runs over the rows, so that both operands lie the
// wrong way round in memory for the matrix instruction (v_mfma_f32_32x32x16, whose
// lanes take 8 adjacent r of one column).  A stage of kStage rows is brought into
// LDS as it lies, dy's columns and x's side by side, x decoded to dy's type on the
// way; the transposing LDS read (ds_read_b64_tr_b16: 16 lanes read four rows of 16
// columns and get four rows of one column each) turns it.  Half a wave reads four
// rows of 64 bytes, whose 64-byte slots are exchanged by the row (slot ^ row), so
// that they lie in different banks.
//
// The stages are double-buffered: a stage's loads are under way in registers while
// the one before is multiplied.  Rows past the segment and columns past the
// matrix enter as zeros.  Where few tiles and many rows leave compute units idle, the
// rows are split over workgroups whose f32 sums meet in the workspace and are added in
// a fixed order by a second kernel.
//
// 8192^3 in bf16: 890 - 930 us, 1180 - 1235 TFLOP/s (a library product of bf16 operands that lie so: 1180).
// 32 experts of 384 rows, 4096 x 4096 to bf16: 540 - 570 us; of a tile's 33.7 thousand cycles
// 18.9 are its six stages (matrix cores busy 35 % of all), 7.0 the start and the first loads, 7.8 the
// results.  Slower there: workgroups that walk tiles and load the next one's first stages early
// (606 - 650), two workgroups a compute unit with half the tile each (621 - 650), stages of 32 rows (643 for 598), a
// second register set of loads (spills).
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
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) rows_u32x4 lds_u32x4;

constexpr int kMostSplit = 16;
constexpr int kStrip = 4;
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

template <bool HI>
__device__ __forceinline__ uint32_t scaled2(Bf16, uint32_t q, float scale)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)q, scale, HI));
}

template <bool HI>
__device__ __forceinline__ uint32_t scaled2(F16, uint32_t q, float scale)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)q, scale, HI));
}

// Byte of element (row, col) of a stage's matrix of COLS 16-bit columns.
template <int COLS>
__device__ __forceinline__ int lds_at(int row, int col)
{
    constexpr int kSlots = COLS / 32 < 8 ? COLS / 32 : 8;
    return row * COLS * 2 + ((col * 2) ^ ((row & (kSlots - 1)) << 6));
}

// Where in its row of LDS x's column c (a multiple of 16) lies: of each 64 columns the 32 even
// ones first, then the odd ones.
__device__ __forceinline__ int x_place(int c) { return (c & ~63) + (c & 63) / 2; }

// Of the 8 rows of column c0 + lane % 32 that the lane gives the matrix instruction, the
// byte where its first read starts: rows 4 (lane / 32) .. + 3, and the same 8 rows on
// (the same set for both operands, whose order the sum does not know).
template <int COLS>
__device__ __forceinline__ int frag_at(int c0, int lane)
{
    return lds_at<COLS>(4 * (lane >> 5) + ((lane & 15) >> 2), c0 + (lane & 16) + 4 * (lane & 3));
}

template <int COLS>
__device__ __forceinline__ Frag read_frag(lds_char* at, int r0)
{
    Frag f;
    f.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + r0 * COLS * 2));
    f.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + (r0 + 8) * COLS * 2));
    return f;
}

// code * scale in f32.  (A product that goes to f16 would be rounded by the instruction that
// converts it, once instead of twice: both types take the f32 value, as the header says.)
template <class E>
__device__ __forceinline__ float product(float code, float scale)
{
    float p = code * scale;
    if constexpr (__is_same(E, F16))
        asm("" : "+v"(p));
    return p;
}

// 16 codes times their scale, rounded to E: the eight of even and the eight of odd columns.
// A power of two in one instruction (equal to the product's rounding for every code and
// scale code, 0 and 0xFF among them; f16 keeps the sign of -0).
template <class E, bool MX>
__device__ __forceinline__ void decode16(rows_u32x4 q, uint32_t sf, rows_u32x4* out)
{
    const float scale = __uint_as_float(!MX ? sf : sf == 0 ? 0x400000u : sf == 0xFFu ? 0x7FC00000u : sf << 23);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // bytes h, h + 2, h + 4, h + 6 of eight codes
            const uint32_t c = __builtin_amdgcn_perm(q[2 * i + 1], q[2 * i], h ? 0x07050301u : 0x06040200u);
            if constexpr (MX) {
                out[h][2 * i] = scaled2<false>(E{}, c, scale);
                out[h][2 * i + 1] = scaled2<true>(E{}, c, scale);
            } else {
                typedef float f2 __attribute__((ext_vector_type(2)));
                const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false);
                const f2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
                out[h][2 * i] = E::pack2(product<E>(a[0], scale), product<E>(a[1], scale));
                out[h][2 * i + 1] = E::pack2(product<E>(b[0], scale), product<E>(b[1], scale));
            }
        }
}

// A buffer of `bytes` bytes, past whose end loads give zeros; p and bytes are the same in
// every lane (said to the compiler, which else loops over the lanes' values).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, unsigned bytes)
{
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)u), hi = __builtin_amdgcn_readfirstlane((int)(u >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uint64_t)hi << 32 | lo), 0,
                                             __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}

// First row and number of rows of a group's share `s` of S (whole stages but the last).
__device__ __forceinline__ void share(const WgradArgs& a, int e, int s, int64_t& first, int& rows)
{
    int lo = 0, all = a.R;
    if (a.offsets) {
        lo = max(a.offsets[e], 0);
        const int64_t hi = a.counts ? (int64_t)lo + max(a.counts[e], 0) : (int64_t)a.offsets[e + 1];
        all = (int)max(min(hi, (int64_t)a.R) - lo, INT64_C(0));
    }
    const int per = ((all + a.split - 1) / a.split + kShareRows - 1) / kShareRows * kShareRows;
    const int at = min(per * s, all);  // (rows are below 2^28, shares at most 16)
    first = (int64_t)lo + at;
    rows = min(per, all - at);
}

// One value to dw (type OUT), added to what is there with `add`.
template <class OUT>
__device__ __forceinline__ void put(char* p, float v, bool add)
{
    if (add)
        v += OUT::load(p);
    OUT::store(p, v);
}

// Two adjacent values of dw, whose address is a multiple of one value's size: as they are
// read, and written.
template <class OUT>
struct Two {
    typedef unsigned int Raw;
    static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t from, unsigned at)
    {
        return __builtin_amdgcn_raw_buffer_load_b32(from, at, 0, 0);
    }
    static __device__ __forceinline__ void store(char* p, float a, float b)
    {
        typedef unsigned int word __attribute__((aligned(2)));
        *reinterpret_cast<word*>(p) = OUT::pack2(a, b);
    }
    static __device__ __forceinline__ void add(char* p, float a, float b, Raw old)
    {
        const char* const o = reinterpret_cast<const char*>(&old);
        store(p, a + OUT::load(o), b + OUT::load(o + 2));
    }
};

template <>
struct Two<F32> {
    typedef unsigned int Raw __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t from, unsigned at)
    {
        return __builtin_amdgcn_raw_buffer_load_b64(from, at, 0, 0);
    }
    static __device__ __forceinline__ void store(char* p, float a, float b)
    {
        typedef float words __attribute__((ext_vector_type(2), aligned(4)));
        *reinterpret_cast<words*>(p) = (words){a, b};
    }
    static __device__ __forceinline__ void add(char* p, float a, float b, Raw old)
    {
        store(p, a + __uint_as_float(old[0]), b + __uint_as_float(old[1]));
    }
};

// A wave's blocks of dw.  Lane l holds rows 8 (k / 4) + 4 (l / 32) + k % 4 of each and,
// x's columns lying in LDS as they do, columns 2 (l % 32) of the first and 2 (l % 32) + 1 of
// the second of two blocks: adjacent ones, which a store writes as whole lines (64-byte
// runs of single columns: 2.6 TB/s for 5.4).  What is added to comes eight rows ahead, by
// loads that no branch parts (32 experts of 384 rows, 4096 x 4096: in bf16 1448 us one after the
// other, 746 so; 550 without, and in f32 1722, 1039 and 720).
template <class OUT, int MB, int NB>
__device__ __forceinline__ void put_blocks(char* dw, const v16f (&acc)[MB][NB], int row0, int col0, int N, int K,
                                           int lane, bool add)
{
    static_assert(NB == 2, "a lane's columns of two blocks are adjacent");
    constexpr int kAhead = 8;
    const bool inside = row0 + MB * 32 <= N && col0 + NB * 32 <= K;
    const bool column = col0 + 2 * (lane & 31) < K;
    char* const at = dw + ((int64_t)row0 * K + col0) * OUT::SIZE;
    const unsigned lane_at = (4 * (lane >> 5) * (unsigned)K + 2 * (lane & 31)) * OUT::SIZE;
    const auto row = [](int q) { return q / 16 * 32 + 8 * (q % 16 / 4) + q % 4; };
    const auto holds = [&](int r) { return inside || (column && row0 + r + 4 * (lane >> 5) < N); };
    const auto place = [&](int r) { return at + (int64_t)r * K * OUT::SIZE + lane_at; };
    if (!add) {
#pragma unroll
        for (int q = 0; q < 16 * MB; ++q)
            if (holds(row(q)))
                Two<OUT>::store(place(row(q)), acc[q / 16][0][q % 16], acc[q / 16][1][q % 16]);
        return;
    }
    typename Two<OUT>::Raw old[2][kAhead];
    const int64_t left = ((int64_t)(N - row0) * K - col0) * OUT::SIZE;
    const auto from = buffer(at, (unsigned)max(min(left, INT64_C(0x7FFFFFFF)), INT64_C(0)));
    const auto read = [&](int q0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = row(q0 + i);
            old[q0 / kAhead & 1][i] = Two<OUT>::load(from, holds(r) ? r * (unsigned)K * OUT::SIZE + lane_at : 0x80000000u);
        }
    };
    read(0);
#pragma unroll
    for (int q0 = 0; q0 < 16 * MB; q0 += kAhead) {
        if (q0 + kAhead < 16 * MB)
            read(q0 + kAhead);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int q = q0 + i, r = row(q);
            if (holds(r))
                Two<OUT>::add(place(r), acc[q / 16][0][q % 16], acc[q / 16][1][q % 16], old[q0 / kAhead & 1][i]);
        }
    }
}

}  // namespace

// A workgroup computes BM rows (dy's columns) by BN columns (x's) of an expert's dw over
// one share of its rows, its waves WM by WN each; kStage rows at a time.
template <class E, bool MX, int BM, int BN, int WM, int WN, int kStage>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, 2) void wgrad_tile(WgradArgs a, int tiles_m, int tiles_n)
{
    constexpr int kThreads = (BM / WM) * (BN / WN) * 64;
    constexpr int kBytes = kStage * (BM + BN) * 2;  // of a stage in LDS
    constexpr int kDy = kStage * BM / 8 / kThreads, kX = kStage * BN / 16 / kThreads;  // pieces a thread loads
    static_assert(kDy >= 1 && kX >= 1 && kStage * BN / 16 % kThreads == 0, "whole pieces");
    static_assert(kThreads % (BM / 8) == 0, "a thread's pieces lie in the same columns of dy");
    __shared__ __attribute__((aligned(16))) char stages_lds[2 * kBytes];
    lds_char* const lds = (lds_char*)stages_lds;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / (BN / WN) * WM, wn = wave % (BN / WN) * WN;

    // Workgroups go to the 8 dies in turn.  Of every unit's (a share of an expert's) tiles, counted
    // down strips of kStrip rows, a die takes a run: a compact block, whose rows and
    // columns its L2 holds (strips of 2, 4, 8 and 16 tiles: 32 experts of 384 rows, 4096 x 4096 567,
    // 564, 585 and 591 us; 8192^3 921, 918, 927 and 933; seven other sizes within 7 %, of 2 and 4
    // within 5); the die that gets the last, shorter run changes from unit to unit.  Shares
    // of one expert are equally long, so that the dies take runs of them all.
    const unsigned tiles = tiles_m * tiles_n, die = workgroup() & 7, turn = workgroup() >> 3;
    unsigned unit, tile;
    if (a.E == 1) {
        const unsigned all = tiles * a.split, at = die * ((all + 7) / 8) + turn;
        unit = turn < (all + 7) / 8 && at < all ? at / tiles : a.split;
        tile = at - unit * tiles;
    } else {
        const unsigned run = (tiles + 7) / 8;
        unit = turn / run;
        tile = ((die + unit) & 7) * run + turn - unit * run;
    }
    if (unit >= (unsigned)(a.E * a.split) || tile >= tiles)
        return;
    const int e = unit / a.split, s = unit - e * a.split;
    const int strip = tile / (kStrip * tiles_n), in_strip = tile - strip * kStrip * tiles_n;
    const int high = min(kStrip, tiles_m - strip * kStrip);
    const int m0 = (strip * kStrip + in_strip % high) * BM, n0 = in_strip / high * BN;
    int64_t first;
    int rows;
    share(a, e, s, first, rows);
    rows = __builtin_amdgcn_readfirstlane(rows);
    const int stages = (rows + kStage - 1) / kStage;
    const int sf_row = MX ? a.K / 32 : a.K / 128 * 4;
    // what is loaded next, and the bytes that are left of the share there
    const char* dy = a.dy + first * a.dy_ld;
    const char* x = reinterpret_cast<const char*>(a.x) + first * a.K;
    const char* sf = a.x_sf + first * sf_row;
    int64_t dy_left = rows > 0 ? (rows - 1) * a.dy_ld + a.N * 2 : 0, x_left = (int64_t)rows * a.K,
            sf_left = (int64_t)rows * sf_row;
    int rows_left = rows;

    // The thread's pieces of a stage: offsets from its first row, kOut for columns past the
    // matrix.  A buffer ends with the share's last row, so that rows past it (and kOut) read as
    // zeros.  A piece that holds a row's last columns reads on into the next row (what it gets goes
    // to rows of dw that are none) but in a stage where that would pass the end: there it is
    // loaded one by one.
    constexpr unsigned kOut = 0x80000000u;
    unsigned d_at[kDy], x_at[kX], sf_at[kX];
    int ragged = 0;  // columns of such a piece
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
    const bool cut_edge = a.N % 8 != 0 && m0 + BM > a.N;
    const auto bytes = [](int64_t left) { return (unsigned)min(max(left, INT64_C(0)), INT64_C(0x7FFFFFFF)); };
    struct Regs {
        rows_u32x4 dy[kDy], x[kX];
        uint32_t sf[kX];
    };
    const auto load = [&](Regs& to) {  // the next stage (zeros past the last)
        const auto db = buffer(dy, bytes(dy_left)), xb = buffer(x, bytes(x_left)), sb = buffer(sf, bytes(sf_left));
        if (cut_edge && dy_left < (kStage - 1) * a.dy_ld + 2 * a.N + 14 && ragged) {
#pragma unroll
            for (int p = 0; p < kDy; ++p) {
                const int r = (p * kThreads + (int)threadIdx.x) / (BM / 8);
                uint16_t v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = i < ragged && r < rows_left ? reinterpret_cast<const uint16_t*>(dy + d_at[p])[i] : 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    to.dy[p][i] = v[2 * i] | (uint32_t)v[2 * i + 1] << 16;
            }
        } else {
#pragma unroll
            for (int p = 0; p < kDy; ++p)
                to.dy[p] = __builtin_bit_cast(rows_u32x4, __builtin_amdgcn_raw_buffer_load_b128(db, d_at[p], 0, 0));
        }
#pragma unroll
        for (int p = 0; p < kX; ++p) {
            to.x[p] = __builtin_bit_cast(rows_u32x4, __builtin_amdgcn_raw_buffer_load_b128(xb, x_at[p], 0, 0));
            if constexpr (MX)
                to.sf[p] = __builtin_amdgcn_raw_buffer_load_b8(sb, sf_at[p], 0, 0);
            else
                to.sf[p] = __builtin_amdgcn_raw_buffer_load_b32(sb, sf_at[p], 0, 0);
        }
        dy += kStage * a.dy_ld;
        x += (int64_t)kStage * a.K;
        sf += (int64_t)kStage * sf_row;
        dy_left -= kStage * a.dy_ld;
        x_left -= (int64_t)kStage * a.K;
        sf_left -= (int64_t)kStage * sf_row;
        rows_left -= kStage;
    };

    int d_to[kDy], x_to[kX][2];
#pragma unroll
    for (int p = 0; p < kDy; ++p) {
        const int piece = p * kThreads + threadIdx.x;
        d_to[p] = lds_at<BM>(piece / (BM / 8), piece % (BM / 8) * 8);
    }
#pragma unroll
    for (int p = 0; p < kX; ++p) {
        const int piece = p * kThreads + threadIdx.x;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            x_to[p][h] = kStage * BM * 2 + lds_at<BN>(piece / (BN / 16), x_place(piece % (BN / 16) * 16) + 32 * h);
    }
    const auto store = [&](int buf, const Regs& from) {
#pragma unroll
        for (int p = 0; p < kDy; ++p)
            *(lds_u32x4*)(lds + buf + d_to[p]) = from.dy[p];
#pragma unroll
        for (int p = 0; p < kX; ++p) {
            rows_u32x4 v[2];
            decode16<E, MX>(from.x[p], from.sf[p], v);
            *(lds_u32x4*)(lds + buf + x_to[p][0]) = v[0];
            *(lds_u32x4*)(lds + buf + x_to[p][1]) = v[1];
        }
    };

    int a_at[WM / 32], b_at[WN / 32];
#pragma unroll
    for (int i = 0; i < WM / 32; ++i)
        a_at[i] = frag_at<BM>(wm + i * 32, lane);
#pragma unroll
    for (int j = 0; j < WN / 32; ++j)
        b_at[j] = kStage * BM * 2 + frag_at<BN>(wn + j * 32, lane);
    v16f acc[WM / 32][WN / 32];
    const auto multiply = [&](int buf, int r0, int r1) {
#pragma unroll
        for (int r = r0; r < r1; r += 16) {
            Frag fa[WM / 32], fb[WN / 32];
#pragma unroll
            for (int i = 0; i < WM / 32; ++i)
                fa[i] = read_frag<BM>(lds + buf + a_at[i], r);
#pragma unroll
            for (int j = 0; j < WN / 32; ++j)
                fb[j] = read_frag<BN>(lds + buf + b_at[j], r);
#pragma unroll
            for (int i = 0; i < WM / 32; ++i)
#pragma unroll
                for (int j = 0; j < WN / 32; ++j)
                    acc[i][j] = mfma(E{}, fa[i], fb[j], acc[i][j]);
        }
    };
    // While stage t is multiplied, t + 1, loaded during t - 1, goes from registers to the
    // other buffer, and t + 2 is loaded in its place.
    Regs regs;
    load(regs);
    store(0, regs);
    load(regs);
#pragma unroll
    for (int i = 0; i < WM / 32; ++i)
#pragma unroll
        for (int j = 0; j < WN / 32; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k)
                acc[i][j][k] = 0.f;
    __syncthreads();
    if (stages > 0) {
        int from = 0;
        for (int t = 1; t < stages; ++t) {
            multiply(from, 0, 16);
            store(kBytes - from, regs);  // (here, not after the last product: its latency lies under the rest)
            load(regs);
            multiply(from, 16, kStage);
            from = kBytes - from;
            __syncthreads();
        }
        const int left = rows - (stages - 1) * kStage;  // (of the last stage only the steps that hold rows)
#pragma unroll
        for (int r = 0; r < kStage; r += 16)
            if (r < left)
                multiply(from, r, r + 16);
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

// The kernels: a tile's rows and columns, workgroups that run at a time, and in us a stage of
// 64 rows with one workgroup on the card and with all of them, and a tile's start and results.
// Fitted to a sweep of all three with 1 to 16 shares over 27 sizes, experts equally long: the
// kernel that is chosen, forced as the others are, is within 5 % of the best (called by itself,
// first in each row of the sweep, it took up to 8 % more than the best).  us of the three, each with
// its best number of shares (bf16, UE8M0, to f32):
//   groups x rows in all, n x k   128 x 128    128 x 256    256 x 256
//   1 x 128, 512 x 512             8.6          8.5          9.7
//   1 x 512, 1024 x 1024          10.1         12.5         18.1
//   4 x 8192, 512 x 512           19.0 in 4    20.3 in 6    23.4 in 8     (in one: 28.2, 34.0, 49.8)
//   1 x 8192, 384 x 7168          64.9 in 3    61.6 in 3    66.9 in 4     (in one: 97.5, 120.6, 178.4)
//   1 x 32768, 384 x 7168        226.5 in 3   210.9 in 3   220.7 in 4
//   8 x 4096, 1024 x 1024         17.7         17.5         21.0
//   1 x 2048, 4096 x 4096         89.2         80.2         68.4
//   32 x 4096, 1024 x 2048        56.8         58.8         59.6          (the worst: the last is chosen)
//   1 x 8192, 4096 x 4096        303.6        275.3        231.7
//   32 x 768, 4096 x 2048        215.2        226.8        190.6
struct Kind {
    int bm, bn, slots;
    float alone, busy, fixed;
};
constexpr Kind kKinds[] = {{128, 128, 512, 0.76f, 1.18f, 5.0f},
                           {128, 256, 256, 0.92f, 1.13f, 5.5f},
                           {256, 256, 256, 1.35f, 1.78f, 7.5f}};

template <class E, bool MX>
hipError_t launch(const WgradArgs& a, hipStream_t s)
{
    const Kind& kind = kKinds[a.kind];
    const int tm = (a.N + kind.bm - 1) / kind.bm, tn = (a.K + kind.bn - 1) / kind.bn;
    const int64_t tiles = (int64_t)tm * tn;
    const int64_t wgs = a.E == 1 ? (tiles * a.split + 7) / 8 * 8 : (int64_t)a.E * a.split * ((tiles + 7) / 8 * 8);
    if (wgs >= (INT64_C(1) << 31))
        return hipErrorInvalidValue;
    const auto kernel = a.kind == 0   ? wgrad_tile<E, MX, 128, 128, 64, 64, 64>
                        : a.kind == 1 ? wgrad_tile<E, MX, 128, 256, 64, 64, 64>
                                      : wgrad_tile<E, MX, 256, 256, 128, 64, 64>;
    hipLaunchKernelGGL(kernel, grid_of(wgs), dim3(a.kind == 0 ? 256 : 512), 0, s, a, tm, tn);
    return hipGetLastError();
}

}  // namespace

void wgrad_choose(int groups, int rows, int n, int k, int& kind, int& split)
{
    float least = 0;
    kind = 0;
    split = 1;
    for (int i = 0; i < 3; ++i) {
        const Kind& t = kKinds[i];
        const int64_t tiles = (int64_t)groups * ((n + t.bm - 1) / t.bm) * ((k + t.bn - 1) / t.bn);
        for (int s = 1; s <= kMostSplit; ++s) {
            const int64_t per = ((int64_t)rows / groups + s - 1) / s;
            if (s > 1 && (per < 4 * kShareRows || tiles * (s - 1) >= t.slots))
                break;
            const int64_t full = tiles * s / t.slots, left = tiles * s - full * t.slots;
            const float stages = (float)((per + 63) / 64);
            float us = (float)full * (stages * t.busy + t.fixed);
            if (left > 0)
                us += stages * (t.alone + (t.busy - t.alone) * (float)left / (float)t.slots) + t.fixed;
            if (s > 1)  // the shares' sums written, read and added
                us += 4.f + (float)groups * (float)n * (float)k * 4.f * (2 * s + 1) / 5e6f;
            if (least == 0 || us < least) {
                least = us;
                kind = i;
                split = s;
            }
        }
    }
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
