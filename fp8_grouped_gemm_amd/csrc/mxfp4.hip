// Rows to and from microscaled 4-bit floating point (include/moe_ops.h:
// moe_quantize_mxfp4, moe_dequantize_mxfp4): per 32 columns
//   sf = the smallest power of two >= max(amax, 1e-10) / 6,  q = e2m1(v / sf),
// the library's rule for e2m1 weights (other MX quantisers take 2^(floor(log2 amax) - 2) and
// let values past 6 saturate).  amax / 6 needs no division: with
// amax = 1.m 2^e, the power of two is 2^(e - 2) if 1.m <= 1.5 and
// 2^(e - 1) otherwise.  v / sf is exact (a power of two), so each value
// rounds once, in v_cvt_scalef32_pk_fp4_f32 (nearest, ties to even).
//
// HBM-bound: 65536 x 4096 bf16 takes 126 us (5.4 TB/s), back 137 us (5.0; a large
// copy reaches 5.2).  A thread takes 16 bytes of values -- 8 columns of a 16-bit
// type, 4 of f32 -- and the 4 or 8 threads of a block share its amax by lane
// swaps, so every access of a wave is one contiguous run (f32 with 8 columns a
// thread, two runs of every other 16 bytes: 129 us at 16384 x 4096, nontemporal
// 163).
#include "../../include/moe_ops.h"
#include "ops_internal.h"
#include "rows_device.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

// The maximum over the 4 (or 8) lanes of a block.
template <int LANES>
__device__ __forceinline__ uint32_t block_max(uint32_t v)
{
    v = max(v, row_perm_u<0xB1>(v));  // quad_perm [1,0,3,2]
    v = max(v, row_perm_u<0x4E>(v));  // quad_perm [2,3,0,1]
    if constexpr (LANES == 8)
        v = max(v, row_perm_u<0x141>(v));  // row_half_mirror
    return v;
}

// Threads along a row of n pieces: the smallest power of two that covers it,
// a block's at least, the workgroup at most.
int row_threads(int n)
{
    int t = 8;
    while (t < kThreads && t < n)
        t *= 2;
    return t;
}

// Whether the values stream past the caches (nontemporal): aligned 16-byte
// pieces, and more than the eight L2s hold twice over.  Cached and streamed, us,
// rows of 4096 bf16, other inputs in every call:
//   values   quantise  dequantise  there and back  written, quantised  dequantised, read
//    32 MB   10.8 10.4 13.8  9.8   23 21           22.5 23.1           25 27
//    64 MB   19.3 18.3 23.6 22.3   40 36           40 39               44 48
//   128 MB   35   34   43   42     76 66           72 71               86 89
//   402 MB   98   97  128  124    233 198         240 218             271 264
// A caller that reads the values next pays for small ones, so those stay cached.
bool streams(const MxQuantArgs& a, int size)
{
    return (int64_t)a.rows * a.cols * size > (INT64_C(64) << 20) &&
           (a.ld | (int64_t)reinterpret_cast<uintptr_t>(a.x)) % 16 == 0;
}

}  // namespace

// The thread's row and its first column; false past the matrix (the threads
// of a block leave together: cols % 32 == 0).
template <int VEC>
__device__ __forceinline__ bool place(const MxQuantArgs& a, int tpr, int pieces, int64_t& row, int& col)
{
    const unsigned wg = workgroup(), g = wg / pieces;
    row = (int64_t)g * (kThreads / tpr) + threadIdx.x / tpr;
    col = ((wg - g * pieces) * tpr + threadIdx.x % tpr) * VEC;
    return row < a.rows && col < a.cols;
}

template <class E, bool NT>
__global__ __launch_bounds__(kThreads) void quantize_mxfp4(MxQuantArgs a, int tpr, int pieces)
{
    int64_t row;
    int col;
    if (!place<E::VEC>(a, tpr, pieces, row, col))
        return;
    float v[E::VEC];
    E::unpack(load16<NT>(a.x + row * a.ld + (int64_t)col * E::SIZE), v);
    // the magnitudes' bits order as the magnitudes do, infinity and NaN on top
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < E::VEC; ++i)
        m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = block_max<32 / E::VEC>(m);
    uint32_t code = 0xFFu, q = 0;
    if (m < 0x7F800000u) {
        const uint32_t u = max(m, __float_as_uint(1e-10f));
        code = (u >> 23) - 2 + ((u & 0x7FFFFFu) > 0x400000u);  // 92 .. 253
        const float sf = __uint_as_float(code << 23);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], sf, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], sf, 1);
        if constexpr (E::VEC == 8) {
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], sf, 2);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], sf, 3);
        }
    }
    uint8_t* const to = a.codes + row * (a.cols / 2) + col / 2;
    if constexpr (E::VEC == 8)
        *reinterpret_cast<uint32_t*>(to) = q;
    else
        *reinterpret_cast<uint16_t*>(to) = (uint16_t)q;
    if (col % 32 == 0)
        a.sf[row * (a.cols / 32) + col / 32] = (uint8_t)code;
}

template <class E, bool NT>
__global__ __launch_bounds__(kThreads) void dequantize_mxfp4(MxQuantArgs a, int tpr, int pieces)
{
    int64_t row;
    int col;
    if (!place<E::VEC>(a, tpr, pieces, row, col))
        return;
    const uint8_t* const from = a.codes + row * (a.cols / 2) + col / 2;
    uint32_t q;
    if constexpr (E::VEC == 8)
        q = *reinterpret_cast<const uint32_t*>(from);
    else
        q = *reinterpret_cast<const uint16_t*>(from);
    const uint32_t code = a.sf[row * (a.cols / 32) + col / 32];
    // 2^(code - 127): code 0 is the subnormal 2^-127, 0xFF NaN
    const float sf = __uint_as_float(code == 0 ? 0x400000u : code == 0xFFu ? 0x7FC00000u : code << 23);
    float v[E::VEC];
#pragma unroll
    for (int i = 0; i < E::VEC; ++i) {
        // e2m1 s.ee.m -> f32: exponent ee - 1 + 127 and the mantissa bit on top;
        // ee = 0 holds 0 or 0.5 (m), the latter 2^-1
        const uint32_t n = (q >> (4 * i)) & 15u, mag = n & 7u;
        const uint32_t bits = mag >= 2 ? (126u << 23) + (mag << 22) : mag ? 126u << 23 : 0u;
        // the sign goes on after the scale: a product folded into the f16
        // conversion as a fused multiply-add of +0 would lose that of -0
        v[i] = __uint_as_float(__float_as_uint(__uint_as_float(bits) * sf) | ((n & 8u) << 28));
    }
    store16<NT>(a.x + row * a.ld + (int64_t)col * E::SIZE, E::pack(v));
}

namespace {

template <class E>
hipError_t launch(const MxQuantArgs& a, bool back, hipStream_t s)
{
    const int n = a.cols / E::VEC, tpr = row_threads(n), per = kThreads / tpr;
    const int pieces = (n + tpr - 1) / tpr;
    const int64_t wgs = ((int64_t)a.rows + per - 1) / per * pieces;
    if (wgs >= (INT64_C(1) << 31))
        return hipErrorInvalidValue;
    const bool nt = streams(a, E::SIZE);
    const auto kernel = back ? (nt ? dequantize_mxfp4<E, true> : dequantize_mxfp4<E, false>)
                             : (nt ? quantize_mxfp4<E, true> : quantize_mxfp4<E, false>);
    hipLaunchKernelGGL(kernel, grid_of(wgs), dim3(kThreads), 0, s, a, tpr, pieces);
    return hipGetLastError();
}

hipError_t launch_type(const MxQuantArgs& a, bool back, hipStream_t s)
{
    switch (a.dtype) {
    case MOE_DTYPE_BF16: return launch<Bf16>(a, back, s);
    case MOE_DTYPE_F16: return launch<F16>(a, back, s);
    case MOE_DTYPE_F32: return launch<F32>(a, back, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_quantize_mxfp4(const MxQuantArgs& a, hipStream_t s) { return launch_type(a, false, s); }

hipError_t launch_dequantize_mxfp4(const MxQuantArgs& a, hipStream_t s) { return launch_type(a, true, s); }

}  // namespace moe
