// Rows to and from microscaled 4-bit floating point (include/moe_ops.h:
// moe_quantize_mxfp4, moe_dequantize_mxfp4): per 32 columns
//   sf = the smallest power of two >= max(amax, 1e-10) / 6,  q = e2m1(v / sf),
// the library's rule for e2m1 weights.  amax / 6 needs no division: with
// amax = 1.m 2^e, the power of two is 2^(e - 2) if 1.m <= 1.5 and
// 2^(e - 1) otherwise.  v / sf is exact (a power of two), so each value
// rounds once, in v_cvt_scalef32_pk_fp4_f32 (nearest, ties to even).
//
// HBM-bound.  A thread takes 8 columns (16 bytes of a 16-bit type), the four
// threads of a block share its amax by two DPP swaps, and codes leave as 4
// bytes per thread: every access of a wave is one contiguous run.
#include "../../include/moe_ops.h"
#include "ops_internal.h"
#include "rows_device.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

// v of the lane with bit 0 (then bit 1) of its index flipped.
__device__ __forceinline__ uint32_t max_of_4(uint32_t v)
{
    v = max(v, row_perm_u<0xB1>(v));  // quad_perm [1,0,3,2]
    v = max(v, row_perm_u<0x4E>(v));  // quad_perm [2,3,0,1]
    return v;
}

template <class E>
__device__ __forceinline__ void load8(const char* p, float* f)
{
    E::unpack(load16(p), f);
    if constexpr (E::VEC == 4)
        E::unpack(load16(p + 16), f + 4);
}

template <class E>
__device__ __forceinline__ void store8(char* p, const float* f)
{
    store16(p, E::pack(f));
    if constexpr (E::VEC == 4)
        store16(p + 16, E::pack(f + 4));
}

// Threads along a row of n 8-column pieces (n a multiple of 4): the smallest
// power of two that covers it, at most the workgroup.
int row_threads(int n)
{
    int t = 4;
    while (t < kThreads && t < n)
        t *= 2;
    return t;
}

}  // namespace

template <class E>
__global__ __launch_bounds__(kThreads) void quantize_mxfp4(MxQuantArgs a, int tpr, int pieces)
{
    const unsigned g = blockIdx.x / pieces;
    const int64_t row = (int64_t)g * (kThreads / tpr) + threadIdx.x / tpr;
    const int c = (blockIdx.x - g * pieces) * tpr + threadIdx.x % tpr;  // 8-column piece
    // (the four threads of a block leave together: cols % 32 == 0)
    if (row >= a.rows || c * 8 >= a.cols)
        return;
    float v[8];
    load8<E>(a.x + row * a.ld + (int64_t)c * 8 * E::SIZE, v);
    // the magnitudes' bits order as the magnitudes do, infinity and NaN on top
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    m = max_of_4(m);
    uint32_t code = 0xFFu, q = 0;
    if (m < 0x7F800000u) {
        const uint32_t u = max(m, __float_as_uint(1e-10f));
        code = (u >> 23) - 2 + ((u & 0x7FFFFFu) > 0x400000u);  // 91 .. 253
        const float sf = __uint_as_float(code << 23);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], sf, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], sf, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], sf, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], sf, 3);
    }
    *reinterpret_cast<uint32_t*>(a.codes + row * (a.cols / 2) + c * 4) = q;
    if ((c & 3) == 0)
        a.sf[row * (a.cols / 32) + c / 4] = (uint8_t)code;
}

template <class E>
__global__ __launch_bounds__(kThreads) void dequantize_mxfp4(MxQuantArgs a, int tpr, int pieces)
{
    const unsigned g = blockIdx.x / pieces;
    const int64_t row = (int64_t)g * (kThreads / tpr) + threadIdx.x / tpr;
    const int c = (blockIdx.x - g * pieces) * tpr + threadIdx.x % tpr;
    if (row >= a.rows || c * 8 >= a.cols)
        return;
    const uint32_t q = *reinterpret_cast<const uint32_t*>(a.codes + row * (a.cols / 2) + c * 4);
    const uint32_t code = a.sf[row * (a.cols / 32) + c / 4];
    // 2^(code - 127): code 0 is the subnormal 2^-127, 0xFF NaN
    const float sf = __uint_as_float(code == 0 ? 0x400000u : code == 0xFFu ? 0x7FC00000u : code << 23);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // e2m1 s.ee.m -> f32: exponent ee - 1 + 127 and the mantissa bit on top;
        // ee = 0 holds 0 or 0.5 (m), the latter 2^-1
        const uint32_t n = (q >> (4 * i)) & 15u, mag = n & 7u;
        const uint32_t bits = mag >= 2 ? (126u << 23) + (mag << 22) : mag ? 126u << 23 : 0u;
        // the sign goes on after the scale: a product folded into the f16
        // conversion as a fused multiply-add of +0 would lose that of -0
        v[i] = __uint_as_float(__float_as_uint(__uint_as_float(bits) * sf) | ((n & 8u) << 28));
    }
    store8<E>(a.x + row * a.ld + (int64_t)c * 8 * E::SIZE, v);
}

template <class F>
static hipError_t launch_rows(const MxQuantArgs& a, F launch)
{
    const int n = a.cols / 8, tpr = row_threads(n), per = kThreads / tpr;
    const int pieces = (n + tpr - 1) / tpr;
    const int64_t wgs = ((int64_t)a.rows + per - 1) / per * pieces;
    if (wgs >= (INT64_C(1) << 31))
        return hipErrorInvalidValue;
    launch(dim3((unsigned)wgs), tpr, pieces);
    return hipGetLastError();
}

hipError_t launch_quantize_mxfp4(const MxQuantArgs& a, hipStream_t s)
{
    return launch_rows(a, [&](dim3 grid, int tpr, int pieces) {
        if (a.dtype == MOE_DTYPE_BF16)
            hipLaunchKernelGGL(quantize_mxfp4<Bf16>, grid, dim3(kThreads), 0, s, a, tpr, pieces);
        else if (a.dtype == MOE_DTYPE_F16)
            hipLaunchKernelGGL(quantize_mxfp4<F16>, grid, dim3(kThreads), 0, s, a, tpr, pieces);
        else
            hipLaunchKernelGGL(quantize_mxfp4<F32>, grid, dim3(kThreads), 0, s, a, tpr, pieces);
    });
}

hipError_t launch_dequantize_mxfp4(const MxQuantArgs& a, hipStream_t s)
{
    return launch_rows(a, [&](dim3 grid, int tpr, int pieces) {
        if (a.dtype == MOE_DTYPE_BF16)
            hipLaunchKernelGGL(dequantize_mxfp4<Bf16>, grid, dim3(kThreads), 0, s, a, tpr, pieces);
        else if (a.dtype == MOE_DTYPE_F16)
            hipLaunchKernelGGL(dequantize_mxfp4<F16>, grid, dim3(kThreads), 0, s, a, tpr, pieces);
        else
            hipLaunchKernelGGL(dequantize_mxfp4<F32>, grid, dim3(kThreads), 0, s, a, tpr, pieces);
    });
}

}  // namespace moe
