// 8-bit rows (e4m3 codes with a scale per block of columns) in the formats and by
// the rule of moe_quantize_act, eight columns per thread: 16 threads share a
// block of 128 columns, 4 one of 32.  Where bytes bound the kernels around them these take no
// time of their own (a large moe_swiglu: 144 us; with a division for each value, and expf, 189).
#pragma once

#include "../../include/moe_ops.h"
#include "rows_device.h"

namespace moe {

// The n <= 8 elements at p (fewer: a row's last ones, the others 0).
template <class T>
__device__ __forceinline__ void load8(const char* p, int n, float* f)
{
    if constexpr (T::VEC == 8) {
        load_vec<T>(p, n, f);
    } else {
        load_vec<T>(p, n, f);
        load_vec<T>(p + 16, n - 4, f + 4);
    }
}

template <class T>
__device__ __forceinline__ void store8(char* p, int n, const float* f)
{
    if constexpr (T::VEC == 8) {
        store_vec<T>(p, n, f);
    } else {
        store_vec<T>(p, n, f);
        store_vec<T>(p + 16, n - 4, f + 4);
    }
}

// Eight elements as they lie in memory, for loads that are used later.
template <class T>
struct Raw8 {
    rows_u32x4 r[T::SIZE / 2];
};

template <class T>
__device__ __forceinline__ Raw8<T> load_raw8(const char* p, int n)
{
    Raw8<T> v;
    if (n >= 8) {
#pragma unroll
        for (int i = 0; i < T::SIZE / 2; ++i)
            v.r[i] = load16(p + 16 * i);
    } else {
        float f[8];
        load8<T>(p, n, f);
#pragma unroll
        for (int i = 0; i < T::SIZE / 2; ++i)
            v.r[i] = T::pack(f + i * T::VEC);
    }
    return v;
}

template <class T>
__device__ __forceinline__ void unpack8(const Raw8<T>& v, float* f)
{
#pragma unroll
    for (int i = 0; i < T::SIZE / 2; ++i)
        T::unpack(v.r[i], f + i * T::VEC);
}

// Rounded to the type and back.
template <class T>
__device__ __forceinline__ void round8(float* f)
{
    if constexpr (T::VEC == 8)
        T::unpack(T::pack(f), f);
}

// v from another lane of the 16-lane row, in a form that the compiler folds into the
// instruction that takes it.
template <int CTRL>
__device__ __forceinline__ uint32_t block_swap(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// The largest of the magnitudes of the block's threads (all of them active); a NaN is
// passed over, as by fmaxf.
template <bool MX>
__device__ __forceinline__ float block_amax(const float* f)
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = fmaxf(m, fabsf(f[i]));
    uint32_t v = __float_as_uint(m);
    v = max(v, block_swap<0xB1>(v));  // quad_perm [1,0,3,2]
    v = max(v, block_swap<0x4E>(v));  // quad_perm [2,3,0,1]
    if constexpr (!MX) {
        v = max(v, block_swap<0x141>(v));  // row_half_mirror
        v = max(v, block_swap<0x140>(v));  // row_mirror
    }
    return __uint_as_float(v);
}

// Four values' codes.  The rule is requant_q's (moe_device.h).  A block's finite values stay
// within 448 of its scale, so that nothing has to saturate: with a power of two the
// converter divides by itself (equal to requant_q for every f32 within 464 scales), and
// otherwise the two ends of the quotient's bracket are converted as they are.
template <bool MX>
__device__ __forceinline__ uint32_t quant4(const float* f, float s, float rsf)
{
    if constexpr (MX) {
        typedef short s2 __attribute__((ext_vector_type(2)));
        s2 q = {0, 0};
        q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, f[0], f[1], s, false);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, f[2], f[3], s, true);
        return __builtin_bit_cast(uint32_t, q);
    } else {
        int lo = 0, hi = 0;
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = f[i] * rsf;
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * (1.0f - 0x1p-20f), y[1] * (1.0f - 0x1p-20f), lo, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * (1.0f - 0x1p-20f), y[3] * (1.0f - 0x1p-20f), lo, true);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * (1.0f + 0x1p-20f), y[1] * (1.0f + 0x1p-20f), hi, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * (1.0f + 0x1p-20f), y[3] * (1.0f + 0x1p-20f), hi, true);
        if (lo == hi)
            return (uint32_t)lo;
        return requant_q2(f[0], f[1], s, rsf, false) | requant_q2(f[2], f[3], s, rsf, false) << 16;
    }
}

// Quantises the eight columns at `col` of a row of `cols`, whose first code and scale are
// at codes and sf.
template <bool MX>
__device__ __forceinline__ void store_codes(const float* f, int col, uint8_t* codes, char* sf)
{
    float rsf;
    const float amax = block_amax<MX>(f), s = requant_sf(amax, MX, rsf);
    uint32_t q[2];
    const bool odd = f[0] != f[0] || f[1] != f[1] || f[2] != f[2] || f[3] != f[3] || f[4] != f[4] || f[5] != f[5] ||
                     f[6] != f[6] || f[7] != f[7] || amax == INFINITY;
    if (odd) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            q[i] = requant_q2(f[4 * i], f[4 * i + 1], s, rsf, MX) | requant_q2(f[4 * i + 2], f[4 * i + 3], s, rsf, MX) << 16;
    } else {
        q[0] = quant4<MX>(f, s, rsf);
        q[1] = quant4<MX>(f + 4, s, rsf);
    }
    *reinterpret_cast<uint2*>(codes + col) = make_uint2(q[0], q[1]);
    if constexpr (MX) {
        if (col % 32 == 0)
            sf[col / 32] = (char)(__float_as_uint(s) >> 23);
    } else {
        if (col % 128 == 0)
            reinterpret_cast<float*>(sf)[col / 128] = s;
    }
}

// The scale of the block that holds column `col` (code 0xFF: NaN).
template <bool MX>
__device__ __forceinline__ float read_scale(const char* sf, int col)
{
    if constexpr (MX) {
        const uint32_t c = (uint8_t)sf[col / 32];
        return __uint_as_float(c == 0 ? 0x400000u : c == 0xFFu ? 0x7FC00000u : c << 23);
    }
    return reinterpret_cast<const float*>(sf)[col / 128];
}

// The values of eight codes (with a power of two the converter multiplies by itself, as the
// product would round for every code and scale code).
template <bool MX>
__device__ __forceinline__ void decode8(uint2 q, float scale, float* f)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    f2 v[4];
    if constexpr (MX) {
        v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)q.x, scale, false);
        v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)q.x, scale, true);
        v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)q.y, scale, false);
        v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)q.y, scale, true);
    } else {
        v[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, false);
        v[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, true);
        v[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, false);
        v[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, true);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = MX ? v[i / 2][i % 2] : v[i / 2][i % 2] * scale;
}

}  // namespace moe
