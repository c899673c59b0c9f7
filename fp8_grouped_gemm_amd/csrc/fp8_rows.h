// 8-bit rows (e4m3 codes with a scale per block of columns) in the formats and by
// the rule of moe_quantize_act, eight columns per thread: 16 threads share a
// block of 128 columns, 4 one of 32.
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
    v = max(v, row_perm_u<0xB1>(v));  // quad_perm [1,0,3,2]
    v = max(v, row_perm_u<0x4E>(v));  // quad_perm [2,3,0,1]
    if constexpr (!MX) {
        v = max(v, row_perm_u<0x141>(v));  // row_half_mirror
        v = max(v, row_perm_u<0x140>(v));  // row_mirror
    }
    return __uint_as_float(v);
}

// Quantises the eight columns at `col` of a row of `cols`, whose first code and scale are
// at codes and sf.
template <bool MX>
__device__ __forceinline__ void store_codes(const float* f, int col, uint8_t* codes, char* sf)
{
    float rsf;
    const float s = requant_sf(block_amax<MX>(f), MX, rsf);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q[i] = requant_q2(f[2 * i], f[2 * i + 1], s, rsf, MX);
    *reinterpret_cast<uint2*>(codes + col) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
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

// The values of eight codes.
__device__ __forceinline__ void decode8(uint2 q, float scale, float* f)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, true);
    const f2 c = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, false), d = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, true);
    f[0] = a[0] * scale; f[1] = a[1] * scale; f[2] = b[0] * scale; f[3] = b[1] * scale;
    f[4] = c[0] * scale; f[5] = c[1] * scale; f[6] = d[0] * scale; f[7] = d[1] * scale;
}

}  // namespace moe
