// Element types and 16-byte accesses of the row operators' kernels.
#pragma once

#include "moe_device.h"

namespace moe {

typedef unsigned int rows_u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes at any byte address: gfx950 global accesses need no alignment, so
// rows of odd width take the same wide accesses as aligned ones.
typedef unsigned int bytes16 __attribute__((ext_vector_type(4), aligned(1)));

template <bool NT = false>
__device__ __forceinline__ rows_u32x4 load16(const char* p)
{
    if constexpr (NT)
        return __builtin_nontemporal_load(reinterpret_cast<const bytes16*>(p));
    return *reinterpret_cast<const bytes16*>(p);
}

template <bool NT = false>
__device__ __forceinline__ void store16(char* p, rows_u32x4 v)
{
    if constexpr (NT)
        __builtin_nontemporal_store((bytes16)v, reinterpret_cast<bytes16*>(p));
    else
        *reinterpret_cast<bytes16*>(p) = v;
}

// An element type: its size, how many fit 16 bytes, and the conversions
// (f32 -> 16 bits rounds to nearest even, once).
struct Bf16 {
    static constexpr int SIZE = 2, VEC = 8;
    static __device__ __forceinline__ void unpack(rows_u32x4 r, float* f)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_to_f32(r[i] & 0xFFFFu);
            f[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ rows_u32x4 pack(const float* f)
    {
        rows_u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = f32x2_to_bf16x2(f[2 * i], f[2 * i + 1]);
        return r;
    }
    static __device__ __forceinline__ uint32_t pack2(float a, float b) { return f32x2_to_bf16x2(a, b); }
    static __device__ __forceinline__ float load(const char* p)
    {
        return bf16_to_f32(*reinterpret_cast<const uint16_t*>(p));
    }
    static __device__ __forceinline__ void store(char* p, float v)
    {
        *reinterpret_cast<uint16_t*>(p) = f32_to_bf16(v);
    }
};

struct F16 {
    static constexpr int SIZE = 2, VEC = 8;
    static __device__ __forceinline__ uint32_t bits(float v)
    {
        return __builtin_bit_cast(uint16_t, (_Float16)v);
    }
    static __device__ __forceinline__ float value(uint32_t b)
    {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
    }
    static __device__ __forceinline__ void unpack(rows_u32x4 r, float* f)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = value(r[i] & 0xFFFFu);
            f[2 * i + 1] = value(r[i] >> 16);
        }
    }
    static __device__ __forceinline__ rows_u32x4 pack(const float* f)
    {
        rows_u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = bits(f[2 * i]) | (bits(f[2 * i + 1]) << 16);
        return r;
    }
    static __device__ __forceinline__ uint32_t pack2(float a, float b) { return bits(a) | bits(b) << 16; }
    static __device__ __forceinline__ float load(const char* p)
    {
        return value(*reinterpret_cast<const uint16_t*>(p));
    }
    static __device__ __forceinline__ void store(char* p, float v)
    {
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)bits(v);
    }
};

struct F32 {
    static constexpr int SIZE = 4, VEC = 4;
    static __device__ __forceinline__ void unpack(rows_u32x4 r, float* f)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = __uint_as_float(r[i]);
    }
    static __device__ __forceinline__ rows_u32x4 pack(const float* f)
    {
        rows_u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = __float_as_uint(f[i]);
        return r;
    }
    static __device__ __forceinline__ float load(const char* p)
    {
        return *reinterpret_cast<const float*>(p);
    }
    static __device__ __forceinline__ void store(char* p, float v)
    {
        *reinterpret_cast<float*>(p) = v;
    }
};

// The n <= VEC elements of one vector at p (n < VEC: a row's last ones).
template <class T, bool NT = false>
__device__ __forceinline__ void load_vec(const char* p, int n, float* f)
{
    if (n >= T::VEC) {
        T::unpack(load16<NT>(p), f);
    } else {
#pragma unroll
        for (int i = 0; i < T::VEC; ++i)
            f[i] = i < n ? T::load(p + i * T::SIZE) : 0.f;
    }
}

template <class T, bool NT = false>
__device__ __forceinline__ void store_vec(char* p, int n, const float* f)
{
    if (n >= T::VEC) {
        store16<NT>(p, T::pack(f));
    } else {
#pragma unroll
        for (int i = 0; i < T::VEC; ++i)
            if (i < n)
                T::store(p + i * T::SIZE, f[i]);
    }
}

}  // namespace moe
