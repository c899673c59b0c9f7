// The activation between the experts' products and its gradient (include/moe_ops.h:
// moe_swiglu, moe_swiglu_bwd).
//   h = g sg u,  sg = 1 / (1 + exp(-g));  dg = dh u sg (1 + g (1 - sg)),  du = dh g sg
// with g and u clamped first, and no gradient where they were.
//
// One thread takes eight columns of g and the same of u, and writes what the call asks
// for: h, h in 8 bits, and gate and up in 8 bits, which the gradient reads in place of
// the input.  Rows that hold no slot are passed over.
//
// Bytes bound both: 49152 rows of 2 x 2048 bf16 in 256 segments to h and gate and up in 8
// bits 144 us, 4.9 TB/s, and their gradient from the 8-bit copy 159, 5.1 TB/s (with expf and
// requant_q's own division 189 and 175: instructions).
#include "../../include/moe_ops.h"
#include "fp8_rows.h"
#include "ops_internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

// Threads along a row of n steps of eight columns: the smallest power of two that
// covers it, a block's at least, the workgroup at most.
int row_threads(int n)
{
    int t = 16;
    while (t < kThreads && t < n)
        t *= 2;
    return t;
}

// The thread's row and its first column; false where there is nothing to do.
__device__ __forceinline__ bool place(const SwigluArgs& a, int tpr, int pieces, int64_t& row, int& col)
{
    const unsigned wg = workgroup(), g = wg / pieces;
    row = (int64_t)g * (kThreads / tpr) + threadIdx.x / tpr;
    col = ((wg - g * pieces) * tpr + threadIdx.x % tpr) * 8;
    const int used = a.used ? min(*a.used, a.R) : a.R;
    return row < used && col < a.inner && (!a.row_src || a.row_src[row] >= 0);
}

// sg = 1 / (1 + exp(-g)) and 1 - sg of an element of type E.  With e = exp(-|g|) and
// r = 1 / (1 + e) they are r and e r (g < 0: the other way round): neither overflows
// nor cancels.  16-bit types take e from the hardware's 2^x: off by 1.25 |g| + 2 roundings of
// f32 at most (the product's, a quarter of log2 e, and its own), of which 2^15 to 2^16 make half a step
// of bf16, 2^12 to 2^13 one of f16 and 2^19 one of e4m3, and zero below 2^-126.  With the part that the
// product loses put back the large calls take 149 - 152 us for 143 and 167 for 158.
template <class E>
__device__ __forceinline__ void sigmoid(float g, float& sg, float& rest)
{
    const float e = E::SIZE == 4 ? expf(-fabsf(g)) : __builtin_amdgcn_exp2f(-1.44269504088896341f * fabsf(g));
    const float r = __builtin_amdgcn_rcpf(1.f + e), er = e * r;
    sg = g < 0.f ? er : r;
    rest = g < 0.f ? r : er;
}

// (NaN stays)
__device__ __forceinline__ float clamped(float v, float c) { return v > c ? c : v < -c ? -c : v; }

template <bool MX>
__device__ __forceinline__ void keep(const float* f, int64_t row, int cols, int col, uint8_t* codes, void* sf)
{
    const int64_t row_bytes = MX ? cols / 32 : cols / 128 * 4;
    store_codes<MX>(f, col, codes + row * cols, static_cast<char*>(sf) + row * row_bytes);
}

}  // namespace

template <class E>
__global__ __launch_bounds__(kThreads) void swiglu_rows(SwigluArgs a, int tpr, int pieces)
{
    int64_t row;
    int col;
    if (!place(a, tpr, pieces, row, col))
        return;
    const int n = a.inner - col;
    const char* const gu = a.gu + row * a.gu_ld + (int64_t)col * E::SIZE;
    float g[8], u[8];
    load8<E>(gu, n, g);
    load8<E>(gu + (int64_t)a.inner * E::SIZE, n, u);
    const bool mx = a.sf_format == MOE_SF_UE8M0_32;
    if (a.gu_codes) {
        if (mx) {
            keep<true>(g, row, 2 * a.inner, col, a.gu_codes, a.gu_sf);
            keep<true>(u, row, 2 * a.inner, a.inner + col, a.gu_codes, a.gu_sf);
        } else {
            keep<false>(g, row, 2 * a.inner, col, a.gu_codes, a.gu_sf);
            keep<false>(u, row, 2 * a.inner, a.inner + col, a.gu_codes, a.gu_sf);
        }
    }
    if (!a.h && !a.h_codes)
        return;
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (a.clamp > 0.f) {
            g[i] = clamped(g[i], a.clamp);
            u[i] = clamped(u[i], a.clamp);
        }
        float sg, rest;
        sigmoid<E>(g[i], sg, rest);
        h[i] = g[i] * sg * u[i];
    }
    if (a.h)
        store8<E>(a.h + row * a.h_ld + (int64_t)col * E::SIZE, n, h);
    if (a.h_codes) {
        if (mx)
            keep<true>(h, row, a.inner, col, a.h_codes, a.h_sf);
        else
            keep<false>(h, row, a.inner, col, a.h_codes, a.h_sf);
    }
}

// FROM: the input's rows, or the format of its 8-bit copy.
enum From { ROWS, CODES_F32, CODES_MX };

template <class E, From FROM>
__global__ __launch_bounds__(kThreads) void swiglu_grad(SwigluArgs a, int tpr, int pieces)
{
    int64_t row;
    int col;
    if (!place(a, tpr, pieces, row, col))
        return;
    const int n = a.inner - col;
    float g[8], u[8], dh[8];
    load8<E>(a.h + row * a.h_ld + (int64_t)col * E::SIZE, n, dh);
    if constexpr (FROM == ROWS) {
        const char* const gu = a.gu + row * a.gu_ld + (int64_t)col * E::SIZE;
        load8<E>(gu, n, g);
        load8<E>(gu + (int64_t)a.inner * E::SIZE, n, u);
    } else {
        constexpr bool MX = FROM == CODES_MX;
        const int64_t cols = 2 * (int64_t)a.inner, row_bytes = MX ? cols / 32 : cols / 128 * 4;
        const uint8_t* const codes = a.gu_codes + row * cols + col;
        const char* const sf = static_cast<const char*>(a.gu_sf) + row * row_bytes;
        decode8<MX>(*reinterpret_cast<const uint2*>(codes), read_scale<MX>(sf, col), g);
        decode8<MX>(*reinterpret_cast<const uint2*>(codes + a.inner), read_scale<MX>(sf, a.inner + col), u);
    }
    float dg[8], du[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool cg = a.clamp > 0.f && (g[i] > a.clamp || g[i] < -a.clamp);
        const bool cu = a.clamp > 0.f && (u[i] > a.clamp || u[i] < -a.clamp);
        const float gc = cg ? clamped(g[i], a.clamp) : g[i], uc = cu ? clamped(u[i], a.clamp) : u[i];
        float sg, rest;
        sigmoid<E>(gc, sg, rest);
        dg[i] = cg ? 0.f : dh[i] * uc * (sg * __builtin_fmaf(gc, rest, 1.f));
        du[i] = cu ? 0.f : dh[i] * (gc * sg);
    }
    char* const out = a.dgu + row * a.dgu_ld + (int64_t)col * E::SIZE;
    store8<E>(out, n, dg);
    store8<E>(out + (int64_t)a.inner * E::SIZE, n, du);
}

// ------------------------------------------------------------ launchers

namespace {

template <class E>
hipError_t launch(const SwigluArgs& a, bool back, hipStream_t s)
{
    const int n = (a.inner + 7) / 8, tpr = row_threads(n), per = kThreads / tpr;
    const int pieces = (n + tpr - 1) / tpr;
    const int64_t wgs = ((int64_t)a.R + per - 1) / per * pieces;
    if (wgs >= (INT64_C(1) << 31))
        return hipErrorInvalidValue;
    const auto kernel = !back   ? swiglu_rows<E>
                        : a.gu  ? swiglu_grad<E, ROWS>
                        : a.sf_format == MOE_SF_UE8M0_32 ? swiglu_grad<E, CODES_MX> : swiglu_grad<E, CODES_F32>;
    hipLaunchKernelGGL(kernel, grid_of(wgs), dim3(kThreads), 0, s, a, tpr, pieces);
    return hipGetLastError();
}

hipError_t launch_type(const SwigluArgs& a, bool back, hipStream_t s)
{
    switch (a.dtype) {
    case MOE_DTYPE_BF16: return launch<Bf16>(a, back, s);
    case MOE_DTYPE_F16: return launch<F16>(a, back, s);
    case MOE_DTYPE_F32: return launch<F32>(a, back, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s) { return launch_type(a, false, s); }

hipError_t launch_swiglu_bwd(const SwigluArgs& a, hipStream_t s) { return launch_type(a, true, s); }

}  // namespace moe
