// Residual and root-mean-square norm of token rows, and the gradients
// (include/moe_ops.h: moe_rms_norm, moe_rms_norm_bwd).
//   z = round(x + residual),  rstd = (mean(z^2) + eps)^(-1/2),  y = z rstd w
//   xh = z rstd,  g = dy w:  dx = rstd (g - xh mean(g xh)) + dz,  dw = sum over rows of dy xh
//
// Both move bytes: a row is read once and stays in registers between its sum and
// its result (rows over kMaxResident columns are read a second time), eight columns
// a thread and step, and y is quantised from the registers, where a block's threads
// share its largest magnitude by lane swaps.  dw needs sums over rows: a workgroup
// walks many rows with its columns' sums in registers, writes them to the workspace
// once, and a second kernel adds those partial rows in a fixed order (no atomics).
//
// 8192 x 7168 bf16 with a residual to z, y and codes: 93 us, 5.7 TB/s (a copy: 5.0).  The gradient
// of 8192 x 4096 with dz, to dx and dw: 56 us in all, 44 + 5 in the two kernels; with 256
// threads a workgroup and more partial rows 94.
#include "../../include/moe_ops.h"
#include "fp8_rows.h"
#include "ops_internal.h"

namespace moe {

namespace {

constexpr int kMaxResident = 16384;
constexpr int kPartials = 256;       // most partial rows of dw
constexpr int kColumnThreads = 256;

// The sum over LANES lanes of a wave, in each of them.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v)
{
    const auto add = [&](uint32_t other) { v += __uint_as_float(other); };
    add(block_swap<0xB1>(__float_as_uint(v)));   // quad_perm [1,0,3,2]
    add(block_swap<0x4E>(__float_as_uint(v)));   // quad_perm [2,3,0,1]
    add(block_swap<0x141>(__float_as_uint(v)));  // row_half_mirror
    if constexpr (LANES > 8)
        add(block_swap<0x140>(__float_as_uint(v)));  // row_mirror
#pragma unroll
    for (int x = 16; x < LANES; x *= 2)
        v += __shfl_xor(v, x);
    return v;
}

// The sum over the TPR threads of a row; `red` (one per wave) is not written again before
// every thread has passed another barrier.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red)
{
    v = lanes_sum<TPR < 64 ? TPR : 64>(v);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i)
            v += red[threadIdx.x / TPR * (TPR / 64) + i];
    }
    return v;
}

template <class W>
__device__ __forceinline__ void load_weight(const char* w, int col, int n, float* f)
{
    if (w) {
        load8<W>(w + (int64_t)col * W::SIZE, n, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = 1.f;
    }
}

// z of eight columns: x, or the rounded sum with the residual.
template <class E>
__device__ __forceinline__ void load_z(const NormArgs& a, int64_t row, int col, int n, float* z)
{
    load8<E>(a.x + row * a.x_ld + (int64_t)col * E::SIZE, n, z);
    if (a.res) {
        float r[8];
        load8<E>(a.res + row * a.res_ld + (int64_t)col * E::SIZE, n, r);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] += r[i];
        round8<E>(z);
    }
}

// y of eight columns from z, to the outputs the call asks for.
template <class E, class W>
__device__ __forceinline__ void finish(const NormArgs& a, int64_t row, int col, int n, float rstd, float* z)
{
    if (n <= 0)
        return;
    float w[8];
    load_weight<W>(a.weight, col, n, w);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        z[i] = z[i] * rstd * w[i];
    if (a.y)
        store8<E>(a.y + row * a.y_ld + (int64_t)col * E::SIZE, n, z);
    if (a.codes) {
        uint8_t* const codes = a.codes + row * a.width;
        if (a.sf_format == MOE_SF_UE8M0_32)
            store_codes<true>(z, col, codes, static_cast<char*>(a.sf) + row * (a.width / 32));
        else
            store_codes<false>(z, col, codes, static_cast<char*>(a.sf) + row * (a.width / 128) * 4);
    }
}

__device__ __forceinline__ float rstd_of(float sum, const NormArgs& a)
{
    return 1.f / sqrtf(sum / (float)a.width + a.eps);
}

constexpr int threads_of(int tpr) { return tpr < 256 ? 256 : tpr; }

constexpr int kGradThreads = 1024;

// Threads along a row of a width that fits the registers: of a narrow one a part of a wave
// (524288 x 128 bf16: 107 us, the gradient 106; with a wave a row 275 and 228).
constexpr int row_threads(int width)
{
    return width <= 64 ? 8 : width <= 128 ? 16 : width <= 256 ? 32 : width <= 1024 ? 64 : width <= 4096 ? 256
         : width <= 8192 ? 512 : 1024;
}

}  // namespace

// TPR threads per row, each with CH steps of eight columns.
template <class E, class W, int TPR, int CH>
__global__ __launch_bounds__(threads_of(TPR)) void norm_rows(NormArgs a)
{
    __shared__ float red[16];
    const int at = threadIdx.x % TPR;
    const int64_t row = (int64_t)workgroup() * (threads_of(TPR) / TPR) + threadIdx.x / TPR;
    if (row >= a.rows)
        return;
    float z[CH][8], sum = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * TPR + at) * 8;
        load_z<E>(a, row, col, a.width - col, z[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * TPR + at) * 8;
        if (a.z)
            store8<E>(a.z + row * a.z_ld + (int64_t)col * E::SIZE, a.width - col, z[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum = __builtin_fmaf(z[c][i], z[c][i], sum);
    }
    const float rstd = rstd_of(row_sum<TPR>(sum, red), a);
    if (a.rstd && at == 0)
        a.rstd[row] = rstd;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * TPR + at) * 8;
        finish<E, W>(a, row, col, a.width - col, rstd, z[c]);
    }
}

// Rows that do not fit the registers: read again for the result.
template <class E, class W>
__global__ __launch_bounds__(1024) void norm_rows_wide(NormArgs a)
{
    __shared__ float red[16];
    const int64_t row = workgroup();
    if (row >= a.rows)
        return;
    float sum = 0.f;
    for (int col = threadIdx.x * 8; col < a.width; col += 1024 * 8) {
        const int n = a.width - col;
        float z[8];
        load_z<E>(a, row, col, n, z);
        if (a.z)
            store8<E>(a.z + row * a.z_ld + (int64_t)col * E::SIZE, n, z);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum = __builtin_fmaf(z[i], z[i], sum);
    }
    const float rstd = rstd_of(row_sum<1024>(sum, red), a);
    if (a.rstd && threadIdx.x == 0)
        a.rstd[row] = rstd;
    for (int col = threadIdx.x * 8; col < a.width; col += 1024 * 8) {
        const int n = a.width - col;
        float z[8];
        if (a.z)  // (x or the residual may be gone: z may stand on it)
            load8<E>(a.z + row * a.z_ld + (int64_t)col * E::SIZE, n, z);
        else
            load_z<E>(a, row, col, n, z);
        finish<E, W>(a, row, col, n, rstd, z);
    }
}

// dx of a row whose mean of g xh is known, eight columns; d: what reaches z on its other way.
template <class E>
__device__ __forceinline__ void store_dx(const NormArgs& a, int64_t row, int col, int n, float rstd, float c,
                                         const float* g, const float* xh, float* d)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        d[i] = __builtin_fmaf(rstd, __builtin_fmaf(-xh[i], c, g[i]), d[i]);
    store8<E>(a.y + row * a.y_ld + (int64_t)col * E::SIZE, n, d);
}

// kGradThreads / TPR rows at a time in each of `wgs` workgroups, whose columns' sums for dw
// stay in registers over all its rows and meet in LDS at the end.
template <class E, class W, int TPR, int CH, bool DX, bool DW>
__global__ __launch_bounds__(kGradThreads) void norm_grad(NormArgs a, int wgs)
{
    constexpr int ROWS = kGradThreads / TPR, SHARES = ROWS < kGradThreads / 64 ? ROWS : kGradThreads / 64;
    __shared__ float red[2][16];
    __shared__ __attribute__((aligned(16))) float part[DW && ROWS > 1 ? TPR * CH * 8 : 1];
    const int at = threadIdx.x % TPR, group = threadIdx.x / TPR;
    float acc[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[c][i] = 0.f;
    const int turns = (a.rows + wgs * ROWS - 1) / (wgs * ROWS);
    for (int turn = 0; turn < turns; ++turn) {
        const int64_t row = ((int64_t)turn * wgs + blockIdx.x) * ROWS + group;
        const int width = row < a.rows ? a.width : 0;
        const float rstd = row < a.rows ? a.rstd[row] : 0.f;
        float g[CH][8], xh[CH][8], sum = 0.f;
        Raw8<E> other[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * TPR + at) * 8, n = width - col;
            const Raw8<E> dy = load_raw8<E>(a.x + row * a.x_ld + (int64_t)col * E::SIZE, n);
            const Raw8<E> z = load_raw8<E>(a.z + row * a.z_ld + (int64_t)col * E::SIZE, n);
            if (DX && a.res)
                other[c] = load_raw8<E>(a.res + row * a.res_ld + (int64_t)col * E::SIZE, n);
            unpack8<E>(dy, g[c]);
            unpack8<E>(z, xh[c]);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * TPR + at) * 8;
            float w[8];
            if (DX)
                load_weight<W>(a.weight, col, a.width - col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                xh[c][i] *= rstd;
                if (DW)
                    acc[c][i] = __builtin_fmaf(g[c][i], xh[c][i], acc[c][i]);
                if (DX) {
                    g[c][i] *= w[i];
                    sum = __builtin_fmaf(g[c][i], xh[c][i], sum);
                }
            }
        }
        if (DX) {
            const float mean = row_sum<TPR>(sum, red[turn & 1]) / (float)a.width;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int col = (c * TPR + at) * 8;
                float d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (a.res)
                    unpack8<E>(other[c], d);
                if (col < width)
                    store_dx<E>(a, row, col, width - col, rstd, mean, g[c], xh[c], d);
            }
        }
    }
    if (DW) {
        // (rows that share a wave first)
#pragma unroll
        for (int x = TPR; x < 64; x *= 2)
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[c][i] += __shfl_xor(acc[c][i], x);
        const int own = TPR < 64 ? threadIdx.x / 64 : group;
        const bool first = TPR >= 64 || threadIdx.x % 64 < TPR;
        if constexpr (SHARES > 1) {
            for (int r = 0; r < SHARES - 1; ++r) {
                if (own == r && first)
#pragma unroll
                    for (int c = 0; c < CH; ++c)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float* const to = part + (c * TPR + at) * 8 + i;
                            *to = r == 0 ? acc[c][i] : *to + acc[c][i];
                        }
                __syncthreads();
            }
        }
        if (own != SHARES - 1 || !first)
            return;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = (c * TPR + at) * 8;
            if constexpr (SHARES > 1)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[c][i] += part[col + i];
            store8<F32>(reinterpret_cast<char*>(a.partial + (int64_t)blockIdx.x * a.width + col), a.width - col, acc[c]);
        }
    }
}

// dx of rows that do not fit the registers.
template <class E, class W>
__global__ __launch_bounds__(1024) void norm_dx_wide(NormArgs a)
{
    __shared__ float red[16];
    const int64_t row = workgroup();
    if (row >= a.rows)
        return;
    const float rstd = a.rstd[row];
    const auto load = [&](int col, float* g, float* xh) {
        const int n = a.width - col;
        float w[8];
        load8<E>(a.x + row * a.x_ld + (int64_t)col * E::SIZE, n, g);
        load8<E>(a.z + row * a.z_ld + (int64_t)col * E::SIZE, n, xh);
        load_weight<W>(a.weight, col, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[i] *= w[i];
            xh[i] *= rstd;
        }
    };
    float sum = 0.f;
    for (int col = threadIdx.x * 8; col < a.width; col += 1024 * 8) {
        float g[8], xh[8];
        load(col, g, xh);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum = __builtin_fmaf(g[i], xh[i], sum);
    }
    const float mean = row_sum<1024>(sum, red) / (float)a.width;
    for (int col = threadIdx.x * 8; col < a.width; col += 1024 * 8) {
        float g[8], xh[8];
        load(col, g, xh);
        float d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (a.res)
            load8<E>(a.res + row * a.res_ld + (int64_t)col * E::SIZE, a.width - col, d);
        store_dx<E>(a, row, col, a.width - col, rstd, mean, g, xh, d);
    }
}

// Partial rows of dw by columns, for rows that do not fit the registers: workgroup
// (c, p) takes rows p, p + groups, ...
template <class E>
__global__ __launch_bounds__(kColumnThreads) void norm_dw_wide(NormArgs a, int groups, unsigned strips)
{
    const unsigned wg = workgroup(), p = wg / strips;
    const int col = (int)((wg - p * strips) * kColumnThreads + threadIdx.x) * 8;
    if (p >= (unsigned)groups || col >= a.width)
        return;
    const int n = a.width - col;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int64_t row = p; row < a.rows; row += groups) {
        const float rstd = a.rstd[row];
        float g[8], z[8];
        load8<E>(a.x + row * a.x_ld + (int64_t)col * E::SIZE, n, g);
        load8<E>(a.z + row * a.z_ld + (int64_t)col * E::SIZE, n, z);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[i] = __builtin_fmaf(g[i], z[i] * rstd, acc[i]);
    }
    store8<F32>(reinterpret_cast<char*>(a.partial + (int64_t)p * a.width + col), n, acc);
}

// dw = sum of the partial rows: 32 columns a workgroup, 8 threads of four columns by 32
// runs of rows, whose sums meet in LDS in ascending order.
__global__ __launch_bounds__(256) void norm_dw_sum(const float* partial, int groups, int width, float* dw)
{
    __shared__ float part[32][32];
    const int lane = threadIdx.x & 7, run = threadIdx.x >> 3;
    const int col = blockIdx.x * 32 + lane * 4, n = width - col;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int p = run; p < groups; p += 32) {
        float v[4];
        load_vec<F32>(reinterpret_cast<const char*>(partial + (int64_t)p * width + col), n, v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        part[run][lane * 4 + i] = acc[i];
    __syncthreads();
    if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < width) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r)
            s += part[r][threadIdx.x];
        dw[blockIdx.x * 32 + threadIdx.x] = s;
    }
}

// ------------------------------------------------------------ launchers

int norm_partials(int rows, int width)
{
    const int at_once = width <= kMaxResident ? kGradThreads / row_threads(width) : 1;
    return min((rows + at_once - 1) / at_once, kPartials);
}

namespace {

template <class E, class W, int TPR, int CH>
hipError_t launch_rows(const NormArgs& a, hipStream_t s)
{
    constexpr int per = threads_of(TPR) / TPR;
    hipLaunchKernelGGL((norm_rows<E, W, TPR, CH>), grid_of(((int64_t)a.rows + per - 1) / per), dim3(threads_of(TPR)), 0,
                       s, a);
    return hipGetLastError();
}

template <class E, class W, int TPR, int CH>
hipError_t launch_grad(const NormArgs& a, hipStream_t s)
{
    const int wgs = norm_partials(a.rows, a.width);
    const auto kernel = a.y ? (a.dw ? norm_grad<E, W, TPR, CH, true, true> : norm_grad<E, W, TPR, CH, true, false>)
                            : norm_grad<E, W, TPR, CH, false, true>;
    hipLaunchKernelGGL(kernel, dim3(wgs), dim3(kGradThreads), 0, s, a, wgs);
    return hipGetLastError();
}

template <class E, class W>
hipError_t launch_wide(const NormArgs& a, bool back, hipStream_t s)
{
    if (!back) {
        hipLaunchKernelGGL((norm_rows_wide<E, W>), grid_of(a.rows), dim3(1024), 0, s, a);
        return hipGetLastError();
    }
    if (a.dw) {  // before dx, which may stand on dy
        const int groups = norm_partials(a.rows, a.width);
        const unsigned strips = (a.width + kColumnThreads * 8 - 1) / (kColumnThreads * 8);
        hipLaunchKernelGGL(norm_dw_wide<E>, grid_of((int64_t)groups * strips), dim3(kColumnThreads), 0, s, a, groups,
                           strips);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    if (a.y)
        hipLaunchKernelGGL((norm_dx_wide<E, W>), grid_of(a.rows), dim3(1024), 0, s, a);
    return hipGetLastError();
}

// One step of eight columns a thread where that occupies at least three quarters of the
// row's threads: more waves have loads under way (8192 rows of 4096, 7168 and 8192 bf16
// columns to z, y and codes: 54.8, 93.1 and 104.9 us, with two steps a thread 59.9, 97.9
// and 110.6; of 5120 columns, five eighths of 1024 threads, 75.6 and 73.9).
template <class E, class W>
hipError_t launch_norm(const NormArgs& a, hipStream_t s)
{
    const auto fills = [&](int threads) { return a.width <= threads * 8 && a.width * 4 >= threads * 8 * 3; };
    if (a.width <= 64)
        return launch_rows<E, W, 8, 1>(a, s);
    if (a.width <= 128)
        return launch_rows<E, W, 16, 1>(a, s);
    if (a.width <= 256)
        return launch_rows<E, W, 32, 1>(a, s);
    if (a.width <= 512)
        return launch_rows<E, W, 64, 1>(a, s);
    if (a.width <= 1024)
        return launch_rows<E, W, 64, 2>(a, s);
    if (a.width <= 2048)
        return launch_rows<E, W, 256, 1>(a, s);
    if (fills(512))
        return launch_rows<E, W, 512, 1>(a, s);
    if (a.width <= 4096)
        return launch_rows<E, W, 256, 2>(a, s);
    if (fills(1024))
        return launch_rows<E, W, 1024, 1>(a, s);
    if (a.width <= 8192)
        return launch_rows<E, W, 512, 2>(a, s);
    if (a.width <= kMaxResident)
        return launch_rows<E, W, 1024, 2>(a, s);
    return launch_wide<E, W>(a, false, s);
}

template <class E, class W>
hipError_t launch_back(const NormArgs& a, hipStream_t s)
{
    if (a.width <= 64)
        return launch_grad<E, W, 8, 1>(a, s);
    if (a.width <= 128)
        return launch_grad<E, W, 16, 1>(a, s);
    if (a.width <= 256)
        return launch_grad<E, W, 32, 1>(a, s);
    if (a.width <= 512)
        return launch_grad<E, W, 64, 1>(a, s);
    if (a.width <= 1024)
        return launch_grad<E, W, 64, 2>(a, s);
    if (a.width <= 2048)
        return launch_grad<E, W, 256, 1>(a, s);
    if (a.width <= 4096)
        return launch_grad<E, W, 256, 2>(a, s);
    if (a.width <= 8192)
        return launch_grad<E, W, 512, 2>(a, s);
    if (a.width <= kMaxResident)
        return launch_grad<E, W, 1024, 2>(a, s);
    return launch_wide<E, W>(a, true, s);
}

template <class E, class W>
hipError_t launch_width(const NormArgs& a, bool back, hipStream_t s)
{
    return back ? launch_back<E, W>(a, s) : launch_norm<E, W>(a, s);
}

template <class E>
hipError_t launch_weight(const NormArgs& a, bool back, hipStream_t s)
{
    return a.w_dtype == a.dtype ? launch_width<E, E>(a, back, s) : launch_width<E, F32>(a, back, s);
}

hipError_t launch_type(const NormArgs& a, bool back, hipStream_t s)
{
    switch (a.dtype) {
    case MOE_DTYPE_BF16: return launch_weight<Bf16>(a, back, s);
    case MOE_DTYPE_F16: return launch_weight<F16>(a, back, s);
    case MOE_DTYPE_F32: return launch_width<F32, F32>(a, back, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) { return launch_type(a, false, s); }

hipError_t launch_rms_norm_bwd(const NormArgs& a, hipStream_t s)
{
    if (a.rows > 0) {
        const hipError_t e = launch_type(a, true, s);
        if (e != hipSuccess)
            return e;
    }
    if (a.dw)
        hipLaunchKernelGGL(norm_dw_sum, dim3((a.width + 31) / 32), dim3(256), 0, s, a.partial,
                           norm_partials(a.rows, a.width), a.width, a.dw);
    return hipGetLastError();
}

}  // namespace moe
