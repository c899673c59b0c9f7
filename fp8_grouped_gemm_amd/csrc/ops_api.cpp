// Host side of the C ABI declared in include/moe_ops.h: every check runs
// before the first HIP call, so invalid calls enqueue nothing.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/moe_ops.h"
#include "ops_internal.h"

namespace {

constexpr int64_t kMaxLd = INT64_C(1) << 30;  // row strides, elements (spans stay below 2^63 bytes)

// Bytes per element, 0 for an unknown type.
int elem_bytes(int32_t dtype)
{
    switch (dtype) {
    case MOE_DTYPE_BF16:
    case MOE_DTYPE_F16: return 2;
    case MOE_DTYPE_F32: return 4;
    case MOE_DTYPE_U8: return 1;
    default: return 0;
    }
}

bool misaligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

// Row stride in elements: 0 stands for the width; -1 if it is invalid.
int64_t stride(int64_t ld, int64_t width)
{
    if (ld == 0)
        return width;
    return ld < width || ld > kMaxLd ? -1 : ld;
}

struct Span {
    uintptr_t lo, hi;
};

// The bytes from the first to the last element of a row matrix (empty for null).
Span span(const void* p, int64_t rows, int64_t ld, int64_t width, int size)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (!p || rows <= 0)
        return {lo, lo};
    return {lo, lo + static_cast<uintptr_t>(((rows - 1) * ld + width) * size)};
}

bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

// The shape checks the permutation entry points share.
int check_rows(int32_t T, int32_t K, int32_t R, int32_t width, int32_t dtype, bool bytes_ok)
{
    const int es = elem_bytes(dtype);
    if (T < 0 || K < 1 || R < 0 || width < 1 || es == 0 || (es == 1 && !bytes_ok))
        return MOE_ERR_INVALID_ARG;
    if (K > 1024 || static_cast<int64_t>(T) * K >= (1 << 24) || R >= (1 << 28) ||
        width >= (1 << 24))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

int launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// dx = sum of a token's pool rows, weighted or not: moe_permute_bwd and moe_unpermute.
int token_sums(int32_t T, int32_t K, int32_t R, int32_t width, int32_t dtype, const void* rows,
               int64_t rows_ld, const int32_t* src_row, const float* w, void* out, int64_t out_ld,
               void* stream)
{
    int rc = check_rows(T, K, R, width, dtype, false);
    if (rc != MOE_OK)
        return rc;
    if (T == 0)
        return MOE_OK;
    const int es = elem_bytes(dtype);
    const int64_t rld = stride(rows_ld, width), old = stride(out_ld, width);
    if ((!rows && R > 0) || !src_row || !out || rld < 0 || old < 0 || misaligned(rows, es) ||
        misaligned(out, es) || misaligned(src_row, 4) || misaligned(w, 4))
        return MOE_ERR_INVALID_ARG;
    const int64_t slots = static_cast<int64_t>(T) * K;
    const Span o = span(out, T, old, width, es);
    if (overlap(o, span(rows, R, rld, width, es)) || overlap(o, span(src_row, 1, slots, slots, 4)) ||
        overlap(o, span(w, 1, slots, slots, 4)))
        return MOE_ERR_INVALID_ARG;
    rc = moe::device_status();
    if (rc != MOE_OK)
        return rc;
    moe::RowsArgs a{};
    a.T = T; a.K = K; a.R = R; a.width = width; a.dtype = dtype;
    a.pool = static_cast<const char*>(rows);
    a.pool_ld = rld * es;
    a.tok_out = static_cast<char*>(out);
    a.tok_ld = old * es;
    a.src_row = src_row;
    a.w = w;
    return launched(moe::launch_unpermute(a, static_cast<hipStream_t>(stream)));
}

int check_mx(int32_t rows, int32_t cols, int32_t dtype, const void* x, int64_t ld,
             const uint8_t* codes, const uint8_t* sf, int64_t& out_ld)
{
    const int es = elem_bytes(dtype);
    if (rows < 0 || cols < 1 || es < 2)
        return MOE_ERR_INVALID_ARG;
    if (cols % 32 != 0 || cols >= (1 << 24) ||
        static_cast<int64_t>(rows) * cols >= (INT64_C(1) << 40))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    out_ld = stride(ld, cols);
    if (rows == 0)
        return MOE_OK;
    if (!x || !codes || !sf || out_ld < 0 || misaligned(x, es) || misaligned(codes, 4))
        return MOE_ERR_INVALID_ARG;
    const Span sx = span(x, rows, out_ld, cols, es), sc = span(codes, rows, cols / 2, cols / 2, 1),
               ss = span(sf, rows, cols / 32, cols / 32, 1);
    if (overlap(sx, sc) || overlap(sx, ss) || overlap(sc, ss))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe::MxQuantArgs mx_args(int32_t rows, int32_t cols, int32_t dtype, const void* x, int64_t ld,
                         const uint8_t* codes, const uint8_t* sf)
{
    moe::MxQuantArgs a{};
    a.rows = rows; a.cols = cols; a.dtype = dtype;
    a.x = static_cast<char*>(const_cast<void*>(x));
    a.ld = ld * elem_bytes(dtype);
    a.codes = const_cast<uint8_t*>(codes);
    a.sf = const_cast<uint8_t*>(sf);
    return a;
}

int check_gemm(int32_t groups, int32_t rows, int32_t n, int32_t k)
{
    if (groups < 1 || rows < 0 || n < 0 || k < 1)
        return MOE_ERR_INVALID_ARG;
    if (k % 32 != 0 || k > (1 << 20) || groups > 1024 || rows >= (1 << 28) || n >= (1 << 28))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_permute(int32_t T, int32_t K, int32_t R, int32_t width, int32_t dtype, const void* x,
                int64_t x_ld, const int32_t* row_src, const int32_t* src_row,
                const int32_t* used, void* xp, int64_t xp_ld, void* stream)
{
    int rc = check_rows(T, K, R, width, dtype, true);
    if (rc != MOE_OK)
        return rc;
    if (R == 0)
        return MOE_OK;
    const int es = elem_bytes(dtype);
    const int64_t ild = stride(x_ld, width), old = stride(xp_ld, width);
    if ((T > 0 && (!x || !src_row)) || !row_src || !xp || ild < 0 || old < 0 ||
        misaligned(x, es) || misaligned(xp, es) || misaligned(row_src, 4) ||
        misaligned(src_row, 4) || misaligned(used, 4))
        return MOE_ERR_INVALID_ARG;
    const int64_t slots = static_cast<int64_t>(T) * K;
    const Span o = span(xp, R, old, width, es);
    if (overlap(o, span(x, T, ild, width, es)) || overlap(o, span(row_src, 1, R, R, 4)) ||
        overlap(o, span(T ? src_row : nullptr, 1, slots, slots, 4)) || overlap(o, span(used, 1, 1, 1, 4)))
        return MOE_ERR_INVALID_ARG;
    rc = moe::device_status();
    if (rc != MOE_OK)
        return rc;
    moe::RowsArgs a{};
    a.T = T; a.K = K; a.R = R; a.width = width; a.dtype = dtype;
    a.tok = static_cast<const char*>(x);
    a.tok_ld = ild * es;
    a.pool_out = static_cast<char*>(xp);
    a.pool_out_ld = old * es;
    a.row_src = row_src;
    a.src_row = src_row;
    a.used = used;
    return launched(moe::launch_permute(a, static_cast<hipStream_t>(stream)));
}

int moe_permute_bwd(int32_t T, int32_t K, int32_t R, int32_t width, int32_t dtype,
                    const void* dxp, int64_t dxp_ld, const int32_t* src_row, void* dx,
                    int64_t dx_ld, void* stream)
{
    return token_sums(T, K, R, width, dtype, dxp, dxp_ld, src_row, nullptr, dx, dx_ld, stream);
}

int moe_unpermute(int32_t T, int32_t K, int32_t R, int32_t width, int32_t dtype, const void* yp,
                  int64_t yp_ld, const int32_t* src_row, const float* topk_w, void* y,
                  int64_t y_ld, void* stream)
{
    return token_sums(T, K, R, width, dtype, yp, yp_ld, src_row, topk_w, y, y_ld, stream);
}

int moe_unpermute_bwd(int32_t T, int32_t K, int32_t R, int32_t width, int32_t dtype,
                      const void* dy, int64_t dy_ld, const void* yp, int64_t yp_ld,
                      const int32_t* row_src, const int32_t* src_row, const int32_t* used,
                      const float* topk_w, void* dyp, int64_t dyp_ld, float* dw, void* stream)
{
    int rc = check_rows(T, K, R, width, dtype, false);
    if (rc != MOE_OK)
        return rc;
    const int es = elem_bytes(dtype);
    const int64_t dld = stride(dy_ld, width), yld = dw ? stride(yp_ld, width) : 0,
                  old = dyp ? stride(dyp_ld, width) : 0;
    // (without tokens or pool rows a requested output may be empty, its address null)
    if ((!dyp && !dw && T > 0 && R > 0) || dld < 0 || yld < 0 || old < 0 || (T > 0 && (!dy || !src_row)) ||
        (T > 0 && dw && !yp && R > 0) || misaligned(dy, es) || (dw && misaligned(yp, es)) ||
        misaligned(dyp, es) || misaligned(dw, 4) || misaligned(topk_w, 4) ||
        misaligned(row_src, 4) || misaligned(src_row, 4) || misaligned(used, 4))
        return MOE_ERR_INVALID_ARG;
    const int64_t slots = static_cast<int64_t>(T) * K;
    const Span op = span(dyp, R, old, width, es), ow = span(dw, 1, slots, slots, 4);
    const Span in[6] = {span(dy, T, dld, width, es), span(dw ? yp : nullptr, R, yld, width, es),
                        span(row_src, 1, R, R, 4), span(src_row, 1, slots, slots, 4),
                        span(topk_w, 1, slots, slots, 4), span(used, 1, 1, 1, 4)};
    for (const Span& i : in)
        if (overlap(op, i) || overlap(ow, i))
            return MOE_ERR_INVALID_ARG;
    if (overlap(op, ow))
        return MOE_ERR_INVALID_ARG;
    if ((!dyp && !dw) || (T == 0 && (!dyp || !row_src || R == 0)))
        return MOE_OK;
    rc = moe::device_status();
    if (rc != MOE_OK)
        return rc;
    moe::RowsArgs a{};
    a.T = T; a.K = K; a.R = R; a.width = width; a.dtype = dtype;
    a.tok = static_cast<const char*>(dy);
    a.tok_ld = dld * es;
    a.pool = static_cast<const char*>(yp);
    a.pool_ld = yld * es;
    a.pool_out = static_cast<char*>(dyp);
    a.pool_out_ld = old * es;
    a.row_src = dyp ? row_src : nullptr;
    a.src_row = src_row;
    a.used = used;
    a.w = topk_w;
    a.dw = dw;
    return launched(moe::launch_unpermute_bwd(a, static_cast<hipStream_t>(stream)));
}

int moe_quantize_mxfp4(int32_t rows, int32_t cols, int32_t dtype, const void* x, int64_t x_ld,
                       uint8_t* codes, uint8_t* sf, void* stream)
{
    int64_t ld;
    int rc = check_mx(rows, cols, dtype, x, x_ld, codes, sf, ld);
    if (rc != MOE_OK || rows == 0)
        return rc;
    rc = moe::device_status();
    if (rc != MOE_OK)
        return rc;
    return launched(moe::launch_quantize_mxfp4(mx_args(rows, cols, dtype, x, ld, codes, sf),
                                               static_cast<hipStream_t>(stream)));
}

int moe_dequantize_mxfp4(int32_t rows, int32_t cols, int32_t dtype, const uint8_t* codes,
                         const uint8_t* sf, void* x, int64_t x_ld, void* stream)
{
    int64_t ld;
    int rc = check_mx(rows, cols, dtype, x, x_ld, codes, sf, ld);
    if (rc != MOE_OK || rows == 0)
        return rc;
    rc = moe::device_status();
    if (rc != MOE_OK)
        return rc;
    return launched(moe::launch_dequantize_mxfp4(mx_args(rows, cols, dtype, x, ld, codes, sf),
                                                 static_cast<hipStream_t>(stream)));
}

int moe_gemm_mxfp4(int32_t groups, int32_t rows, int32_t n, int32_t k, int32_t dtype,
                   const uint8_t* a, const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf,
                   const int32_t* offsets, const int32_t* counts, int32_t slots, void* y,
                   int64_t y_ld, void* stream)
{
    const int es = elem_bytes(dtype);
    if (es < 2 || slots < 0 || (!offsets && (groups != 1 || counts)))
        return MOE_ERR_INVALID_ARG;
    const int sizes = check_gemm(groups, rows, n, k);
    if (sizes != MOE_OK)
        return sizes;
    if (rows == 0 || n == 0)
        return MOE_OK;
    const int64_t ld = stride(y_ld, n);
    if (!a || !a_sf || !b || !b_sf || !y || ld < 0 || misaligned(a, 16) || misaligned(b, 16) ||
        misaligned(y, es) || misaligned(offsets, 4) || misaligned(counts, 4))
        return MOE_ERR_INVALID_ARG;
    const int64_t wrows = static_cast<int64_t>(groups) * n;
    const Span o = span(y, rows, ld, n, es);
    if (overlap(o, span(a, rows, k / 2, k / 2, 1)) || overlap(o, span(a_sf, rows, k / 32, k / 32, 1)) ||
        overlap(o, span(b, wrows, k / 2, k / 2, 1)) || overlap(o, span(b_sf, wrows, k / 32, k / 32, 1)) ||
        overlap(o, span(offsets, 1, groups + 1, groups + 1, 4)) ||
        overlap(o, span(counts, 1, groups, groups, 4)))
        return MOE_ERR_INVALID_ARG;
    const int rc = moe::device_status();
    if (rc != MOE_OK)
        return rc;
    moe::MxGemmArgs g{};
    g.E = groups; g.R = rows; g.N = n; g.K = k; g.dtype = dtype;
    // (without counts the segments take in their padding, which slots leaves out)
    g.slots = offsets && counts && slots > 0 && slots < rows ? slots : rows;
    g.a = a; g.a_sf = a_sf; g.b = b; g.b_sf = b_sf;
    g.offsets = offsets; g.counts = counts;
    g.y = static_cast<char*>(y);
    g.y_ld = ld * es;
    return launched(moe::launch_gemm_mxfp4(g, static_cast<hipStream_t>(stream)));
}

int moe_gemm_mxfp4_info(int32_t groups, int32_t rows, int32_t n, int32_t k, int32_t* tile_m,
                        int32_t* tile_n)
{
    if (!tile_m || !tile_n || groups < 0)
        return MOE_ERR_INVALID_ARG;
    const int rc = check_gemm(groups == 0 ? 1 : groups, rows, n, k);
    if (rc == MOE_OK)
        moe::gemm_mxfp4_tile(groups == 0 ? 1 : groups, rows, n, k, groups != 0, *tile_m, *tile_n);
    return rc;
}

}  // extern "C"
