// Host side of the C ABI declared in include/moe_ops.h: every check runs
// before the first HIP call, so invalid calls enqueue nothing.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/moe_ops.h"
#include "ops_internal.h"

namespace {

constexpr int64_t kMaxLd = INT64_C(1) << 30;  // row strides, elements (spans stay below 2^63 bytes)

constexpr int64_t kMaxWgradLd = INT64_C(1) << 24;  // (a stage of 64 of dy's rows spans at most 2^31 bytes)

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

// Bytes per row and alignment of the scales of 8-bit rows; false for an unknown format.
bool sf_layout(int32_t format, int64_t cols, int64_t& row_bytes, int& align)
{
    row_bytes = format == MOE_SF_F32_128 ? cols / 128 * 4 : cols / 32;
    align = format == MOE_SF_F32_128 ? 4 : 1;
    return format == MOE_SF_F32_128 || format == MOE_SF_UE8M0_32;
}

int sf_block(int32_t format) { return format == MOE_SF_F32_128 ? 128 : 32; }

// Whether two row matrices are one and the same.
bool same_rows(const void* a, int64_t a_ld, const void* b, int64_t b_ld) { return a == b && a_ld == b_ld; }

// Whether an output of a call overlaps an input or another output; bit i of
// allowed[o]: output o may stand on input i.
template <int O, int I>
bool any_overlap(const Span (&out)[O], const Span (&in)[I], const unsigned (&allowed)[O])
{
    for (int o = 0; o < O; ++o) {
        for (int i = 0; i < I; ++i)
            if (!(allowed[o] >> i & 1) && overlap(out[o], in[i]))
                return true;
        for (int p = 0; p < o; ++p)
            if (overlap(out[o], out[p]))
                return true;
    }
    return false;
}

int check_gate(int32_t T, int32_t E, int32_t K, int32_t dtype, int32_t score)
{
    if (T < 0 || E < 1 || K < 1 || K > E || elem_bytes(dtype) < 2 ||
        (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID))
        return MOE_ERR_INVALID_ARG;
    if (E > 1024 || K > 64 || T >= (1 << 28))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

int check_norm(int32_t rows, int32_t width, int32_t dtype, int32_t w_dtype)
{
    if (rows < 0 || width < 1 || elem_bytes(dtype) < 2 || (w_dtype != dtype && w_dtype != MOE_DTYPE_F32))
        return MOE_ERR_INVALID_ARG;
    if (rows >= (1 << 28) || width >= (1 << 24))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

size_t norm_workspace(int32_t rows, int32_t width)
{
    return static_cast<size_t>(moe::norm_partials(rows, width)) * width * 4;
}

int check_swiglu(int32_t R, int32_t inner, int32_t dtype, bool codes, int32_t format)
{
    int64_t unused;
    int align;
    if (R < 0 || inner < 1 || elem_bytes(dtype) < 2 || (codes && !sf_layout(format, inner, unused, align)))
        return MOE_ERR_INVALID_ARG;
    if (R >= (1 << 28) || inner >= (1 << 23) || (codes && inner % sf_block(format) != 0))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

int check_wgrad(int32_t groups, int32_t rows, int32_t n, int32_t k)
{
    if (groups < 1 || rows < 0 || n < 0 || k < 1)
        return MOE_ERR_INVALID_ARG;
    if (k % 32 != 0 || k > (1 << 20) || groups > 1024 || rows >= (1 << 28) || n >= (1 << 20))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

size_t wgrad_workspace(int32_t groups, int32_t rows, int32_t n, int32_t k)
{
    int kind, split = 1;
    if (rows > 0 && n > 0)
        moe::wgrad_choose(groups, rows, n, k, kind, split);
    return split > 1 ? static_cast<size_t>(split) * groups * n * k * 4 : 0;
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

int moe_gate(int32_t T, int32_t E, int32_t K, int32_t dtype, const void* logits, int64_t logits_ld,
             const float* bias, const uint8_t* mask, int32_t score, int32_t groups,
             int32_t top_groups, int32_t group_top, int32_t renorm, float scale,
             int32_t* topk_idx, float* topk_w, void* stream)
{
    int rc = check_gate(T, E, K, dtype, score);
    if (rc != MOE_OK)
        return rc;
    if (groups < 1 || E % groups != 0 || top_groups < 1 || top_groups > groups || group_top < 1 ||
        group_top > E / groups || K > E / groups * top_groups)
        return MOE_ERR_INVALID_ARG;
    if (groups > 64)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0)
        return MOE_OK;
    const int es = elem_bytes(dtype);
    const int64_t ld = stride(logits_ld, E), slots = static_cast<int64_t>(T) * K;
    if (!logits || !topk_idx || !topk_w || ld < 0 || misaligned(logits, es) || misaligned(bias, 4) ||
        misaligned(topk_idx, 4) || misaligned(topk_w, 4))
        return MOE_ERR_INVALID_ARG;
    const Span out[2] = {span(topk_idx, 1, slots, slots, 4), span(topk_w, 1, slots, slots, 4)};
    const Span in[3] = {span(logits, T, ld, E, es), span(bias, 1, E, E, 4), span(mask, 1, T, T, 1)};
    const unsigned allowed[2] = {};
    if (any_overlap(out, in, allowed))
        return MOE_ERR_INVALID_ARG;
    rc = moe::device_status();
    if (rc != MOE_OK)
        return rc;
    moe::GateArgs a{};
    a.T = T; a.E = E; a.K = K; a.dtype = dtype;
    a.logits = static_cast<const char*>(logits);
    a.ld = ld * es;
    a.bias = bias;
    a.mask = mask;
    a.score = score;
    a.groups = groups; a.top_groups = top_groups; a.group_top = group_top;
    a.renorm = renorm != 0;
    a.scale = scale;
    a.idx = topk_idx;
    a.w = topk_w;
    return launched(moe::launch_gate(a, static_cast<hipStream_t>(stream)));
}

int moe_gate_bwd(int32_t T, int32_t E, int32_t K, int32_t dtype, const void* logits,
                 int64_t logits_ld, const int32_t* topk_idx, const float* dw, int32_t score,
                 int32_t renorm, float scale, void* dlogits, int64_t dlogits_ld, void* stream)
{
    int rc = check_gate(T, E, K, dtype, score);
    if (rc != MOE_OK)
        return rc;
    if (T == 0)
        return MOE_OK;
    const int es = elem_bytes(dtype);
    const int64_t ld = stride(logits_ld, E), old = stride(dlogits_ld, E), slots = static_cast<int64_t>(T) * K;
    if (!logits || !topk_idx || !dw || !dlogits || ld < 0 || old < 0 || misaligned(logits, es) ||
        misaligned(dlogits, es) || misaligned(topk_idx, 4) || misaligned(dw, 4))
        return MOE_ERR_INVALID_ARG;
    const Span out[1] = {span(dlogits, T, old, E, es)};
    const Span in[3] = {span(logits, T, ld, E, es), span(topk_idx, 1, slots, slots, 4),
                        span(dw, 1, slots, slots, 4)};
    const unsigned allowed[1] = {};
    if (any_overlap(out, in, allowed))
        return MOE_ERR_INVALID_ARG;
    rc = moe::device_status();
    if (rc != MOE_OK)
        return rc;
    moe::GateArgs a{};
    a.T = T; a.E = E; a.K = K; a.dtype = dtype;
    a.logits = static_cast<const char*>(logits);
    a.ld = ld * es;
    a.score = score;
    a.renorm = renorm != 0;
    a.scale = scale;
    a.idx = const_cast<int32_t*>(topk_idx);
    a.w = const_cast<float*>(dw);
    a.dlogits = static_cast<char*>(dlogits);
    a.dlogits_ld = old * es;
    return launched(moe::launch_gate_bwd(a, static_cast<hipStream_t>(stream)));
}

int moe_rms_norm(int32_t rows, int32_t width, int32_t dtype, const void* x, int64_t x_ld,
                 const void* residual, int64_t residual_ld, const void* weight, int32_t w_dtype,
                 float eps, void* z, int64_t z_ld, float* rstd, void* y, int64_t y_ld,
                 uint8_t* codes, void* sf, int32_t sf_format, void* stream)
{
    int rc = check_norm(rows, width, dtype, w_dtype);
    if (rc != MOE_OK)
        return rc;
    int64_t sf_row = 0;
    int sf_align = 1;
    if (codes || sf) {
        if (!sf_layout(sf_format, width, sf_row, sf_align))
            return MOE_ERR_INVALID_ARG;
        if (width % sf_block(sf_format) != 0)
            return MOE_ERR_UNSUPPORTED_SHAPE;
    }
    if (rows == 0)
        return MOE_OK;
    const int es = elem_bytes(dtype), ws = elem_bytes(w_dtype);
    const int64_t xld = stride(x_ld, width), rld = residual ? stride(residual_ld, width) : 0,
                  zld = z ? stride(z_ld, width) : 0, yld = y ? stride(y_ld, width) : 0;
    if (!x || (!y && !codes) || !codes != !sf || (z && !residual) || xld < 0 || rld < 0 || zld < 0 ||
        yld < 0 || misaligned(x, es) || misaligned(residual, es) || misaligned(z, es) ||
        misaligned(y, es) || misaligned(weight, ws) || misaligned(rstd, 4) || misaligned(codes, 8) ||
        misaligned(sf, sf_align))
        return MOE_ERR_INVALID_ARG;
    const Span out[5] = {span(z, rows, zld, width, es), span(y, rows, yld, width, es),
                         span(rstd, 1, rows, rows, 4), span(codes, rows, width, width, 1),
                         span(sf, rows, sf_row, sf_row, 1)};
    const Span in[3] = {span(x, rows, xld, width, es), span(residual, rows, rld, width, es),
                        span(weight, 1, width, width, ws)};
    const auto onto = [&](const void* p, int64_t ld) {
        return p ? (same_rows(p, ld, x, xld) ? 1u : 0u) | (residual && same_rows(p, ld, residual, rld) ? 2u : 0u) : 0u;
    };
    const unsigned allowed[5] = {onto(z, zld), onto(y, yld)};
    if (any_overlap(out, in, allowed))
        return MOE_ERR_INVALID_ARG;
    rc = moe::device_status();
    if (rc != MOE_OK)
        return rc;
    moe::NormArgs a{};
    a.rows = rows; a.width = width; a.dtype = dtype; a.w_dtype = w_dtype;
    a.x = static_cast<const char*>(x); a.x_ld = xld * es;
    a.res = static_cast<const char*>(residual); a.res_ld = rld * es;
    a.weight = static_cast<const char*>(weight);
    a.eps = eps;
    a.z = static_cast<char*>(z); a.z_ld = zld * es;
    a.rstd = rstd;
    a.y = static_cast<char*>(y); a.y_ld = yld * es;
    a.codes = codes; a.sf = sf; a.sf_format = sf_format;
    return launched(moe::launch_rms_norm(a, static_cast<hipStream_t>(stream)));
}

int moe_rms_norm_bwd(int32_t rows, int32_t width, int32_t dtype, const void* dy, int64_t dy_ld,
                     const void* z, int64_t z_ld, const void* weight, int32_t w_dtype,
                     const float* rstd, const void* dz, int64_t dz_ld, void* dx, int64_t dx_ld,
                     float* dw, void* workspace, size_t workspace_bytes, void* stream)
{
    int rc = check_norm(rows, width, dtype, w_dtype);
    if (rc != MOE_OK)
        return rc;
    if (!dx && !dw)
        return rows == 0 ? MOE_OK : MOE_ERR_INVALID_ARG;
    if (rows == 0 && !dw)
        return MOE_OK;
    const int es = elem_bytes(dtype), ws = elem_bytes(w_dtype);
    const int64_t dyld = stride(dy_ld, width), zld = stride(z_ld, width),
                  dzld = dz ? stride(dz_ld, width) : 0, dxld = dx ? stride(dx_ld, width) : 0;
    if ((rows > 0 && (!dy || !z || !rstd)) || dyld < 0 || zld < 0 || dzld < 0 || dxld < 0 ||
        misaligned(dy, es) || misaligned(z, es) || misaligned(dz, es) || misaligned(dx, es) ||
        misaligned(weight, ws) || misaligned(rstd, 4) || misaligned(dw, 4) || misaligned(workspace, 16))
        return MOE_ERR_INVALID_ARG;
    const size_t need = dw ? norm_workspace(rows, width) : 0;
    if (need > 0 && !workspace)
        return MOE_ERR_INVALID_ARG;
    if (need > workspace_bytes)
        return MOE_ERR_WORKSPACE_TOO_SMALL;
    const Span out[3] = {span(dx, rows, dxld, width, es), span(dw, 1, width, width, 4),
                         span(need ? workspace : nullptr, 1, need, need, 1)};
    const Span in[5] = {span(dy, rows, dyld, width, es), span(dz, rows, dzld, width, es),
                        span(z, rows, zld, width, es), span(weight, 1, width, width, ws),
                        span(rstd, 1, rows, rows, 4)};
    const unsigned allowed[3] = {!dx ? 0u : (same_rows(dx, dxld, dy, dyld) ? 1u : 0u) |
                                                (dz && same_rows(dx, dxld, dz, dzld) ? 2u : 0u)};
    if (any_overlap(out, in, allowed))
        return MOE_ERR_INVALID_ARG;
    rc = moe::device_status();
    if (rc != MOE_OK)
        return rc;
    moe::NormArgs a{};
    a.rows = rows; a.width = width; a.dtype = dtype; a.w_dtype = w_dtype;
    a.x = static_cast<const char*>(dy); a.x_ld = dyld * es;
    a.res = static_cast<const char*>(dz); a.res_ld = dzld * es;
    a.weight = static_cast<const char*>(weight);
    a.z = static_cast<char*>(const_cast<void*>(z)); a.z_ld = zld * es;
    a.rstd = const_cast<float*>(rstd);
    a.y = static_cast<char*>(dx); a.y_ld = dxld * es;
    a.dw = dw;
    a.partial = static_cast<float*>(workspace);
    return launched(moe::launch_rms_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

int moe_rms_norm_bwd_workspace_bytes(int32_t rows, int32_t width, size_t* bytes)
{
    if (!bytes)
        return MOE_ERR_INVALID_ARG;
    const int rc = check_norm(rows, width, MOE_DTYPE_F32, MOE_DTYPE_F32);
    if (rc == MOE_OK)
        *bytes = norm_workspace(rows, width);
    return rc;
}

int moe_swiglu(int32_t R, int32_t inner, int32_t dtype, const void* gu, int64_t gu_ld, float clamp,
               const int32_t* row_src, const int32_t* used, void* h, int64_t h_ld,
               uint8_t* h_codes, void* h_sf, uint8_t* gu_codes, void* gu_sf, int32_t sf_format,
               void* stream)
{
    const bool eight = h_codes || h_sf || gu_codes || gu_sf;
    int rc = check_swiglu(R, inner, dtype, eight, sf_format);
    if (rc != MOE_OK)
        return rc;
    if (R == 0)
        return MOE_OK;
    const int es = elem_bytes(dtype);
    const int64_t width = 2 * static_cast<int64_t>(inner), gld = stride(gu_ld, width),
                  hld = h ? stride(h_ld, inner) : 0;
    int64_t sf_row = 0;
    int sf_align = 1;
    if (eight)
        sf_layout(sf_format, inner, sf_row, sf_align);
    if (!gu || (!h && !h_codes && !gu_codes) || !h_codes != !h_sf || !gu_codes != !gu_sf || gld < 0 ||
        hld < 0 || misaligned(gu, es) || misaligned(h, es) || misaligned(h_codes, 8) ||
        misaligned(gu_codes, 8) || misaligned(h_sf, sf_align) || misaligned(gu_sf, sf_align) ||
        misaligned(row_src, 4) || misaligned(used, 4))
        return MOE_ERR_INVALID_ARG;
    const Span out[5] = {span(h, R, hld, inner, es), span(h_codes, R, inner, inner, 1),
                         span(h_sf, R, sf_row, sf_row, 1), span(gu_codes, R, width, width, 1),
                         span(gu_sf, R, 2 * sf_row, 2 * sf_row, 1)};
    const Span in[3] = {span(gu, R, gld, width, es), span(row_src, 1, R, R, 4), span(used, 1, 1, 1, 4)};
    const unsigned allowed[5] = {};
    if (any_overlap(out, in, allowed))
        return MOE_ERR_INVALID_ARG;
    rc = moe::device_status();
    if (rc != MOE_OK)
        return rc;
    moe::SwigluArgs a{};
    a.R = R; a.inner = inner; a.dtype = dtype;
    a.gu = static_cast<const char*>(gu); a.gu_ld = gld * es;
    a.clamp = clamp;
    a.row_src = row_src; a.used = used;
    a.h = static_cast<char*>(h); a.h_ld = hld * es;
    a.h_codes = h_codes; a.h_sf = h_sf;
    a.gu_codes = gu_codes; a.gu_sf = gu_sf;
    a.sf_format = sf_format;
    return launched(moe::launch_swiglu(a, static_cast<hipStream_t>(stream)));
}

int moe_swiglu_bwd(int32_t R, int32_t inner, int32_t dtype, const void* dh, int64_t dh_ld,
                   const void* gu, int64_t gu_ld, const uint8_t* gu_codes, const void* gu_sf,
                   int32_t sf_format, float clamp, const int32_t* row_src, const int32_t* used,
                   void* dgu, int64_t dgu_ld, void* stream)
{
    const bool eight = gu_codes || gu_sf;
    int rc = check_swiglu(R, inner, dtype, eight, sf_format);
    if (rc != MOE_OK)
        return rc;
    if (R == 0)
        return MOE_OK;
    const int es = elem_bytes(dtype);
    const int64_t width = 2 * static_cast<int64_t>(inner), hld = stride(dh_ld, inner),
                  gld = gu ? stride(gu_ld, width) : 0, old = stride(dgu_ld, width);
    int64_t sf_row = 0;
    int sf_align = 1;
    if (eight)
        sf_layout(sf_format, width, sf_row, sf_align);
    if (!dh || !dgu || !gu == !gu_codes || !gu_codes != !gu_sf || hld < 0 || gld < 0 || old < 0 ||
        misaligned(dh, es) || misaligned(gu, es) || misaligned(dgu, es) || misaligned(gu_codes, 8) ||
        misaligned(gu_sf, sf_align) || misaligned(row_src, 4) || misaligned(used, 4))
        return MOE_ERR_INVALID_ARG;
    const Span out[1] = {span(dgu, R, old, width, es)};
    const Span in[6] = {span(gu, R, gld, width, es), span(dh, R, hld, inner, es),
                        span(gu_codes, R, width, width, 1), span(gu_sf, R, sf_row, sf_row, 1),
                        span(row_src, 1, R, R, 4), span(used, 1, 1, 1, 4)};
    const unsigned allowed[1] = {gu && same_rows(dgu, old, gu, gld) ? 1u : 0u};
    if (any_overlap(out, in, allowed))
        return MOE_ERR_INVALID_ARG;
    rc = moe::device_status();
    if (rc != MOE_OK)
        return rc;
    moe::SwigluArgs a{};
    a.R = R; a.inner = inner; a.dtype = dtype;
    a.gu = static_cast<const char*>(gu); a.gu_ld = gld * es;
    a.clamp = clamp;
    a.row_src = row_src; a.used = used;
    a.h = static_cast<char*>(const_cast<void*>(dh)); a.h_ld = hld * es;
    a.gu_codes = const_cast<uint8_t*>(gu_codes); a.gu_sf = const_cast<void*>(gu_sf);
    a.sf_format = sf_format;
    a.dgu = static_cast<char*>(dgu); a.dgu_ld = old * es;
    return launched(moe::launch_swiglu_bwd(a, static_cast<hipStream_t>(stream)));
}

int moe_gemm_wgrad(int32_t groups, int32_t rows, int32_t n, int32_t k, int32_t dtype,
                   const void* dy, int64_t dy_ld, const uint8_t* x, const void* x_sf,
                   int32_t sf_format, const int32_t* offsets, const int32_t* counts,
                   int32_t accumulate, void* dw, int32_t dw_dtype, void* workspace,
                   size_t workspace_bytes, void* stream)
{
    const int ds = elem_bytes(dw_dtype);
    int64_t sf_row;
    int sf_align;
    if ((dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) || ds < 2 ||
        !sf_layout(sf_format, k, sf_row, sf_align) || (!offsets && (groups != 1 || counts)))
        return MOE_ERR_INVALID_ARG;
    int rc = check_wgrad(groups, rows, n, k);
    if (rc != MOE_OK)
        return rc;
    if (k % sf_block(sf_format) != 0)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (n == 0 || (rows == 0 && accumulate))
        return MOE_OK;
    const int64_t ld = stride(dy_ld, n);
    if (!dw || ld < 0 || ld > kMaxWgradLd || (rows > 0 && (!dy || !x || !x_sf)) || misaligned(dy, 2) || misaligned(x, 16) ||
        misaligned(x_sf, sf_align) || misaligned(dw, ds) || misaligned(workspace, 16) ||
        misaligned(offsets, 4) || misaligned(counts, 4))
        return MOE_ERR_INVALID_ARG;
    const size_t need = wgrad_workspace(groups, rows, n, k);
    if (need > 0 && !workspace)
        return MOE_ERR_INVALID_ARG;
    if (need > workspace_bytes)
        return MOE_ERR_WORKSPACE_TOO_SMALL;
    const int64_t cells = static_cast<int64_t>(groups) * n;
    const Span out[2] = {span(dw, cells, k, k, ds), span(need ? workspace : nullptr, 1, need, need, 1)};
    const Span in[5] = {span(dy, rows, ld, n, 2), span(x, rows, k, k, 1), span(x_sf, rows, sf_row, sf_row, 1),
                        span(offsets, 1, groups + 1, groups + 1, 4), span(counts, 1, groups, groups, 4)};
    const unsigned allowed[2] = {};
    if (any_overlap(out, in, allowed))
        return MOE_ERR_INVALID_ARG;
    rc = moe::device_status();
    if (rc != MOE_OK)
        return rc;
    moe::WgradArgs a{};
    a.E = groups; a.R = rows; a.N = n; a.K = k;
    a.dtype = dtype; a.dw_dtype = dw_dtype;
    a.dy = static_cast<const char*>(dy); a.dy_ld = ld * 2;
    a.x = x;
    a.x_sf = static_cast<const char*>(x_sf);
    a.sf_format = sf_format;
    a.offsets = offsets; a.counts = counts;
    a.accumulate = accumulate != 0;
    a.dw = static_cast<char*>(dw);
    a.partial = static_cast<float*>(workspace);
    moe::wgrad_choose(groups, rows, n, k, a.kind, a.split);
    return launched(moe::launch_gemm_wgrad(a, static_cast<hipStream_t>(stream)));
}

int moe_gemm_wgrad_workspace_bytes(int32_t groups, int32_t rows, int32_t n, int32_t k, size_t* bytes)
{
    if (!bytes)
        return MOE_ERR_INVALID_ARG;
    const int rc = check_wgrad(groups, rows, n, k);
    if (rc == MOE_OK)
        *bytes = wgrad_workspace(groups, rows, n, k);
    return rc;
}

}  // extern "C"
