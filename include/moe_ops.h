/*
 * moe_ops.h — C ABI of the row operators of libmoe_fp8.so: what a layer that
 * does not run as one moe_forward needs around and instead of it.
 *   - moe_permute / moe_unpermute: token rows into the expert order of
 *     moe_route and back with the router weights applied, each with its
 *     gradient;
 *   - moe_quantize_mxfp4 / moe_dequantize_mxfp4: rows of bf16, f16 or f32 to
 *     and from microscaled 4-bit floating point (e2m1 codes, one UE8M0 scale
 *     per 32), the operand format of moe_forward_mx's weights;
 *   - moe_gemm_mxfp4: the product of two such matrices, dense or over the
 *     row segments of the experts.
 *
 * Conventions as in moe_fp8.h: device pointers owned by the caller, no
 * allocation, no host synchronisation, work enqueued on `stream` of the
 * current device, every argument checked on the host before any HIP call,
 * MOE_OK or a negative MOE_ERR_* code returned.  What differs: no plan (the
 * shapes are arguments), no workspace, and the matrices of bf16 / f16 / f32
 * rows have a row stride (`*_ld`, in elements, at least the row's width and at
 * most 2^30; 0 = densely packed).  Rows need only the alignment of their
 * element type.  Where an output must not overlap another tensor, that counts
 * whole spans, from a matrix's first element to its last, the gaps between
 * its rows among them.
 * No entry point uses atomics on results: equal calls give equal bits.
 * Every call may be captured into a HIP graph and replayed, and calls on
 * different streams are independent as long as their outputs are.
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "moe_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of row matrices. */
#define MOE_DTYPE_BF16 0
#define MOE_DTYPE_F16 1
#define MOE_DTYPE_F32 2
#define MOE_DTYPE_U8 3 /* moe_permute only: e4m3 or e2m1 codes, scale codes */

/*
 * Token rows into expert order.
 *   x        [T, width]          token rows, row stride x_ld
 *   row_src  int32 [pool_rows]   moe_route's slot f = t*K + j per pool row, -1 = padding
 *   src_row  int32 [T*K]         moe_route's pool row per slot, -1 = masked
 *   used     int32 [1]           pool rows in use: moe_route's offsets + E (a device
 *                                address; NULL: all pool_rows)
 *   xp       [pool_rows, width]  written: xp[src_row[f]] = x[f / K] for every routed slot,
 *                                zeros for the padding rows below *used; rows from *used
 *                                on are left as they were
 * Entries outside their range (row_src >= T*K, src_row >= pool_rows) count as
 * padding resp. masked.  The lists are moe_route's or equally consistent
 * (row_src[src_row[f]] == f); otherwise a row named twice holds either.
 * 1 <= width < 2^24, 1 <= K <= 1024, T*K < 2^24, 0 <= pool_rows < 2^28.
 * T == 0 still clears padding rows.  xp must not overlap an input.
 */
int moe_permute(int32_t num_tokens, int32_t top_k, int32_t pool_rows, int32_t width,
                int32_t dtype, const void* x, int64_t x_ld, const int32_t* row_src,
                const int32_t* src_row, const int32_t* used, void* xp, int64_t xp_ld,
                void* stream);

/*
 * Gradient of moe_permute: dx[t] = sum over j, ascending, of
 * dxp[src_row[t*K + j]], masked slots skipped; f32 sums, rounded once; a
 * token with no routed slot gets zeros.  dxp rows no slot names are not
 * read.  dtype bf16, f16 or f32.
 */
int moe_permute_bwd(int32_t num_tokens, int32_t top_k, int32_t pool_rows, int32_t width,
                    int32_t dtype, const void* dxp, int64_t dxp_ld, const int32_t* src_row,
                    void* dx, int64_t dx_ld, void* stream);

/*
 * Expert rows back to token order with the router weights:
 * y[t] = sum over j, ascending, of topk_w[t*K + j] * yp[src_row[t*K + j]];
 * masked slots are skipped (their weight and row are not read), f32 sums,
 * rounded once.  topk_w f32 [T, K], NULL: every weight 1.
 */
int moe_unpermute(int32_t num_tokens, int32_t top_k, int32_t pool_rows, int32_t width,
                  int32_t dtype, const void* yp, int64_t yp_ld, const int32_t* src_row,
                  const float* topk_w, void* y, int64_t y_ld, void* stream);

/*
 * Gradients of moe_unpermute for dy [T, width]:
 *   dyp [pool_rows, width]  topk_w[f] * dy[f / K] in the row of every routed slot (rounded
 *                           once), zeros for the padding rows below *used, rows from
 *                           *used on left as they were; NULL: not computed
 *   dw  f32 [T, K]          dot of dy[f / K] and yp[src_row[f]] in f32, 0 for a masked
 *                           slot; NULL: not computed (yp and its stride are then unused)
 * At least one of dyp and dw, unless T or pool_rows is 0 (an empty output may have
 * no address; the call then does what is left, if anything).  row_src and used serve dyp only (NULL
 * row_src: padding rows are left as they were).  topk_w NULL: every weight 1.
 * Neither output may overlap an input or the other.
 */
int moe_unpermute_bwd(int32_t num_tokens, int32_t top_k, int32_t pool_rows, int32_t width,
                      int32_t dtype, const void* dy, int64_t dy_ld, const void* yp,
                      int64_t yp_ld, const int32_t* row_src, const int32_t* src_row,
                      const int32_t* used, const float* topk_w, void* dyp, int64_t dyp_ld,
                      float* dw, void* stream);

/*
 * Rows to microscaled 4-bit floating point, 32 columns per block:
 *   sf = the smallest power of two >= max(amax, 1e-10) / 6, q = e2m1(v / sf)
 * rounded to nearest, ties to the even code (no value saturates).  This is the
 * library's rule for e2m1 weights; the OCP MX specification's conversion takes
 * sf = 2^(floor(log2(amax)) - 2) instead and saturates what then exceeds 6.  A block
 * whose amax is 2^-37 or less becomes zeros (the floor of 1e-10 keeps sf >= 2^-35).
 *   x      [rows, cols] bf16, f16 or f32, row stride x_ld; cols % 32 == 0
 *   codes  uint8 [rows, cols/2]   element k of a row in byte k/2, even k in the low nibble
 *   sf     uint8 [rows, cols/32]  UE8M0: 2^(code - 127)
 * A block holding an infinity or a NaN gets scale code 0xFF (NaN), so that
 * every value read from it is NaN.  codes 4-byte aligned.
 * 0 <= rows < 2^31, 32 <= cols < 2^24, rows * cols < 2^40.
 */
int moe_quantize_mxfp4(int32_t rows, int32_t cols, int32_t dtype, const void* x, int64_t x_ld,
                       uint8_t* codes, uint8_t* sf, void* stream);

/* The values the codes stand for, rounded to dtype (exact in bf16 and f32
 * above their subnormals): x [rows, cols], row stride x_ld.  Scale code
 * 0xFF gives NaN.  Ranges and alignment as for moe_quantize_mxfp4. */
int moe_dequantize_mxfp4(int32_t rows, int32_t cols, int32_t dtype, const uint8_t* codes,
                         const uint8_t* sf, void* x, int64_t x_ld, void* stream);

/*
 * Product of microscaled 4-bit matrices (the format above), f32 accumulation:
 *   y[r, n] = sum over k of a[r, k] * b[e, n, k]
 *   a     uint8 [rows, k/2], a_sf uint8 [rows, k/32]
 *   b     uint8 [groups, n, k/2], b_sf uint8 [groups, n, k/32]
 *   y     [rows, n] bf16, f16 or f32 (dtype), row stride y_ld, rounded once
 *         to nearest: a sum beyond the type's range becomes an infinity
 * Dense (offsets NULL, groups 1): every row.  Grouped: expert e's rows are
 * offsets[e] .. offsets[e] + counts[e] - 1 (counts NULL: up to
 * offsets[e + 1]), int32 device arrays as moe_route writes them; the rows of
 * y outside the segments (padding among them) are left as they were, and
 * a segment is cut at `rows`.  Segments do not overlap.  slots: an upper bound
 * of the counts' sum (T*K of the routing), for calls whose `rows` counts a
 * padded pool; it sizes the launch and picks the tile (if the counts hold more,
 * some of their rows are left as they were).  0: rows.  Calls without counts,
 * whose segments take in their padding, and dense ones ignore it.
 * k % 32 == 0, 32 <= k <= 2^20, groups <= 1024, rows < 2^28, n < 2^28.
 * Scale code 0xFF on a block makes the sums it enters NaN.  a and b 16-byte
 * aligned.  y must not overlap an input.  Products and block sums are exact
 * in the matrix instruction up to f32 rounding of its result; K is summed in
 * an order that depends on the tile a call takes (moe_gemm_mxfp4_info): of
 * calls with the same sizes, equal rows give equal bits.
 */
int moe_gemm_mxfp4(int32_t groups, int32_t rows, int32_t n, int32_t k, int32_t dtype,
                   const uint8_t* a, const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf,
                   const int32_t* offsets, const int32_t* counts, int32_t slots, void* y,
                   int64_t y_ld, void* stream);

/* Tile a moe_gemm_mxfp4 call of these sizes takes (host only): the rows and
 * columns of y per workgroup.  groups 0: dense; else that many segments, of
 * `rows` rows in all (a call's slots, if it states them).  Ranges as for
 * moe_gemm_mxfp4; MOE_ERR_INVALID_ARG also for a null output. */
int moe_gemm_mxfp4_info(int32_t groups, int32_t rows, int32_t n, int32_t k, int32_t* tile_m,
                        int32_t* tile_n);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
