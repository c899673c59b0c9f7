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
 *     row segments of the experts;
 *   - moe_gate: the router's choice of experts and their weights, from its
 *     logits, with the gradient;
 *   - moe_rms_norm: the residual's addition and a root-mean-square norm, in the
 *     rows' type and in 8 bits, with the gradients;
 *   - moe_swiglu: the activation between the experts' two products, in the rows'
 *     type and in 8 bits, with an 8-bit copy of its input and the gradient
 *     that reads that copy;
 *   - moe_gemm_wgrad: the experts' weight gradients from rows kept in 8 bits.
 *
 * Conventions as in moe_fp8.h: device pointers owned by the caller, no
 * allocation, no host synchronisation, work enqueued on `stream` of the
 * current device, every argument checked on the host before any HIP call,
 * MOE_OK or a negative MOE_ERR_* code returned.  What differs: no plan (the
 * shapes are arguments), no workspace but where an entry point names one (its
 * size is a host-side query; calls that overlap need one each, and nothing in it
 * has to be set or is kept), and the matrices of bf16 / f16 / f32
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

/*
 * The router's choice.  For token t with logits l = logits[t], over experts e:
 *   s = softmax(l) or 1 / (1 + exp(-l));  c = s + bias, or without a bias the order of l
 *   (the softmax's own order, and the sigmoid's also where it saturates)
 *   groups > 1: the E / groups adjacent experts of a group stand for it with the
 *   sum of their group_top largest c (group_top 1 without a bias: the largest l; 2 and
 *   more: of s), and only the experts of the top_groups best groups are chosen from
 *   topk_idx[t] = the K largest c, largest first
 *   topk_w[t, j] = scale * s[i_j] / (sum over j of s[i_j] + 1e-20) with renorm, scale * s[i_j]
 *                  without
 * Equal values: the lower id (or group) first.  c and the groups' sums are formed in
 * 64 bits, so that near neighbours keep their order; weights are f32.
 * An expert whose logit or bias is -infinity is never chosen; slots left without an
 * expert are -1 with weight 0 (moe_route's masked slots), and a group without
 * any expert comes last.  A token whose mask is 0 gets -1 and 0 throughout and its
 * logits are not read.  A NaN counts as the largest value; it makes its own weight
 * NaN, and with softmax or renorm the token's.
 *   logits   [T, E]  bf16, f16 or f32, row stride logits_ld
 *   bias     f32 [E], may be null;  mask uint8 [T], may be null
 *   score    MOE_SCORE_*;  groups 1: none (top_groups is then 1, group_top without effect)
 *   topk_idx int32 [T, K], topk_w f32 [T, K]: what moe_forward and moe_route take
 * 1 <= E <= 1024, 1 <= K <= 64, K <= E / groups * top_groups, E % groups == 0,
 * groups <= 64, group_top <= E / groups, T < 2^28.  T == 0 is a no-op.  Outputs
 * overlap nothing.
 */
#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1
int moe_gate(int32_t num_tokens, int32_t num_experts, int32_t top_k, int32_t dtype,
             const void* logits, int64_t logits_ld, const float* bias, const uint8_t* mask,
             int32_t score, int32_t groups, int32_t top_groups, int32_t group_top, int32_t renorm,
             float scale, int32_t* topk_idx, float* topk_w, void* stream);

/*
 * Gradient of moe_gate's weights with respect to the logits, the choice fixed
 * (bias, groups and mask have done their part in it):
 *   dlogits[t, e] = sum over j of dw[t, j] * d topk_w[t, j] / d l[e]
 * over the slots with 0 <= topk_idx < E (the others' dw counts for nothing); a token
 * with no such slot gets zeros whatever its logits are.  A slot's expert may be
 * named twice.  dlogits [T, E] in the logits' type, rounded once from f32.
 * Ranges as for moe_gate.  dlogits overlaps nothing.
 */
int moe_gate_bwd(int32_t num_tokens, int32_t num_experts, int32_t top_k, int32_t dtype,
                 const void* logits, int64_t logits_ld, const int32_t* topk_idx, const float* dw,
                 int32_t score, int32_t renorm, float scale, void* dlogits, int64_t dlogits_ld,
                 void* stream);

/* Scale formats of 8-bit rows (e4m3 codes), as moe_quantize_act writes them. */
#define MOE_SF_F32_128 0  /* f32 per 128 columns: max(amax, 1e-10) / 448 */
#define MOE_SF_UE8M0_32 1 /* uint8 per 32 columns: the smallest power of two >= that, 2^(c - 127) */

/*
 * Residual and norm of token rows:
 *   z = x + residual (rounded to the type; no residual: x),  rstd = (mean(z^2) + eps)^(-1/2)
 *   y = z * rstd * weight
 *   x, residual, z, y  [rows, width] bf16, f16 or f32 (dtype); residual may be null
 *   weight  [width] of type w_dtype (dtype or f32), null: 1
 *   z       written, needs residual (null: not written; z may be x or residual itself)
 *   rstd    f32 [rows], written unless null
 *   y       written unless null (may be x, or residual, itself, if z is not)
 *   codes   uint8 [rows, width] e4m3 and sf [rows, width / 128] f32 or [rows, width / 32]
 *           uint8, by sf_format: y in 8 bits, quantised from the f32 values by
 *           moe_quantize_act's rule, moe_forward's x and x_sf; both null: not written
 * At least one of y and codes.  Sums are f32.  rows < 2^28, 1 <= width < 2^24, with
 * codes width % 128 == 0 (MOE_SF_UE8M0_32: % 32); codes 8-byte, sf 4-byte aligned
 * (UE8M0: any).  rows == 0 is a no-op.  "Itself": the same address and row stride;
 * outputs overlap nothing else.
 */
int moe_rms_norm(int32_t rows, int32_t width, int32_t dtype, const void* x, int64_t x_ld,
                 const void* residual, int64_t residual_ld, const void* weight, int32_t w_dtype,
                 float eps, void* z, int64_t z_ld, float* rstd, void* y, int64_t y_ld,
                 uint8_t* codes, void* sf, int32_t sf_format, void* stream);

/*
 * Gradients of moe_rms_norm for dy [rows, width], through the stored z and rstd
 * (8-bit rows pass their gradient straight through):
 *   xh = z * rstd,  g = dy * weight
 *   dx = rstd * (g - xh * mean(g * xh)) + dz   (the gradient of x and of residual alike)
 *   dw[k] = sum over rows of dy * xh, f32 [width]
 * dz [rows, width]: the gradient that reaches z on its other way, null: 0.  dx in
 * dtype, rounded once, may be dy or dz itself; null: not computed.  dw null: not
 * computed; else workspace holds moe_rms_norm_bwd_workspace_bytes.  rows == 0
 * makes dw zeros.  At least one of dx and dw.  workspace 16-byte aligned,
 * overlapping nothing.
 */
int moe_rms_norm_bwd(int32_t rows, int32_t width, int32_t dtype, const void* dy, int64_t dy_ld,
                     const void* z, int64_t z_ld, const void* weight, int32_t w_dtype,
                     const float* rstd, const void* dz, int64_t dz_ld, void* dx, int64_t dx_ld,
                     float* dw, void* workspace, size_t workspace_bytes, void* stream);
int moe_rms_norm_bwd_workspace_bytes(int32_t rows, int32_t width, size_t* bytes);

/*
 * The activation between the experts' two products, per pool row:
 *   h = silu(g) * u,  g = gu[:, :inner], u = gu[:, inner:], both clamped to [-clamp, clamp]
 *   first if clamp > 0
 *   gu       [pool_rows, 2 inner] bf16, f16 or f32
 *   row_src  int32 [pool_rows], moe_route's: rows with an entry < 0 are padding; null: none
 *   used     int32 [1]: pool rows in use (moe_route's offsets + E); null: all
 *   h        [pool_rows, inner] in dtype, rounded once from f32; null: not written
 *   h_codes, h_sf    h in 8 bits, from the f32 values: the second product's rows, and what
 *                    moe_gemm_wgrad takes for its weights; null: not written
 *   gu_codes, gu_sf  gu (not clamped) in 8 bits [pool_rows, 2 inner]: what
 *                    moe_swiglu_bwd needs, at half of gu's bytes or less; null: not written
 * Padding rows and rows from *used on are not read, and left as they were in every
 * output.  Of h, h_codes and gu_codes at least one.  pool_rows < 2^28, 1 <= inner <
 * 2^23, with codes inner % 128 == 0 (MOE_SF_UE8M0_32: % 32); codes 8-byte, sf
 * 4-byte aligned (UE8M0: any).  Outputs overlap nothing.
 */
int moe_swiglu(int32_t pool_rows, int32_t inner, int32_t dtype, const void* gu, int64_t gu_ld,
               float clamp, const int32_t* row_src, const int32_t* used, void* h, int64_t h_ld,
               uint8_t* h_codes, void* h_sf, uint8_t* gu_codes, void* gu_sf, int32_t sf_format,
               void* stream);

/*
 * Gradient of moe_swiglu for dh [pool_rows, inner]: with sg = 1 / (1 + exp(-g))
 *   dgu[:, :inner] = dh * u * sg * (1 + g * (1 - sg)),  dgu[:, inner:] = dh * g * sg
 * and 0 where g, or u, lies outside [-clamp, clamp] (clamp > 0; the other factor
 * is the clamped one).  The input is gu, or the 8-bit copy gu_codes and gu_sf
 * (exactly one of the two; the gradient is then taken at the values the codes stand for).
 * dgu [pool_rows, 2 inner] in dtype, rounded once; it may be gu itself.  Rows
 * and ranges as for moe_swiglu.
 */
int moe_swiglu_bwd(int32_t pool_rows, int32_t inner, int32_t dtype, const void* dh, int64_t dh_ld,
                   const void* gu, int64_t gu_ld, const uint8_t* gu_codes, const void* gu_sf,
                   int32_t sf_format, float clamp, const int32_t* row_src, const int32_t* used,
                   void* dgu, int64_t dgu_ld, void* stream);

/*
 * Weight gradients from rows kept in 8 bits:
 *   dw[e, i, k] = sum over the rows r of expert e of dy[r, i] * x[r, k]
 *   dy     [rows, n] bf16 or f16 (dtype), row stride dy_ld, here at most 2^24
 *   x      uint8 [rows, k] e4m3, x_sf by sf_format: x[r, k] = the f32 product code * scale,
 *          rounded to dy's type (exact in bf16 with UE8M0 scales above its subnormals)
 *   dw     [groups, n, k] bf16, f16 or f32 (dw_dtype), densely packed, rounded once from f32
 * Segments as in moe_gemm_mxfp4: offsets null: dense, groups 1, every row; else
 * expert e's rows are offsets[e] .. offsets[e] + counts[e] - 1 (counts null: up to
 * offsets[e + 1]), cut at `rows`; rows outside are not read.  An expert without rows gets
 * zeros.  accumulate: dw is added to (the stored value plus the f32 sum, rounded once) in
 * place of overwritten; an expert without rows keeps its values.
 * workspace holds moe_gemm_wgrad_workspace_bytes of these sizes (0 for most: null then;
 * the rows of few experts are split over workgroups, whose sums meet there in a fixed order).
 * k % 32 == 0 (MOE_SF_F32_128: % 128), 1 <= k <= 2^20, groups <= 1024, rows < 2^28,
 * n < 2^20.  x and workspace 16-byte aligned, x_sf 4-byte (UE8M0: any).
 * Outputs overlap nothing.  Equal calls give equal bits.
 */
int moe_gemm_wgrad(int32_t groups, int32_t rows, int32_t n, int32_t k, int32_t dtype,
                   const void* dy, int64_t dy_ld, const uint8_t* x, const void* x_sf,
                   int32_t sf_format, const int32_t* offsets, const int32_t* counts,
                   int32_t accumulate, void* dw, int32_t dw_dtype, void* workspace,
                   size_t workspace_bytes, void* stream);
int moe_gemm_wgrad_workspace_bytes(int32_t groups, int32_t rows, int32_t n, int32_t k,
                                   size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
