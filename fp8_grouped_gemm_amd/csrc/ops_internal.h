// Internal interface between the host entry points of the row operators
// (ops_api.cpp) and their kernels.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Row permutation and its relatives.  Strides in bytes.
struct RowsArgs {
    int32_t T, K, R;           // tokens, slots per token, pool rows
    int32_t width;             // elements per row
    int32_t dtype;             // MOE_DTYPE_*
    const char* tok;           // token-order rows read: x, dy
    const char* pool;          // pool rows read: dxp, yp
    char* tok_out;             // token-order rows written: dx, y
    char* pool_out;            // pool rows written: xp, dyp
    int64_t tok_ld, pool_ld, pool_out_ld;  // (tok_ld serves tok or tok_out)
    const int32_t* row_src;
    const int32_t* src_row;
    const int32_t* used;       // may be null: R
    const float* w;            // [T*K], may be null: 1
    float* dw;                 // [T*K]
};

struct MxQuantArgs {
    int32_t rows, cols, dtype;
    char* x;                   // read by quantisation, written by dequantisation
    int64_t ld;                // bytes
    uint8_t* codes;
    uint8_t* sf;
};

struct MxGemmArgs {
    int32_t E, R, N, K;
    int32_t slots;             // most rows of all segments together (dense: R)
    int32_t dtype;
    const uint8_t* a;
    const uint8_t* a_sf;
    const uint8_t* b;
    const uint8_t* b_sf;
    const int32_t* offsets;    // null: dense
    const int32_t* counts;     // may be null
    char* y;
    int64_t y_ld;              // bytes
};

hipError_t launch_permute(const RowsArgs& a, hipStream_t s);
hipError_t launch_unpermute(const RowsArgs& a, hipStream_t s);  // also permute's gradient
hipError_t launch_unpermute_bwd(const RowsArgs& a, hipStream_t s);
hipError_t launch_quantize_mxfp4(const MxQuantArgs& a, hipStream_t s);
hipError_t launch_dequantize_mxfp4(const MxQuantArgs& a, hipStream_t s);
hipError_t launch_gemm_mxfp4(const MxGemmArgs& a, hipStream_t s);
// Tile of a call (host only): only E, R, N, K and whether it is grouped count.
void gemm_mxfp4_tile(int E, int R, int N, int K, bool grouped, int& bm, int& bn);

// A launch takes fewer than 2^32 threads along an axis: of its workgroups (up to
// 1024 threads each), numbered through, those from 2^kGridBits on go along y.
// The grid is whole rows of them, so a kernel ignores numbers past its last.
constexpr int kGridBits = 21;

inline dim3 grid_of(int64_t wgs)
{
    const int64_t row = INT64_C(1) << kGridBits;
    return wgs <= row ? dim3((unsigned)wgs) : dim3((unsigned)row, (unsigned)((wgs + row - 1) / row));
}

__device__ __forceinline__ unsigned workgroup() { return (blockIdx.y << kGridBits) + blockIdx.x; }

// MOE_OK if the current device is gfx950 (moe_api.cpp).
int device_status();

}  // namespace moe
