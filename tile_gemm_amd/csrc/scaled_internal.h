// Internal declarations shared by the block-scaled 8-bit half of the C API and its gfx950 kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hts.h"
#include "serve_internal.h"

namespace hts {

constexpr int kScaleBlock = 128;
inline int64_t scale_blocks(int64_t n) { return (n + kScaleBlock - 1) / kScaleBlock; }

// Rows to E4M3.  rows 1: a scale for each row and block at S[block * lds + row]; rows 128: one for each 128 x 128 block
// at S[row / 128 * lds + block].
struct QuantArgs {
    int32_t dtype;
    int64_t M, K;
    const void* X;
    int64_t ldx;
    uint8_t* Q;
    int64_t ldq;
    float* S;
    int64_t lds;
};
hipError_t launch_quantize_rows(const QuantArgs& a, hipStream_t s);
hipError_t launch_quantize_weight(const QuantArgs& a, hipStream_t s);

// One block-scaled product, or the gated pair of them.
struct ScaledArgs {
    int64_t M, N, K;
    const uint8_t* X;
    int64_t ldx;
    const float* xs;           // [blocks of K][ldxs], entry m
    int64_t ldxs;
    const uint8_t* W[2];       // the weight, or gate and up
    int64_t ldw[2];
    const float* ws[2];        // [blocks of N][ldws], entry = block of K
    int64_t ldws[2];
    int32_t act;               // HTS_ACT_* (gated)
    int32_t gated;
    void* Y;
    int64_t ldy;
    int32_t y_dtype;           // HTS_F32, HTS_F16, HTS_BF16, or HTS_FP8_E4M3 with ys (gated)
    float* ys;                 // [blocks of N][ldys], entry m
    int64_t ldys;
    // part not NULL: the blocks of K are cut into nsplit parts, the 32-bit sums of part p and weight w go to
    // part[(p * weights + w) * M * ldp], and launch_scaled_sum makes Y of them
    float* part;
    int64_t ldp;
    int32_t nsplit;
};

// Whether no product of the sums may lose bits.  The 8-bit matrix instruction is off by 1.5e-5 of a result's norm, a
// hundredth of a bfloat16 rounding and a fourteenth of a binary16 one, and a hundred times what 32-bit sums are off by: an
// HTS_F32 output would show all of it.  A value that becomes E4M3 lands on the other
// neighbour, an eighth of itself away, where it lies that near a tie: one in a few thousand does, and a feed-forward part in
// binary16 is then 1e-3 of its norm from its definition, five times its rounding.
inline bool whole_sums(int32_t y_dtype) { return y_dtype == HTS_F32 || y_dtype == HTS_FP8_E4M3; }

// The kernels of a product.  Streaming: 16 outputs a workgroup, up to kScaledStreamRows rows.  RING_*, TILE_*: rows of W
// (gated: half of them gate, half up) x rows of X a workgroup.
constexpr int64_t kScaledStreamRows = 32;
enum ScaledKernel {
    SCALED_STREAM = 0,
    RING_32x16, RING_64x16, RING_32x32, RING_64x32, RING_64x64, RING_128x64, RING_128x128,
    TILE_128x128, TILE_256x128, TILE_256x256,
    SCALED_KERNELS
};
// One whose workgroups hold whole blocks of 128 outputs makes E4M3 rows itself; the others leave their sums in a.part.
// (TILE_256x256 has no whole sums: its accumulators and converted operands are more than a wave's registers.)
inline bool writes_e4m3(ScaledKernel k) { return k == TILE_256x128; }
hipError_t launch_scaled_stream(const ScaledArgs& a, hipStream_t s);
// The same on rows that its workgroups make themselves (a.X in x_dtype, a.xs unused): gated of HTS_F16 or HTS_BF16 rows, plain
// of HTS_F32 rows.  Few rows, and few blocks of them: they lie in LDS.
constexpr int64_t kMadeRows = 4, kMadeBlocks = 384;
hipError_t launch_scaled_stream_made(const ScaledArgs& a, int32_t x_dtype, hipStream_t s);
hipError_t launch_scaled_ring(const ScaledArgs& a, ScaledKernel k, hipStream_t s);
hipError_t launch_scaled_tile(const ScaledArgs& a, ScaledKernel k, hipStream_t s);
// The sum of a.nsplit parts, gated and rounded to Y.
hipError_t launch_scaled_sum(const ScaledArgs& a, hipStream_t s);

}  // namespace hts
