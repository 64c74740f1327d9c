// Rows and weights to E4M3 values with a 32-bit scale for each block of 128.
//
//   a = max(max |x|, 2^-100) over the block,   s = a / 448,   q = E4M3(x * (448 / a))
//
// Each quotient and product is one 32-bit operation, rounded to nearest; E4M3 rounds to nearest even and x * (448 / a)
// stays within 448 up to its last bit.  NaN counts for nothing in a and stays NaN; an infinity makes s infinite and the
// block's finite values 0.
#include "scaled_device.h"

namespace hts {
namespace {

// Eight lanes to a block of a row, 16 values each.  A workgroup takes 8 rows by 4 blocks: 1 KB of a 16-bit row in one piece,
// and 8 scales, which lie together, in one (4-byte writes on their own cost 32 bytes of traffic each).  Bound by memory:
// 16384 x 13824 bfloat16 in 124.6 us, 686 MB at 5.5 TB/s (a copy of 2 GiB: 4.9 TB/s).  32 blocks along a row in place of
// 8 x 4 (us): 16384 x 13824 125.1 : 124.6, 16384 x 4096 40.8 : 37.7, 2048 x 4096 7.4 : 6.9, 1 x 4096 2.4 : 2.6.
template <int DT>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const QuantArgs a, int64_t KB) {
    const int64_t id = blockIdx.y * kGridX + blockIdx.x, K4 = (KB + 3) / 4;
    const int b = threadIdx.x >> 3;
    const int64_t m = id / K4 * 8 + (b >> 2), kb = id % K4 * 4 + (b & 3);
    if (m >= a.M || kb >= KB) return;
    const int64_t c = kb * kScaleBlock + 16 * (threadIdx.x & 7);
    const bool in = c < a.K;
    float f[16] = {};
    constexpr int ES = DT == HTS_F32 ? 4 : 2;
    if (in) load_values16<DT>(static_cast<const uint8_t*>(a.X) + m * a.ldx * ES, c, f);
    const float t = block_top(f);
    if (in) st16(a.Q + m * a.ldq + c, scaled16(f, kE4m3Max / t));
    if ((threadIdx.x & 7) == 0) a.S[kb * a.lds + m] = t / kE4m3Max;
}

// A workgroup to a 128 x 128 block: eight lanes to a row, 32 rows at a time.  Bound by memory: 13824 x 5120 bfloat16 in 43.8 us, 212
// MB at 4.8 TB/s; 4096 x 4096 14.2 us.
template <int DT>
__global__ __launch_bounds__(256) void quantize_weight_kernel(const QuantArgs a, int64_t KB) {
    __shared__ float wave_top[4];
    const int64_t id = blockIdx.y * kGridX + blockIdx.x;
    const int64_t nb = id / KB, kb = id % KB;
    if (nb * kScaleBlock >= a.M) return;
    const int64_t c = kb * kScaleBlock + 16 * (threadIdx.x & 7);
    const int64_t row0 = nb * kScaleBlock + (threadIdx.x >> 3);
    constexpr int ES = DT == HTS_F32 ? 4 : 2;
    float f[4][16] = {};
    float t = 0.f;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const int64_t n = row0 + 32 * v;
        if (n < a.M && c < a.K) load_values16<DT>(static_cast<const uint8_t*>(a.X) + n * a.ldx * ES, c, f[v]);
        t = fmaxf(t, top16(f[v]));
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) t = fmaxf(t, __shfl_xor(t, o));
    if ((threadIdx.x & 63) == 0) wave_top[threadIdx.x >> 6] = t;
    __syncthreads();
    t = fmaxf(fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3])), kLeastTop);
    const float r = kE4m3Max / t;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const int64_t n = row0 + 32 * v;
        if (n < a.M && c < a.K) st16(a.Q + n * a.ldq + c, scaled16(f[v], r));
    }
    if (threadIdx.x == 0) a.S[nb * a.lds + kb] = t / kE4m3Max;
}

}  // namespace

hipError_t launch_quantize_rows(const QuantArgs& a, hipStream_t s) {
    const int64_t KB = scale_blocks(a.K);
    const WideGrid wide = wide_grid((a.M + 7) / 8 * ((KB + 3) / 4));
    const dim3 grid(wide.x, wide.rest), block(256);
    if (a.dtype == HTS_F32) quantize_rows_kernel<HTS_F32><<<grid, block, 0, s>>>(a, KB);
    else if (a.dtype == HTS_BF16) quantize_rows_kernel<HTS_BF16><<<grid, block, 0, s>>>(a, KB);
    else quantize_rows_kernel<HTS_F16><<<grid, block, 0, s>>>(a, KB);
    return hipGetLastError();
}

hipError_t launch_quantize_weight(const QuantArgs& a, hipStream_t s) {
    const int64_t KB = scale_blocks(a.K);
    const WideGrid wide = wide_grid(scale_blocks(a.M) * KB);
    const dim3 grid(wide.x, wide.rest), block(256);
    if (a.dtype == HTS_F32) quantize_weight_kernel<HTS_F32><<<grid, block, 0, s>>>(a, KB);
    else if (a.dtype == HTS_BF16) quantize_weight_kernel<HTS_BF16><<<grid, block, 0, s>>>(a, KB);
    else quantize_weight_kernel<HTS_F16><<<grid, block, 0, s>>>(a, KB);
    return hipGetLastError();
}

}  // namespace hts
