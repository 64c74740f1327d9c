// Block-scaled 8-bit product for few rows (M <= 32): the weights stream past the rows, and the sum of parts.
//
// A workgroup owns 16 outputs (the gated form: 16 gate rows and the same up rows) and KS waves; wave w takes the blocks
// w, w + KS, .. of K.  W and X go from global memory straight into the operands of the 16x16x128
// instruction, NT blocks of loads ahead of their use; each block's sum is multiplied by both scales and added in 32 bits.
// The waves' sums meet in LDS and are added in wave order.
//
// Bound by the weights' bytes: 1 x 11008 x 4096 with two weights, 90 MB, in 20.6 us, 4.4 TB/s (a streaming read of
// 131 MB: 5.8 to 6.1); its waves wait for data 55% of their cycles, the vector units are busy 15%.  A small one is latency: 1 x
// 4096 x 4096, 17 MB, 6.7 us, of which the bytes are 3.8.  Measured against this form (us): a wave's blocks in one contiguous
// run, no difference; loads that claim no place in the caches, none.
#include "scaled_device.h"

namespace hts {
namespace {

__device__ __forceinline__ u32x4 load16(rsrc_t r, uint32_t voff, uint32_t soff) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

// XT: the type of X.  HTS_FP8_E4M3: rows and scales as hts_quantize_rows makes them.  Others: every workgroup makes them
// itself, in LDS, while its first weights are on their way.
// WHOLE: no product loses bits (whole_sums; the rows that become E4M3 in the next launch are 32-bit here).
template <bool GATED, int KS, int NT, int MG, int XT, bool WHOLE>
__global__ __launch_bounds__(64 * KS) void scaled_stream_kernel(const ScaledArgs a) {
    constexpr int PP = GATED ? 2 : 1;
    constexpr bool MAKE = XT != HTS_FP8_E4M3;
    static_assert(!MAKE || MG == 1, "few rows");
    __shared__ f32x4 red[KS][MG * PP * 64];
    extern __shared__ __attribute__((aligned(16))) uint8_t made[];        // M rows of KB blocks, then their scales
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int KB = (int)((a.K + 127) / 128);
    const int rows = (int)(a.N - n0 < 16 ? a.N - n0 : 16);

    rsrc_t wr[PP];
    uint32_t wvo[PP];
#pragma unroll
    for (int p = 0; p < PP; ++p) {
        wr[p] = make_rsrc(a.W[p] + n0 * a.ldw[p], (uint32_t)((rows - 1) * a.ldw[p] + a.K));
        wvo[p] = (uint32_t)((i < rows ? i : rows - 1) * a.ldw[p]) + 16 * g;
    }
    const rsrc_t xr = make_rsrc(a.X, MAKE ? 0u : (uint32_t)((a.M - 1) * a.ldx + a.K));
    uint32_t xvo[MG];
    const float* xs[MG];
    float* made_s = reinterpret_cast<float*>(made + a.M * KB * 128);
#pragma unroll
    for (int h = 0; h < MG; ++h) {
        const int m = 16 * h + i < (int)a.M ? 16 * h + i : (int)a.M - 1;
        xvo[h] = MAKE ? (uint32_t)(m * KB * 128) + 16 * g : (uint32_t)(m * a.ldx) + 16 * g;
        xs[h] = MAKE ? made_s + m * KB : a.xs + m;
    }
    const int tail = (int)(a.K - (int64_t)128 * (KB - 1));
    const float* ws[PP];
#pragma unroll
    for (int p = 0; p < PP; ++p) ws[p] = a.ws[p] + n0 / 128 * a.ldws[p];

    f32x4 acc[MG][PP];
#pragma unroll
    for (int h = 0; h < MG; ++h)
#pragma unroll
        for (int p = 0; p < PP; ++p) acc[h][p] = f32x4{0.f, 0.f, 0.f, 0.f};

    u32x4 W[NT][PP][2], X[NT][MG][2];
    float sx[NT][MG], sw[NT][PP];
    auto load_w = [&](int t) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < NT; ++s) {
            if (t + KS * s >= KB) break;
            const int kb = t + KS * s;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bool out = kb == KB - 1 && 16 * (g + 4 * u) >= tail;
#pragma unroll
                for (int p = 0; p < PP; ++p) W[s][p][u] = load16(wr[p], out ? kOutside : wvo[p] + 64 * u, 128u * kb);
            }
#pragma unroll
            for (int p = 0; p < PP; ++p) sw[s][p] = ws[p][kb];
        }
    };
    auto load_x = [&](int s, int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < MG; ++h) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if constexpr (MAKE) X[s][h][u] = ld16(made + xvo[h] + 128 * kb + 64 * u);
                else X[s][h][u] = load16(xr, kb == KB - 1 && 16 * (g + 4 * u) >= tail ? kOutside : xvo[h] + 64 * u, 128u * kb);
            }
            sx[s][h] = xs[h][MAKE ? kb : kb * a.ldxs];
        }
    };
    if constexpr (MAKE) {
        // eight lanes to a block, as in hts_quantize_rows; columns past K are zeros
        load_w(wave);
        constexpr int ES = XT == HTS_F32 ? 4 : 2;
        for (int id = threadIdx.x >> 3; id < (int)a.M * KB; id += 8 * KS) {
            const int m = id / KB, kb = id % KB, c = kb * 128 + 16 * (threadIdx.x & 7);
            float f[16] = {};
            if (c < a.K) load_values16<XT>(a.X + m * a.ldx * ES, c, f);
            const float top = block_top(f);
            st16(made + (int64_t)id * 128 + 16 * (threadIdx.x & 7), scaled16(f, kE4m3Max / top));
            if ((threadIdx.x & 7) == 0) made_s[id] = top / kE4m3Max;
        }
        __syncthreads();
    }
    for (int t = wave; t < KB; t += NT * KS) {
        if (!MAKE || t != wave) load_w(t);
        if (!MAKE)
#pragma unroll
            for (int s = 0; s < NT; ++s) {
                if (t + KS * s >= KB) break;
                load_x(s, t + KS * s);
            }
#pragma unroll
        for (int s = 0; s < NT; ++s) {
            if (t + KS * s >= KB) break;
            if (MAKE) load_x(s, t + KS * s);           // from LDS, and only then: 16 registers fewer
#pragma unroll
            for (int h = 0; h < MG; ++h)
#pragma unroll
                for (int p = 0; p < PP; ++p) {
                    const u32x8 w = cat8(W[s][p][0], W[s][p][1]), x = cat8(X[s][h][0], X[s][h][1]);
                    const f32x4 v = WHOLE ? mfma_block_whole(e4m3_halves(w), e4m3_halves(x)) : mfma_block(w, x);
                    const float sc = sx[s][h] * sw[s][p];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[h][p][e] = __builtin_fmaf(v[e], sc, acc[h][p][e]);
                }
        }
    }
#pragma unroll
    for (int h = 0; h < MG; ++h)
#pragma unroll
        for (int p = 0; p < PP; ++p) red[wave][(h * PP + p) * 64 + lane] = acc[h][p];
    __syncthreads();
    // output (row m, column r of the 16): four columns of a row lie in one lane's f32x4
    for (int o = threadIdx.x; o < MG * 64; o += 64 * KS) {
        const int h = o >> 6, l = o & 63;
        f32x4 sum[PP];
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            sum[p] = red[0][(h * PP + p) * 64 + l];
#pragma unroll
            for (int w = 1; w < KS; ++w) {
                const f32x4 v = red[w][(h * PP + p) * 64 + l];
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[p][e] += v[e];
            }
        }
        const int64_t m = 16 * h + (l & 15), n = n0 + 4 * (l >> 4);
        if (m >= a.M || n >= a.N) continue;
        if (a.part) {                  // the gated sums as one part, for E4M3 rows
#pragma unroll
            for (int p = 0; p < PP; ++p) *reinterpret_cast<f32x4*>(a.part + (p * a.M + m) * a.ldp + n) = sum[p];
            continue;
        }
        if constexpr (GATED)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[0][e] = act_value(a.act, sum[0][e]) * sum[1][e];
        store_upto4(a.Y, m * a.ldy + n, a.N - n, a.y_dtype, sum[0]);
    }
}

// Parts of a product in part order, the gate, and the output's type.  32 lanes to a row's block of 128 columns.
template <bool GATED>
__global__ __launch_bounds__(256) void scaled_sum_kernel(const ScaledArgs a, int64_t NBK) {
    const int64_t id = (blockIdx.y * kGridX + blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t m = id / NBK, nb = id % NBK;
    if (m >= a.M) return;
    const int64_t n = nb * 128 + 4 * (threadIdx.x & 31);
    const bool in = n < a.N;
    constexpr int PP = GATED ? 2 : 1;
    f32x4 sum[PP];
#pragma unroll
    for (int p = 0; p < PP; ++p) sum[p] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (in)
        for (int k = 0; k < a.nsplit; ++k)
#pragma unroll
            for (int p = 0; p < PP; ++p) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(a.part + (((int64_t)k * PP + p) * a.M + m) * a.ldp + n);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[p][e] = k ? sum[p][e] + v[e] : v[e];
            }
    if constexpr (GATED)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[0][e] = n + e < a.N ? act_value(a.act, sum[0][e]) * sum[1][e] : 0.f;
    if (a.y_dtype == HTS_FP8_E4M3) {
        float t = kLeastTop;
#pragma unroll
        for (int e = 0; e < 4; ++e) t = fmaxf(t, fabsf(sum[0][e]));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor(t, o));
        const float r = kE4m3Max / t;
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = sum[0][e] * r;
        if (in) *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.Y) + m * a.ldy + n) = narrow4_e4m3(f);
        if ((threadIdx.x & 31) == 0) a.ys[nb * a.ldys + m] = t / kE4m3Max;
        return;
    }
    if (in) store_upto4(a.Y, m * a.ldy + n, a.N - n, a.y_dtype, sum[0]);
}

constexpr int kWaves = 8;
// Four blocks of loads ahead where a wave has as many (4096 x 11008, one row: 12.1 us against 12.5 with one ahead); below, they
// would not all be used, and their registers cost waves.
inline bool far_ahead(int64_t K) { return K > kWaves * 4 * 128; }

template <bool GATED, int NT, int MG, int XT, bool WHOLE>
hipError_t launch_rows(const ScaledArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.N + 15) / 16)), block(64 * kWaves);
    const size_t lds = XT == HTS_FP8_E4M3 ? 0 : a.M * scale_blocks(a.K) * (128 + 4);
    scaled_stream_kernel<GATED, kWaves, NT, MG, XT, WHOLE><<<grid, block, lds, s>>>(a);
    return hipGetLastError();
}
template <bool GATED, int MG, int XT = HTS_FP8_E4M3, bool WHOLE = false>
hipError_t launch_mg(const ScaledArgs& a, hipStream_t s) {
    return far_ahead(a.K) ? launch_rows<GATED, 4, MG, XT, WHOLE>(a, s) : launch_rows<GATED, 1, MG, XT, WHOLE>(a, s);
}

}  // namespace

hipError_t launch_scaled_stream(const ScaledArgs& a, hipStream_t s) {
    if (a.M > kScaledStreamRows || (a.y_dtype == HTS_FP8_E4M3 && !a.part)) return hipErrorInvalidValue;
    constexpr int E4M3 = HTS_FP8_E4M3;
    if (whole_sums(a.y_dtype)) {
        // two weights: one block ahead at any K (E4M3 rows, 1 x 13824 x 5120: 34.2 us, 41.2 with four)
        if (a.gated) return a.M <= 16 ? launch_rows<true, 1, 1, E4M3, true>(a, s) : launch_rows<true, 1, 2, E4M3, true>(a, s);
        return a.M <= 16 ? launch_mg<false, 1, E4M3, true>(a, s) : launch_mg<false, 2, E4M3, true>(a, s);
    }
    if (a.gated) return a.M <= 16 ? launch_mg<true, 1>(a, s) : launch_mg<true, 2>(a, s);
    return a.M <= 16 ? launch_mg<false, 1>(a, s) : launch_mg<false, 2>(a, s);
}

hipError_t launch_scaled_stream_made(const ScaledArgs& a, int32_t x_dtype, hipStream_t s) {
    if (a.M > kMadeRows || a.M * scale_blocks(a.K) > kMadeBlocks || a.part || a.y_dtype == HTS_FP8_E4M3) return hipErrorInvalidValue;
    if (a.gated) return x_dtype == HTS_BF16 ? launch_mg<true, 1, HTS_BF16, true>(a, s) : launch_mg<true, 1, HTS_F16, true>(a, s);
    return launch_mg<false, 1, HTS_F32>(a, s);
}

hipError_t launch_scaled_sum(const ScaledArgs& a, hipStream_t s) {
    const int64_t NBK = scale_blocks(a.N);
    const WideGrid wide = wide_grid((a.M * NBK + 7) / 8);
    const dim3 grid(wide.x, wide.rest), block(256);
    if (a.gated) scaled_sum_kernel<true><<<grid, block, 0, s>>>(a, NBK);
    else scaled_sum_kernel<false><<<grid, block, 0, s>>>(a, NBK);
    return hipGetLastError();
}

}  // namespace hts
