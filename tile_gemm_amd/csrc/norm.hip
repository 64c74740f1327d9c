// The step between two blocks (hts_residual_norm): R' = R + scale * act(gate) * post(block),
// Y = pre(R').
//
// A row is held in registers as floats, 8 entries per chunk and thread, so it is read once and every
// statistic -- the post norm's, then the pre norm's over the sum -- is a reduction over registers; a
// layer norm's variance is summed around its mean.  Rows of up to 256 entries take 16 or 32 lanes of
// a wave (no barrier, 16 or 8 rows per workgroup); longer ones a workgroup each.
// Bound by HBM: block, R and a per-token gate in, R' and Y out, once each.  The outputs are written past the
// caches' normal lines (non-temporal): another XCD will read them, and the inputs keep their place (1000 x
// 16384: 21.1 us against 30.4 with ordinary stores).  16384 x 4096, layer norms on both sides and a sigmoid gate:
// 126 us, 5.3 TB/s (a copy of 4 GB reaches 4.8); 1 x 4096: 3.0 us.  Sums go by row moves within a wave and one
// barrier each (10 x 6568, two layer norms: a fifth less time than with shuffles through LDS and two barriers).
#include "serve_device.h"
#include "serve_internal.h"

namespace hts {
namespace {

template <int CTRL, int ROWS> __device__ __forceinline__ float add_moved(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xF, false));
}
// Sum over each row of 16 lanes, in every lane of it (row rotations by 8, 4, 2 and 1: no trip through LDS).
__device__ __forceinline__ float sum16(float x) {
    return add_moved<0x121, 0xF>(add_moved<0x122, 0xF>(add_moved<0x124, 0xF>(add_moved<0x128, 0xF>(x))));
}

// Sum over the threads of a row: LANES of a wave, or (LANES = 0) the whole workgroup, with one barrier: lds is used
// by one sum only.
template <int LANES> __device__ __forceinline__ float row_sum(float v, float* lds) {
    v = sum16(v);
    if (LANES == 16) return v;
    if (LANES == 32) return v + __shfl_xor(v, 16);
    v = add_moved<0x142, 0xA>(v);        // row 0's sum to row 1, row 2's to row 3
    v = add_moved<0x143, 0xC>(v);        // row 1's to rows 2 and 3: lane 63 has all
    const int waves = blockDim.x >> 6, lane = threadIdx.x & 63;
    if (waves > 1) {
        if (lane == 63) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        const float part = lds[lane & 15];
        v = sum16((lane & 15) < waves ? part : 0.0f);
    }
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

template <typename T, bool R32, int LANES, int CH>
__global__ __launch_bounds__(LANES ? 256 : 1024) void residual_norm_kernel(NormArgs a) {
    __shared__ float sums[4][16];        // a layer norm takes two sums, and there are two norms
    const int per_row = LANES ? LANES : blockDim.x, me = LANES ? threadIdx.x % LANES : threadIdx.x;
    const int64_t group = blockIdx.y * kGridX + blockIdx.x;
    const int64_t m = LANES ? group * (256 / LANES) + threadIdx.x / LANES : group;
    if (m >= a.M) return;                // rows of one wave end apart: their shuffles stay within a row
    float x[CH][8];
    // entry of chunk c; past the row's end a chunk holds zeros and stays out of the sums
    const auto col = [&](int c) { return (c * per_row + me) * 8; };
    const auto norm = [&](int kind, float eps, const uint16_t* w, const uint16_t* b, float (*lds)[16]) {
        const float inv_n = 1.0f / (float)a.N;
        // the weights' loads go out ahead of the sums
        u32x4 wv[CH], bv[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (w && col(c) < a.N) wv[c] = ld16(w + col(c));
            if (b && col(c) < a.N) bv[c] = ld16(b + col(c));
        }
        if (kind == HTS_NORM_LAYER) {
            float s = 0.0f;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += x[c][e];
            const float mean = row_sum<LANES>(s, lds[0]) * inv_n;
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (col(c) < a.N)
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[c][e] -= mean;
        }
        float q = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) q = fmaf(x[c][e], x[c][e], q);
        const float r = 1.0f / sqrtf(row_sum<LANES>(q, lds[1]) * inv_n + eps);
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (col(c) < a.N) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[c][e] *= r;
                if (w) {
                    widen8<T>(wv[c], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[c][e] *= f[e];
                }
                if (b) {
                    widen8<T>(bv[c], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[c][e] += f[e];
                }
            }
    };

    // everything the row needs is asked for at once
    u32x4 rv[CH][R32 ? 2 : 1], gv[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[c][e] = 0.0f;
        if (col(c) >= a.N) continue;
        if (a.block) widen8<T>(ld16(a.block + m * a.ldb + col(c)), x[c]);
        if (a.gate) gv[c] = ld16(a.gate + m * a.ldg + col(c));
        if (a.R) {
            const char* p = (const char*)a.R + (m * a.ldr + col(c)) * (R32 ? 4 : 2);
            rv[c][0] = ld16(p);
            if (R32) rv[c][R32 ? 1 : 0] = ld16(p + 16);
        }
    }
    if (a.post != HTS_NORM_NONE) norm(a.post, a.post_eps, a.post_w, a.post_b, sums);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if (col(c) >= a.N) continue;
        if (a.gate) {
            float g[8];
            widen8<T>(gv[c], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = g[e];
                if (a.gate_act != HTS_GATE_PLAIN) {
                    const float sg = 1.0f / (1.0f + expf(-v));
                    v = a.gate_act == HTS_GATE_SIGMOID ? sg : v * sg;
                }
                x[c][e] *= v;
            }
        }
        if (a.block)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[c][e] *= a.scale;
        if (a.R) {
            float r[8];
            if (R32) {
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] = __uint_as_float(rv[c][R32 ? e / 4 : 0][e & 3]);
            } else {
                widen8<T>(rv[c][0], r);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) x[c][e] += r[e];
        }
        if (a.R_out) {
            char* p = (char*)a.R_out + (m * a.ldro + col(c)) * (R32 ? 4 : 2);
            if (R32) {
                stream16(p, u32x4{__float_as_uint(x[c][0]), __float_as_uint(x[c][1]), __float_as_uint(x[c][2]),
                              __float_as_uint(x[c][3])});
                stream16(p + 16, u32x4{__float_as_uint(x[c][4]), __float_as_uint(x[c][5]), __float_as_uint(x[c][6]),
                                   __float_as_uint(x[c][7])});
            } else {
                stream16(p, narrow8<T>(x[c]));
            }
        }
    }
    if (!a.Y) return;
    if (a.pre != HTS_NORM_NONE) norm(a.pre, a.pre_eps, a.pre_w, a.pre_b, sums + 2);
#pragma unroll
    for (int c = 0; c < CH; ++c)
        if (col(c) < a.N) stream16(a.Y + m * a.ldy + col(c), narrow8<T>(x[c]));
}

template <typename T, bool R32>
hipError_t launch(const NormArgs& a, hipStream_t s) {
    const int chunks = a.N / 8;
    const auto rows_of = [&](int per) {
        const WideGrid wide = wide_grid((a.M + per - 1) / per);
        return dim3(wide.x, wide.rest);
    };
    const auto threads = [&](int ch) { return dim3((unsigned)(((chunks + ch - 1) / ch + 63) / 64 * 64)); };
    const dim3 grid = rows_of(1);
    // Lanes of a wave for short rows (65536 x 128: 11.8 us against 20.9 with a workgroup of one wave each, 65536 x 256:
    // 21.9 against 22.6).  Else one chunk per thread while the rows are few, for the shortest chain (1 x 4096:
    // 3.5 us against 3.8 with two; 2048 x 4096: 12.1 against 12.4), two for many (16384 x 4096 with gate and layer
    // norms: 144 against 160 with one), four past 8192 entries (1000 x 16384, two layer norms: 25.8 against 26.3 with
    // two; one RMS norm 21.1 and 20.8), but two in a small batch (10 x 15328: 6.8 against 7.2 with four; 64 x 16384: 7.1
    // and 7.7).  Replays of a graph, whose kernels follow one another: a large one takes longer there than by itself.
    const bool few = a.M <= 2048;
    if (chunks <= 16) residual_norm_kernel<T, R32, 16, 1><<<rows_of(16), 256, 0, s>>>(a);
    else if (chunks <= 32) residual_norm_kernel<T, R32, 32, 1><<<rows_of(8), 256, 0, s>>>(a);
    else if (chunks <= 256 || (few && chunks <= 1024)) residual_norm_kernel<T, R32, 0, 1><<<grid, threads(1), 0, s>>>(a);
    else if (chunks <= 1024 || (a.M <= 64 && chunks <= 2048))
        residual_norm_kernel<T, R32, 0, 2><<<grid, threads(2), 0, s>>>(a);
    else residual_norm_kernel<T, R32, 0, 4><<<grid, threads(4), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs& a, hipStream_t s) {
    if (a.dtype == HTS_BF16) return a.r32 ? launch<BF16T, true>(a, s) : launch<BF16T, false>(a, s);
    return a.r32 ? launch<F16T, true>(a, s) : launch<F16T, false>(a, s);
}

}  // namespace hts
