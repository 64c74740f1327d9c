// The step between two blocks (hts_residual_norm): R' = R + scale * act(gate) * post(block),
// Y = pre(R').
//
// One workgroup per row.  A thread keeps its entries of the row (8 per chunk) in registers as
// floats, so the row is read once and every statistic -- the post norm's, then the pre norm's over
// the sum -- is a reduction over registers; a layer norm's variance is summed around its mean.
// Bound by HBM: block, R and a per-token gate in, R' and Y out, once each.
#include "serve_device.h"
#include "serve_internal.h"

namespace hts {
namespace {

// Sum over the NT threads of a row's workgroup.
template <int NT> __device__ __forceinline__ float row_sum(float v, float* lds) {
    v = wave_sum(v);
    if (NT == 64) return v;
    __syncthreads();                     // the last sum has been read by all
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) s += lds[w];
    return s;
}

// x -> norm(x) * w + b over the row (columns past N hold 0 and stay 0 in the sums).
template <typename T, int NT, int CH>
__device__ __forceinline__ void norm_row(float (&x)[CH][8], int kind, float eps, const uint16_t* w, const uint16_t* b,
                                         int N, float* lds) {
    const float inv_n = 1.0f / (float)N;
    if (kind == HTS_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) s += x[c][e];
        const float mean = row_sum<NT>(s, lds) * inv_n;
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if ((c * NT + (int)threadIdx.x) * 8 < N)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[c][e] -= mean;
    }
    float q = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(x[c][e], x[c][e], q);
    const float r = 1.0f / sqrtf(row_sum<NT>(q, lds) * inv_n + eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * NT + (int)threadIdx.x) * 8;
        if (col < N) {
            float wv[8], bv[8];
            if (w) widen8<T>(ld16(w + col), wv);
            if (b) widen8<T>(ld16(b + col), bv);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float y = x[c][e] * r;
                if (w) y *= wv[e];
                if (b) y += bv[e];
                x[c][e] = y;
            }
        }
    }
}

template <typename T, bool R32, int NT, int CH>
__global__ __launch_bounds__(NT) void residual_norm_kernel(NormArgs a) {
    __shared__ float lds[NT / 64];
    const int64_t m = blockIdx.x;
    float x[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * NT + (int)threadIdx.x) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[c][e] = 0.0f;
        if (a.block && col < a.N) widen8<T>(ld16(a.block + m * a.ldb + col), x[c]);
    }
    if (a.post != HTS_NORM_NONE) norm_row<T, NT, CH>(x, a.post, a.post_eps, a.post_w, a.post_b, a.N, lds);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * NT + (int)threadIdx.x) * 8;
        if (col < a.N) {
            if (a.gate) {
                float g[8];
                widen8<T>(ld16(a.gate + m * a.ldg + col), g);
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
                    const float* p = (const float*)a.R + m * a.ldr + col;
                    *reinterpret_cast<f32x4*>(r) = *reinterpret_cast<const f32x4*>(p);
                    *reinterpret_cast<f32x4*>(r + 4) = *reinterpret_cast<const f32x4*>(p + 4);
                } else {
                    widen8<T>(ld16((const uint16_t*)a.R + m * a.ldr + col), r);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) x[c][e] += r[e];
            }
            if (a.R_out) {
                if (R32) {
                    float* p = (float*)a.R_out + m * a.ldro + col;
                    *reinterpret_cast<f32x4*>(p) = f32x4{x[c][0], x[c][1], x[c][2], x[c][3]};
                    *reinterpret_cast<f32x4*>(p + 4) = f32x4{x[c][4], x[c][5], x[c][6], x[c][7]};
                } else {
                    st16((uint16_t*)a.R_out + m * a.ldro + col, narrow8<T>(x[c]));
                }
            }
        }
    }
    if (!a.Y) return;
    if (a.pre != HTS_NORM_NONE) norm_row<T, NT, CH>(x, a.pre, a.pre_eps, a.pre_w, a.pre_b, a.N, lds);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (c * NT + (int)threadIdx.x) * 8;
        if (col < a.N) st16(a.Y + m * a.ldy + col, narrow8<T>(x[c]));
    }
}

template <typename T, bool R32>
hipError_t launch(const NormArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.M);
    const int chunks = a.N / 8;
    if (chunks <= 64) residual_norm_kernel<T, R32, 64, 1><<<grid, 64, 0, s>>>(a);
    else if (chunks <= 256) residual_norm_kernel<T, R32, 256, 1><<<grid, 256, 0, s>>>(a);
    else if (chunks <= 512) residual_norm_kernel<T, R32, 256, 2><<<grid, 256, 0, s>>>(a);
    else if (chunks <= 1024) residual_norm_kernel<T, R32, 256, 4><<<grid, 256, 0, s>>>(a);
    else residual_norm_kernel<T, R32, 1024, 4><<<grid, 1024, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs& a, hipStream_t s) {
    if (a.dtype == HTS_BF16) return a.r32 ? launch<BF16T, true>(a, s) : launch<BF16T, false>(a, s);
    return a.r32 ? launch<F16T, true>(a, s) : launch<F16T, false>(a, s);
}

}  // namespace hts
