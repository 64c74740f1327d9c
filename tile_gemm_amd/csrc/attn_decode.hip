// Attention of one new token per request over a paged key-value cache (hts_paged_attn).
//
// s_t = scale q.k_t, O = sum e^(s_t - m) v_t / sum e^(s_t - m): one pass over the tokens with a
// running maximum m, sum l and accumulator, rescaled when the maximum grows.  One wave per request
// and query head; a lane holds four entries of the head.
#include "serve_device.h"
#include "serve_internal.h"

namespace hts {
namespace {

template <typename T> __device__ __forceinline__ void load4(const uint16_t* p, float* f) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    f[0] = widen<T>(v.x & 0xFFFFu);
    f[1] = widen<T>(v.x >> 16);
    f[2] = widen<T>(v.y & 0xFFFFu);
    f[3] = widen<T>(v.y >> 16);
}
template <typename T, bool C8> __device__ __forceinline__ void load_cache4(const void* base, int64_t off, float* f) {
    if (C8) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>((const uint8_t*)base + off);
        f[0] = __builtin_amdgcn_cvt_f32_fp8(w, 0);
        f[1] = __builtin_amdgcn_cvt_f32_fp8(w, 1);
        f[2] = __builtin_amdgcn_cvt_f32_fp8(w, 2);
        f[3] = __builtin_amdgcn_cvt_f32_fp8(w, 3);
    } else {
        load4<T>((const uint16_t*)base + off, f);
    }
}

template <typename T, bool C8>
__global__ __launch_bounds__(64) void attn_kernel(AttnArgs a) {
    const int b = blockIdx.x, h = blockIdx.y, hk = h / (a.q_heads / a.k_heads);
    const int d = threadIdx.x * 4;
    const bool on = d < a.dim;
    const int64_t cap = a.width << a.page_shift;
    const int64_t len = min((int64_t)max(a.lengths[b], 0), cap);
    const float sk = a.scale * (C8 && a.k_scale ? a.k_scale[hk] : 1.0f);
    float q[4] = {}, acc[4] = {}, m = -INFINITY, l = 0.0f;
    if (on) load4<T>(a.Q + b * a.ldq + (int64_t)h * a.dim + d, q);
    for (int64_t t = a.window ? max((int64_t)0, len - a.window) : 0; t < len; ++t) {
        const int64_t id = a.table[b * a.ldt + (t >> a.page_shift)];
        if (id < 0 || id >= a.pages) continue;
        const int64_t off = id * a.page_stride + (t & ((1 << a.page_shift) - 1)) * a.token_stride + hk * a.head_stride + d;
        float k[4] = {}, v[4] = {};
        if (on) {
            load_cache4<T, C8>(a.kc, off, k);
            load_cache4<T, C8>(a.vc, off, v);
        }
        const float s = wave_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]) * sk;
        const float top = fmaxf(m, s), ref = top == -INFINITY ? 0.0f : top;
        const float old = expf(m - ref), p = expf(s - ref);
        l = l * old + p;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = acc[e] * old + p * v[e];
        m = top;
    }
    const float sv = C8 && a.v_scale ? a.v_scale[hk] : 1.0f;
    const float inv = l == 0.0f ? 0.0f : sv / l;
    if (on) {
        uint16_t* o = a.O + b * a.ldo + (int64_t)h * a.dim + d;
        *reinterpret_cast<uint2*>(o) =
            uint2{narrow<T>(acc[0] * inv) | (narrow<T>(acc[1] * inv) << 16),
                  narrow<T>(acc[2] * inv) | (narrow<T>(acc[3] * inv) << 16)};
    }
    if (a.lse && threadIdx.x == 0) a.lse[(int64_t)b * a.q_heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.B, (unsigned)a.q_heads), block(64);
    if (a.dtype == HTS_BF16) {
        if (a.cache8) attn_kernel<BF16T, true><<<grid, block, 0, s>>>(a);
        else attn_kernel<BF16T, false><<<grid, block, 0, s>>>(a);
    } else {
        if (a.cache8) attn_kernel<F16T, true><<<grid, block, 0, s>>>(a);
        else attn_kernel<F16T, false><<<grid, block, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace hts
