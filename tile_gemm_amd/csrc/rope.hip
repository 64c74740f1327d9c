// Rotary positions on q and k, with k and v optionally written to a paged cache (hts_rope,
// hts_rope_cache).
//
// Pair i of a head turns by position * f_i: (x, y) -> m (x cos - y sin, x sin + y cos).  The angle
// in turns, position * (f_i / 2 pi), is formed in 64 bits and reduced to [-1/2, 1/2] before its
// sine and cosine are taken in 32 (at position 10^6 the fastest pair has gone 159155 turns: 32
// bits would leave 1/64 of a turn).  All heads of a token share the angles, so a workgroup takes one
// token, makes its rot/2 sines and cosines once in LDS, and streams the token's heads through
// 16-byte loads and stores.
#include "serve_device.h"
#include "serve_internal.h"

namespace hts {
namespace {

constexpr int kThreads = 256;

// V consecutive 16-bit values (4 or 8) to and from floats.
template <typename T, int V> __device__ __forceinline__ void load_v(const uint16_t* p, float* f) {
    if (V == 8) {
        widen8<T>(ld16(p), f);
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        f[0] = widen<T>(v.x & 0xFFFFu);
        f[1] = widen<T>(v.x >> 16);
        f[2] = widen<T>(v.y & 0xFFFFu);
        f[3] = widen<T>(v.y >> 16);
    }
}
template <typename T, int V> __device__ __forceinline__ void store_v(uint16_t* p, const float* f) {
    if (V == 8) {
        st16(p, narrow8<T>(f));
    } else {
        *reinterpret_cast<uint2*>(p) = uint2{narrow<T>(f[0]) | (narrow<T>(f[1]) << 16),
                                             narrow<T>(f[2]) | (narrow<T>(f[3]) << 16)};
    }
}
template <int V> __device__ __forceinline__ void store_e4m3(uint8_t* p, const float* f, float scale) {
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = f[i] / scale;
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<uint32_t*>(p + i) = narrow4_e4m3(x + i);
}

// V pairs per item: entries [i, i+V) and [rot/2 + i, ...) (half) or [2i, 2i + 2V) (interleaved)
template <typename T, int LAYOUT, int V, bool C8>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a) {
    __shared__ float cs[128], sn[128];
    const int64_t t = blockIdx.x;
    const int pos = a.positions[t];
    if (pos < 0) return;
    const int half = a.rot / 2;
    if ((int)threadIdx.x < half) {
        double turn = (double)pos * a.turns[threadIdx.x];
        turn -= rint(turn);
        float s, c;
        sincospif(2.0f * (float)turn, &s, &c);
        cs[threadIdx.x] = c * a.magnitude;
        sn[threadIdx.x] = s * a.magnitude;
    }
    __syncthreads();

    const int turned = half / V, items = turned + (a.dim - a.rot) / 8;   // items of a q or k head
    const int nq = a.q_heads * items, nk = a.k_heads * items;
    int64_t at = -1;                    // the token's place in the cache
    if (a.slots) {
        const int64_t slot = a.slots[t];
        if (slot >= 0 && slot < a.n_slots)
            at = (slot >> a.page_shift) * a.page_stride + (slot & ((1 << a.page_shift) - 1)) * a.token_stride;
    }
    const bool write_k = a.Ko || at >= 0;
    const int nv = at >= 0 ? a.k_heads * (a.dim / 8) : 0;
    const int total = nq + (write_k ? nk : 0);

    for (int it = threadIdx.x; it < total; it += kThreads) {
        const bool is_q = it < nq;
        const int x = is_q ? it : it - nq, h = x / items, w = x - h * items;
        const uint16_t* src = (is_q ? a.Q + t * a.ldq : a.K + t * a.ldk) + h * a.dim;
        const bool cached = !is_q && !a.Ko;
        uint16_t* dst = is_q ? a.Qo + t * a.ldqo + h * a.dim
                             : (cached ? (uint16_t*)a.kc + at + h * a.head_stride : a.Ko + t * a.ldko + h * a.dim);
        uint8_t* dst8 = (uint8_t*)a.kc + at + h * a.head_stride;
        const float scale = C8 && cached && a.k_scale ? a.k_scale[h] : 1.0f;
        if (w < turned) {
            const int i = w * V;
            const int o0 = LAYOUT == HTS_ROPE_HALF ? i : 2 * i, o1 = LAYOUT == HTS_ROPE_HALF ? half + i : 2 * i + V;
            float u[2 * V], r[2 * V];
            load_v<T, V>(src + o0, u);
            load_v<T, V>(src + o1, u + V);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int ix = LAYOUT == HTS_ROPE_HALF ? e : 2 * e, iy = LAYOUT == HTS_ROPE_HALF ? V + e : 2 * e + 1;
                const float c = cs[i + e], s = sn[i + e];
                r[ix] = fmaf(u[ix], c, -(u[iy] * s));
                r[iy] = fmaf(u[ix], s, u[iy] * c);
            }
            if (C8 && cached) {
                store_e4m3<V>(dst8 + o0, r, scale);
                store_e4m3<V>(dst8 + o1, r + V, scale);
            } else {
                store_v<T, V>(dst + o0, r);
                store_v<T, V>(dst + o1, r + V);
            }
        } else {
            const int o = a.rot + (w - turned) * 8;
            if (C8 && cached) {
                float u[8];
                load_v<T, 8>(src + o, u);
                store_e4m3<8>(dst8 + o, u, scale);
            } else {
                st16(dst + o, ld16(src + o));
            }
        }
    }
    for (int it = threadIdx.x; it < nv; it += kThreads) {
        const int per = a.dim / 8, h = it / per, o = (it - h * per) * 8;
        const uint16_t* src = a.V + t * a.ldv + h * a.dim + o;
        if (C8) {
            float u[8];
            load_v<T, 8>(src, u);
            store_e4m3<8>((uint8_t*)a.vc + at + h * a.head_stride + o, u, a.v_scale ? a.v_scale[h] : 1.0f);
        } else {
            st16((uint16_t*)a.vc + at + h * a.head_stride + o, ld16(src));
        }
    }
}

template <typename T, int LAYOUT>
hipError_t launch(const RopeArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.T), block(kThreads);
    if (a.rot % 16 == 0) {
        if (a.cache8) rope_kernel<T, LAYOUT, 8, true><<<grid, block, 0, s>>>(a);
        else rope_kernel<T, LAYOUT, 8, false><<<grid, block, 0, s>>>(a);
    } else {
        if (a.cache8) rope_kernel<T, LAYOUT, 4, true><<<grid, block, 0, s>>>(a);
        else rope_kernel<T, LAYOUT, 4, false><<<grid, block, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) {
    if (a.dtype == HTS_BF16)
        return a.layout == HTS_ROPE_HALF ? launch<BF16T, HTS_ROPE_HALF>(a, s) : launch<BF16T, HTS_ROPE_INTERLEAVED>(a, s);
    return a.layout == HTS_ROPE_HALF ? launch<F16T, HTS_ROPE_HALF>(a, s) : launch<F16T, HTS_ROPE_INTERLEAVED>(a, s);
}

}  // namespace hts
