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
        stream16(p, narrow8<T>(f));
    } else {
        *reinterpret_cast<uint2*>(p) = uint2{narrow2<T>(f[0], f[1]), narrow2<T>(f[2], f[3])};
    }
}
template <int V> __device__ __forceinline__ void store_e4m3(uint8_t* p, const float* f, float scale) {
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = f[i] / scale;
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<uint32_t*>(p + i) = narrow4_e4m3(x + i);
}

// An item of a q or k head: P pairs, entries [i, i+P) and [rot/2 + i, ...) (half, P = 8 or 4) or the
// 2P = 8 consecutive entries [2i, 2i + 8) (interleaved, P = 4); or 8 entries past the rotated part.
template <typename T, int LAYOUT, int P, bool C8>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a) {
    __shared__ float cs[128], sn[128];
    const int64_t t = blockIdx.z * kGridX + blockIdx.x;
    if (t >= a.T) return;
    int64_t token = t;
    bool lost = false;                  // the row's request adds more than one token, or one that is not there
    if (a.starts) {
        const int first = a.starts[t], end = a.starts[t + 1];
        if (first < 0 || first >= end) return;
        lost = end - first > 1 || first >= a.tokens;
        token = lost ? 0 : first;
    }
    const int pos = lost ? 0 : a.positions[token];
    if (pos < 0) return;
    const int half = a.rot / 2;
    if ((int)threadIdx.x < half) {
        double turn = (double)pos * a.turns[threadIdx.x];
        turn -= rint(turn);
        float s, c;
        sincospif(lost ? __builtin_nanf("") : 2.0f * (float)turn, &s, &c);
        cs[threadIdx.x] = c * a.magnitude;
        sn[threadIdx.x] = s * a.magnitude;
    }
    int64_t at = -1;                    // the token's place in the cache
    if (a.slots) {
        const int64_t slot = a.slots[token];
        if (slot >= 0 && slot < a.n_slots && !lost)
            at = (slot >> a.page_shift) * a.page_stride + (slot & ((1 << a.page_shift) - 1)) * a.token_stride;
    }
    // items: all q heads, then all k heads, then v in chunks of 8
    const int turned = half / P, items = turned + (a.dim - a.rot) / 8, per_v = a.dim / 8;
    const int step = gridDim.y * kThreads, first = blockIdx.y * kThreads + threadIdx.x;
    const int heads = a.q_heads + (a.Ko || at >= 0 ? a.k_heads : 0);
    __syncthreads();

    // (head, item) and its step, so that the loop has no division
    int h = first / items, w = first - h * items;
    const int dh = step / items, dw = step - dh * items;
    for (; h < heads; h += dh) {
        const bool is_q = h < a.q_heads, cached = !is_q && !a.Ko;
        const int hh = is_q ? h : h - a.q_heads;
        const uint16_t* src = (is_q ? a.Q + t * a.ldq : a.K + t * a.ldk) + hh * a.dim;
        uint16_t* dst = is_q ? a.Qo + t * a.ldqo + hh * a.dim
                             : (cached ? (uint16_t*)a.kc + at + hh * a.head_stride : a.Ko + t * a.ldko + hh * a.dim);
        uint8_t* dst8 = (uint8_t*)a.kc + at + hh * a.head_stride;
        const float scale = C8 && cached && a.k_scale ? a.k_scale[hh] : 1.0f;
        if (w < turned) {
            const int i = w * P;
            float u[2 * P], r[2 * P];
            if constexpr (LAYOUT == HTS_ROPE_HALF) {
                load_v<T, P>(src + i, u);
                load_v<T, P>(src + half + i, u + P);
            } else {
                load_v<T, 8>(src + 2 * i, u);
            }
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const int ix = LAYOUT == HTS_ROPE_HALF ? e : 2 * e, iy = LAYOUT == HTS_ROPE_HALF ? P + e : 2 * e + 1;
                const float c = cs[i + e], s = sn[i + e];
                r[ix] = fmaf(u[ix], c, -(u[iy] * s));
                r[iy] = fmaf(u[ix], s, u[iy] * c);
            }
            if constexpr (LAYOUT == HTS_ROPE_HALF) {
                if (C8 && cached) {
                    store_e4m3<P>(dst8 + i, r, scale);
                    store_e4m3<P>(dst8 + half + i, r + P, scale);
                } else {
                    store_v<T, P>(dst + i, r);
                    store_v<T, P>(dst + half + i, r + P);
                }
            } else {
                if (C8 && cached) store_e4m3<8>(dst8 + 2 * i, r, scale);
                else store_v<T, 8>(dst + 2 * i, r);
            }
        } else {
            const int o = a.rot + (w - turned) * 8;
            if (C8 && cached) {
                float u[8];
                load_v<T, 8>(src + o, u);
                store_e4m3<8>(dst8 + o, u, scale);
            } else {
                stream16(dst + o, ld16(src + o));
            }
        }
        w += dw;
        if (w >= items) {
            w -= items;
            ++h;
        }
    }
    if (at < 0) return;
    // v
    h = first / per_v;
    w = first - h * per_v;
    const int vh = step / per_v, vw = step - vh * per_v;
    for (; h < a.k_heads; h += vh) {
        const uint16_t* src = a.V + t * a.ldv + h * a.dim + w * 8;
        const int64_t to = at + h * a.head_stride + w * 8;
        if (C8) {
            float u[8];
            load_v<T, 8>(src, u);
            store_e4m3<8>((uint8_t*)a.vc + to, u, a.v_scale ? a.v_scale[h] : 1.0f);
        } else {
            stream16((uint16_t*)a.vc + to, ld16(src));
        }
        w += vw;
        if (w >= per_v) {
            w -= per_v;
            ++h;
        }
    }
}

template <typename T>
hipError_t launch(const RopeArgs& a, hipStream_t s) {
    // one workgroup per token; where that leaves CUs idle, up to 4 that share the token's items, each making the angles
    // (heads of 128, with one workgroup and shared: 1 token of 32/32 heads 3.9 and 3.5 us, 61 of 40/8 4.0 and 3.7, 200 of
    // 32/32 4.4 and 4.2)
    const int64_t items = ((int64_t)(a.q_heads + a.k_heads) * (a.dim / 16) + (int64_t)a.k_heads * (a.dim / 8)) / kThreads;
    const int64_t share = a.T >= 256 ? 1 : items < 1 ? 1 : items > 4 ? 4 : items;
    const WideGrid wide = wide_grid(a.T);
    const dim3 grid(wide.x, (unsigned)share, wide.rest), block(kThreads);
    if (a.layout == HTS_ROPE_INTERLEAVED) {
        if (a.cache8) rope_kernel<T, HTS_ROPE_INTERLEAVED, 4, true><<<grid, block, 0, s>>>(a);
        else rope_kernel<T, HTS_ROPE_INTERLEAVED, 4, false><<<grid, block, 0, s>>>(a);
    } else if (a.rot % 16 == 0) {
        if (a.cache8) rope_kernel<T, HTS_ROPE_HALF, 8, true><<<grid, block, 0, s>>>(a);
        else rope_kernel<T, HTS_ROPE_HALF, 8, false><<<grid, block, 0, s>>>(a);
    } else {
        if (a.cache8) rope_kernel<T, HTS_ROPE_HALF, 4, true><<<grid, block, 0, s>>>(a);
        else rope_kernel<T, HTS_ROPE_HALF, 4, false><<<grid, block, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) {
    return a.dtype == HTS_BF16 ? launch<BF16T>(a, s) : launch<F16T>(a, s);
}

}  // namespace hts
