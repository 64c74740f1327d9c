// Attention of one new token per request over a paged key-value cache (hts_paged_attn).
//
// s_t = scale q.k_t, O = sum_t 2^(s_t log2e - m) v_t / sum_t 2^(s_t log2e - m): one pass over the
// tokens with a running maximum m, sum l and accumulator.  Bound by HBM: K and V are read once, and
// a new token brings only 4 operations per cached value and query head.
//
// A workgroup (4 waves) takes one request, one cache head, up to 16 of the query heads that share
// it, and a range of tokens; each wave takes every fourth step of 32 tokens.  Both products run on
// 16x16x32 MFMA with the tokens' data straight from global memory in registers, no LDS:
//   S^T = K Q^T   A = 16 tokens x 32 entries (16-byte loads of a token's row), B = the heads' q;
//                 lane (head + 16 g) then holds the scores of its head for tokens 4g .. 4g+3.
//   O^T = V^T P^T the same lane's weights are already the B operand if slot 8g + j of the product is
//                 token 4g + j (j < 4) or 16 + 4g + j - 4: the order of the sum is free.  V^T needs 8
//                 tokens of one entry per lane: a lane loads 8 entries of those 8 tokens and
//                 transposes them in registers (one byte permute per two values).
// So the maximum, the sum and the accumulators of a head stay in the lanes of that head, and no
// value crosses lanes in the loop but the maximum -- and that only when a score passes the last
// reference by 2^8, which rescales; below that the weights stay under 256 and nothing is lost.
// Weights are split into two 16-bit parts (their sum holds 16 bits and more), so that the product
// with V rounds them no further than 2^-16: the matrix cores are idle most of the time.
// K's registers are reloaded for the next step as soon as the scores are out, V's as soon as O is.
//
// Few requests with long contexts would leave the chip idle, so the tokens of a request are split
// over workgroups: every workgroup reads the lengths, derives the same chunk size (total / target)
// and finds its request and chunk by a scan; chunks of split requests leave (O, m, l) in the
// workspace, and a second kernel joins them in order.
#include "serve_device.h"
#include "serve_internal.h"

namespace hts {
namespace {

constexpr int kWaves = 4;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

// Two E4M3 bytes (the low or high half of w) to two 16-bit values, exactly.
template <typename T, bool HI> __device__ __forceinline__ uint32_t pair_e4m3(uint32_t w);
template <> __device__ __forceinline__ uint32_t pair_e4m3<BF16T, false>(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}
template <> __device__ __forceinline__ uint32_t pair_e4m3<BF16T, true>(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
}
template <> __device__ __forceinline__ uint32_t pair_e4m3<F16T, false>(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
}
template <> __device__ __forceinline__ uint32_t pair_e4m3<F16T, true>(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
}

// N 16-bit values (N/2 words) as stored: 16-bit values, or E4M3 bytes until they are used.
template <bool C8, int N> struct Raw {
    static constexpr int words = C8 ? N / 4 : N / 2;
    uint32_t w[words];
    __device__ __forceinline__ void load(const char* p) {
        if (words == 4) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
            for (int i = 0; i < words; ++i) w[i] = v[i];
        } else if (words == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x;
            w[words - 1] = v.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < words; ++i) w[i] = 0;
    }
    template <typename T> __device__ __forceinline__ uint32_t pair(int i) const {   // values 2i, 2i + 1
        if (!C8) return w[i];
        return (i & 1) ? pair_e4m3<T, true>(w[i / 2]) : pair_e4m3<T, false>(w[i / 2]);
    }
};

// Tokens of request b: [start, len), counted from begin = start rounded down to a step.
struct Span {
    uint32_t start, begin, len;
    __device__ __forceinline__ uint32_t size() const { return len - begin; }
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b) {
    Span s;
    s.len = min((uint32_t)max(a.lengths[b], 0), a.cap);
    s.start = a.window && s.len > a.window ? s.len - a.window : 0;
    s.begin = s.start & ~31u;
    return s;
}

struct Place {
    int b;                       // request, -1: this workgroup has no work
    uint32_t split, count, slot, chunk;
};

// The x-th workgroup's request and chunk.  Every wave of every workgroup finds the same division.
__device__ __forceinline__ Place find_place(const AttnArgs& a, uint32_t x, int lane) {
    const int per = (a.B + 63) / 64, b0 = lane * per;
    uint64_t total = 0;
    for (int i = 0; i < per; ++i)
        if (b0 + i < a.B) total += span_of(a, b0 + i).size();
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
    total = ((uint64_t)uniform((uint32_t)(total >> 32)) << 32) | uniform((uint32_t)total);
    const uint64_t want = (total / (uint32_t)a.target + 32) & ~uint64_t(31);
    // (lengths are below 2^31: a chunk of that size splits nothing)
    const uint32_t chunk = (uint32_t)min(max(want, (uint64_t)a.min_chunk), uint64_t(1) << 31);
    uint32_t n = 0, ns = 0;
    for (int i = 0; i < per; ++i)
        if (b0 + i < a.B) {
            const uint32_t k = max(1u, (span_of(a, b0 + i).size() + chunk - 1) / chunk);
            n += k;
            ns += k > 1 ? k : 0;
        }
    uint32_t in = n, ins = ns;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t u = __shfl_up(in, o), us = __shfl_up(ins, o);
        if (lane >= o) {
            in += u;
            ins += us;
        }
    }
    Place p;
    p.chunk = chunk;
    p.b = -1;
    const uint64_t past = __ballot(in > x);
    if (!past) return p;
    const int owner = __builtin_ctzll(past);
    uint32_t base = __builtin_amdgcn_readlane(in - n, owner), slot = __builtin_amdgcn_readlane(ins - ns, owner);
    for (int i = 0; i < per; ++i) {
        const int b = owner * per + i;
        if (b >= a.B) break;
        const uint32_t k = max(1u, (span_of(a, b).size() + chunk - 1) / chunk);
        if (x < base + k) {
            p.b = b;
            p.split = x - base;
            p.count = k;
            p.slot = slot;
            break;
        }
        base += k;
        slot += k > 1 ? k : 0;
    }
    return p;
}

// DP: the head size rounded up to 64, 128 or 256; FULL: it is the head size.
template <typename T, bool C8, int DP, bool FULL>
__global__ __launch_bounds__(64 * kWaves, DP == 256 ? 2 : 3) void attn_kernel(AttnArgs a) {
    constexpr int NK = DP / 32;                 // 32-entry steps of q.k
    constexpr int VEC = DP == 64 ? 4 : 8;       // entries of V a lane holds per token and half
    constexpr int NH = DP == 256 ? 2 : 1;       // 128-entry halves of V
    constexpr int ES = C8 ? 1 : 2;
    constexpr int W = DP < 128 ? DP : 128, PAD = 4;
    __shared__ float lds_o[kWaves][16][W + PAD];
    __shared__ float lds_m[kWaves][16], lds_l[kWaves][16];

    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int wave = uniform(tid >> 6);
    const int y = blockIdx.y, hk = y / a.head_tiles, ht = y - hk * a.head_tiles;
    const int group = a.q_heads / a.k_heads;
    const int heads = min(16, group - ht * 16), head0 = hk * group + ht * 16;

    Place p{(int)blockIdx.x, 0, 1, 0, 0};
    if (a.part_o) {
        p = find_place(a, blockIdx.x, lane);
        if (p.b < 0) return;
    }
    const Span sp = span_of(a, p.b);
    const uint32_t first = sp.begin + p.split * p.chunk;
    const uint32_t last = p.count > 1 && p.split + 1 < p.count ? first + p.chunk : sp.len;
    if (a.part_o && y == 0 && p.split == 0 && tid == 0) a.plan[p.b] = uint2{p.slot, p.count};

    u32x4 q[NK];
    {
        const uint16_t* row = a.Q + p.b * a.ldq + (int64_t)(head0 + c) * a.dim;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            q[k] = u32x4{0, 0, 0, 0};
            const int d = 32 * k + 8 * g;
            if (c < heads && (FULL || d < a.dim)) q[k] = ld16(row + d);
        }
    }

    const int32_t* table = a.table + p.b * a.ldt;
    const char* kbase = (const char*)a.kc + (int64_t)hk * a.head_stride * ES;
    const char* vbase = (const char*)a.vc + (int64_t)hk * a.head_stride * ES;
    const uint32_t k_lane = ((uint32_t)c * (uint32_t)a.token_stride + 8 * g) * ES;
    const uint32_t v_lane = ((uint32_t)(4 * g) * (uint32_t)a.token_stride + VEC * c) * ES;
    const uint32_t v_step = (uint32_t)a.token_stride * ES, page_mask = (1u << a.page_shift) - 1;
    const float s_scale = a.scale * kLog2e * (C8 && a.k_scale ? a.k_scale[hk] : 1.0f);

    // the two 16-token halves of the step at t: byte offset of the first token, and whether a page holds it
    struct Half {
        int64_t off;
        bool ok;
    };
    const auto half = [&](uint32_t t) {
        Half h;
        const uint32_t j = t >> a.page_shift;
        const int64_t id = t < a.cap ? table[j] : -1;
        h.ok = id >= 0 && id < a.pages;
        h.off = ((h.ok ? id : 0) * a.page_stride + (int64_t)(t & page_mask) * a.token_stride) * ES;
        return h;
    };
    Raw<C8, 8> kr[2][NK];
    Raw<C8, VEC> vr[NH][8];
    const auto load_k = [&](const Half* h) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                if (FULL || 32 * k + 8 * g < a.dim) kr[j][k].load(kbase + h[j].off + (k_lane + 32 * k * ES));
                else kr[j][k].clear();
            }
    };
    const auto load_v = [&](const Half* h) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                if (FULL || 128 * n + VEC * c < a.dim)
                    vr[n][i].load(vbase + h[i >> 2].off + (v_lane + (i & 3) * v_step + 128 * n * ES));
                else vr[n][i].clear();
            }
    };

    f32x4 o[NH][VEC];
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[n][j] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, ref = 0.0f, l = 0.0f;   // of head c; l: this lane's tokens only

    uint32_t t = first + 32 * wave;
    Half now[2], next[2];
    if (t < last) {
        now[0] = half(t);
        now[1] = half(t + 16);
        load_k(now);
        load_v(now);
    }
    for (; t < last; t += 32 * kWaves) {
        const uint32_t tn = t + 32 * kWaves;
        const bool more = tn < last && tn > t;
        if (more) {
            next[0] = half(tn);
            next[1] = half(tn + 16);
        }
        f32x4 s[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            s[j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                const u32x4 x = {kr[j][k].template pair<T>(0), kr[j][k].template pair<T>(1),
                                 kr[j][k].template pair<T>(2), kr[j][k].template pair<T>(3)};
                s[j] = mfma_dense<T>(x, q[k], s[j]);
            }
        }
        if (more) load_k(next);
        // outside the span, or in no page: no weight (and no value: 0 * NaN is NaN)
        const bool whole = t >= sp.start && t + 32 <= last && t + 32 > t && now[0].ok && now[1].ok;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] *= s_scale;
        if (!whole) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t at = t + 16 * j + 4 * g + i;
                    if (at < sp.start || at >= last || at < t || !now[j].ok) {
                        s[j][i] = -INFINITY;
#pragma unroll
                        for (int n = 0; n < NH; ++n) vr[n][4 * j + i].clear();
                    }
                }
        }
        float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                          fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
        if (__any(top > m + 8.0f)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            top = fmaxf(top, m);
            const float f = exp2f(m - (top == -INFINITY ? 0.0f : top));
            m = top;
            ref = top == -INFINITY ? 0.0f : top;
            l *= f;
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int j = 0; j < VEC; ++j) o[n][j] *= f;
        }
        u32x4 hi, lo;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float p0 = __builtin_amdgcn_exp2f(s[j][2 * i] - ref);
                const float p1 = __builtin_amdgcn_exp2f(s[j][2 * i + 1] - ref);
                l += p0 + p1;
                const uint32_t h0 = narrow<T>(p0), h1 = narrow<T>(p1);
                hi[2 * j + i] = h0 | (h1 << 16);
                lo[2 * j + i] = narrow<T>(p0 - widen<T>(h0)) | (narrow<T>(p1 - widen<T>(h1)) << 16);
            }
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int w = 0; w < VEC / 2; ++w) {
                uint32_t x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = vr[n][i].template pair<T>(w);
                u32x4 even, odd;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    even[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x05040100);
                    odd[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x07060302);
                }
                o[n][2 * w] = mfma_dense<T>(even, hi, o[n][2 * w]);
                o[n][2 * w + 1] = mfma_dense<T>(odd, hi, o[n][2 * w + 1]);
                o[n][2 * w] = mfma_dense<T>(even, lo, o[n][2 * w]);
                o[n][2 * w + 1] = mfma_dense<T>(odd, lo, o[n][2 * w + 1]);
            }
        if (more) load_v(next);
        now[0] = next[0];
        now[1] = next[1];
    }

    // the four waves' parts of each head, in order
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
        lds_m[wave][c] = m;
        lds_l[wave][c] = l;
    }
    __syncthreads();
    float all = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) all = fmaxf(all, lds_m[w][c]);
    const float f = m == -INFINITY ? 0.0f : exp2f(m - all);
    const bool split = p.count > 1;
    const int64_t part = ((int64_t)(p.slot + p.split) * gridDim.y + y) * a.tile_heads;
    const float v_scale = C8 && a.v_scale ? a.v_scale[hk] : 1.0f;
#pragma unroll
    for (int n = 0; n < NH; ++n) {
        if (n) __syncthreads();
        // lane (c, g): entries 4 VEC g .. of head c
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < VEC; j += 4)
                *reinterpret_cast<f32x4*>(&lds_o[wave][c][4 * VEC * g + VEC * i + j]) =
                    f32x4{o[n][j][i] * f, o[n][j + 1][i] * f, o[n][j + 2][i] * f, o[n][j + 3][i] * f};
        __syncthreads();
        for (int it = tid; it < heads * (W / 4); it += 64 * kWaves) {
            const int h = it / (W / 4), d = (it - h * (W / 4)) * 4, at = 128 * n + d;
            if (!FULL && at >= a.dim) continue;
            f32x4 sum = {0, 0, 0, 0};
            float top = -INFINITY, den = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                sum += *reinterpret_cast<const f32x4*>(&lds_o[w][h][d]);
                top = fmaxf(top, lds_m[w][h]);
            }
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                den += lds_m[w][h] == -INFINITY ? 0.0f : lds_l[w][h] * exp2f(lds_m[w][h] - top);
            if (split) {
                *reinterpret_cast<f32x4*>(a.part_o + (part + h) * a.dim + at) = sum;
                if (at == 0) a.part_ml[part + h] = float2{top, den};
            } else {
                const float inv = den == 0.0f ? 0.0f : v_scale / den;
                uint16_t* out = a.O + p.b * a.ldo + (int64_t)(head0 + h) * a.dim + at;
                *reinterpret_cast<uint2*>(out) = uint2{narrow<T>(sum[0] * inv) | (narrow<T>(sum[1] * inv) << 16),
                                                       narrow<T>(sum[2] * inv) | (narrow<T>(sum[3] * inv) << 16)};
                if (at == 0 && a.lse)
                    a.lse[(int64_t)p.b * a.q_heads + head0 + h] = den == 0.0f ? -INFINITY : (top + log2f(den)) * kLn2;
            }
        }
    }
}

// Join the parts of a split request: one workgroup per request and query head; wave w takes parts
// w, w + 4, ..., a lane four entries; the waves' sums are added in order.
template <typename T>
__global__ __launch_bounds__(64 * kWaves) void join_kernel(AttnArgs a) {
    __shared__ f32x4 lds[kWaves][64];
    __shared__ float lds_l[kWaves];
    const int b = blockIdx.x, h = blockIdx.y;
    const uint2 plan = a.plan[b];
    if (plan.y <= 1) return;
    const int group = a.q_heads / a.k_heads, hk = h / group, gh = h - hk * group;
    const int y = hk * a.head_tiles + gh / 16, rows = a.k_heads * a.head_tiles;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const auto part = [&](uint32_t i) { return ((int64_t)(plan.x + i) * rows + y) * a.tile_heads + (gh & 15); };
    float top = -INFINITY;
    for (uint32_t i = lane; i < plan.y; i += 64) top = fmaxf(top, a.part_ml[part(i)].x);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    f32x4 sum = {0, 0, 0, 0};
    float l = 0.0f;
    const bool on = lane * 4 < a.dim;
#pragma unroll 4
    for (uint32_t i = wave; i < plan.y; i += kWaves) {
        const float2 ml = a.part_ml[part(i)];
        const float f = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - top);
        l += ml.y * f;
        if (on) sum += *reinterpret_cast<const f32x4*>(a.part_o + part(i) * a.dim + lane * 4) * f;
    }
    lds[wave][lane] = sum;
    if (lane == 0) lds_l[wave] = l;
    __syncthreads();
    if (wave) return;
    l = 0.0f;
    sum = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        sum += lds[w][lane];
        l += lds_l[w];
    }
    const float inv = l == 0.0f ? 0.0f : (a.v_scale ? a.v_scale[hk] : 1.0f) / l;
    if (on)
        *reinterpret_cast<uint2*>(a.O + b * a.ldo + (int64_t)h * a.dim + lane * 4) =
            uint2{narrow<T>(sum[0] * inv) | (narrow<T>(sum[1] * inv) << 16),
                  narrow<T>(sum[2] * inv) | (narrow<T>(sum[3] * inv) << 16)};
    if (lane == 0 && a.lse) a.lse[(int64_t)b * a.q_heads + h] = l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
}

template <typename T, bool C8>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.part_o ? a.B + a.target : a.B), (unsigned)(a.k_heads * a.head_tiles)), block(64 * kWaves);
    if (a.dim == 64) attn_kernel<T, C8, 64, true><<<grid, block, 0, s>>>(a);
    else if (a.dim < 64) attn_kernel<T, C8, 64, false><<<grid, block, 0, s>>>(a);
    else if (a.dim == 128) attn_kernel<T, C8, 128, true><<<grid, block, 0, s>>>(a);
    else if (a.dim < 128) attn_kernel<T, C8, 128, false><<<grid, block, 0, s>>>(a);
    else if (a.dim == 256) attn_kernel<T, C8, 256, true><<<grid, block, 0, s>>>(a);
    else attn_kernel<T, C8, 256, false><<<grid, block, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part_o) return e;
    join_kernel<T><<<dim3((unsigned)a.B, (unsigned)a.q_heads), block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, hipStream_t s) {
    if (a.dtype == HTS_BF16) return a.cache8 ? launch<BF16T, true>(a, s) : launch<BF16T, false>(a, s);
    return a.cache8 ? launch<F16T, true>(a, s) : launch<F16T, false>(a, s);
}

}  // namespace hts
