// Attention of one new token per request over a paged key-value cache (hts_paged_attn).
//
// s_t = scale q.k_t, O = sum_t 2^(s_t log2e - m) v_t / sum_t 2^(s_t log2e - m): one pass over the
// tokens with a running maximum m, sum l and accumulator.  Bound by HBM: K and V are read once per 16
// query heads of a cache head, and a new token brings only 4 operations per cached value and query head.
//
// A workgroup (4 waves) takes one request, one cache head, up to 16 of the query heads that share
// it, and a range of tokens; each wave takes every fourth step of 32 tokens (or 16, with halves of the
// second product).  Both products run on 16x16x32 MFMA with the tokens' data straight from global
// memory in registers, no LDS:
//   S^T = K Q^T   A = 16 tokens x 32 entries (16-byte loads of a token's row), B = the heads' q;
//                 lane (head + 16 g) then holds the scores of its head for tokens 4g .. 4g+3.
//   O^T = V^T P^T the same lane's weights are already the B operand if slot 8g + j of the product is
//                 token 4g + j (j < 4) or 16 + 4g + j - 4: the order of the sum is free.  V^T needs 8
//                 tokens of one entry per lane: a lane loads 8 entries of those 8 tokens and
//                 transposes them in registers (one byte permute per two values).
// So the maximum, the sum and the accumulators of a head stay in the lanes of that head, and no
// value crosses lanes in the loop but the maximum -- and that only when a score passes the last
// reference by 2^8, which rescales; below that the weights stay in range and nothing is lost.
// Weights go to the product with V in 16-bit parts that hold 24 bits (bfloat16, three parts) or 22 (binary16, two, the
// second 2^11 times as large, so that it reaches below binary16's smallest value): the matrix cores are idle most of the
// time (no case measured is slower than with two unscaled parts).
// K's registers are reloaded for the next step as soon as the scores are out, V's as soon as O is.
//
// The work is divided evenly: per cache head, the steps of all requests in a row are cut into as
// many equal runs as there are workgroups for that head on the chip at once.  Every workgroup reads
// the lengths, finds its run by a scan over them and goes through the requests in it; a request that
// lies whole in one run is written at once, the parts of one that is cut leave (O, m, l) in the
// workspace, and a second kernel joins them in order.  All workgroups then end together, whatever the
// mix of lengths (one request and chunk to a workgroup left a tail: 64 requests of 128 .. 8191 tokens).
#include <type_traits>

#include "serve_device.h"
#include "serve_internal.h"

namespace hts {
namespace {

constexpr int kWaves = 4;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
// Weights are 2^(s - m + 7): at most 2^15, since m is at least the maximum less 8, which binary16 holds.
constexpr float kShift = 7.0f;

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

// Read of an index that is the same in all lanes, by way of the scalar cache: a vector load would
// have to wait for every load of K and V before it (they return in order).  Nothing writes these
// arrays while the kernel runs.
typedef const __attribute__((address_space(4))) int32_t* ScalarPtr;
__device__ __forceinline__ int32_t scalar_load(const int32_t* p, int64_t i) {
    return reinterpret_cast<ScalarPtr>(reinterpret_cast<uintptr_t>(p))[i];
}

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

constexpr uint32_t kBufferEnd = 0xFFFFF000u;   // past every offset in a half step (15 token strides and a head)

// N 16-bit values (N/2 words) as stored: 16-bit values, or E4M3 bytes until they are used.
template <bool C8, int N> struct Raw {
    static constexpr int words = C8 ? N / 4 : N / 2;
    uint32_t w[words];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t from, uint32_t lane_off, uint32_t off) {
        if constexpr (words == 4) {
            const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(from, lane_off, off, 0));
#pragma unroll
            for (int i = 0; i < words; ++i) w[i] = v[i];
        } else if constexpr (words == 2) {
            const uint2 v = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(from, lane_off, off, 0));
            w[0] = v.x;
            w[1] = v.y;
        } else {
            w[0] = __builtin_amdgcn_raw_buffer_load_b32(from, lane_off, off, 0);
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

// Two weights as 16-bit parts, a word each.  A part takes what those before it left out, which 32 bits hold exactly.
//   bfloat16: three parts of 8 bits, to nearest: 24 bits, a 32-bit weight's own.
//   binary16: 11 bits, towards zero, then 2^11 times the rest, to nearest: off by at most 2^-21 of the weight, or 2^-36
//             where that is more (below 2^-14 the first part's steps are 2^-24).  The largest weight is 2^7 and more, so
//             a token of a long context loses at most 2^-43 of the largest, however many there are of them; with the
//             rest unscaled it lost up to 2^-31, always downwards (100000 tokens of e^-18 beside a large one: 2%).
constexpr float kRest = 2048.0f;
template <typename T> constexpr int kParts = T::id == BF16T::id ? 3 : 2;
template <typename T> __device__ __forceinline__ void split2(float lo, float hi, uint32_t* part) {
    if constexpr (T::id == BF16T::id) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            part[k] = narrow2<T>(lo, hi);
            lo -= widen<T>(part[k] & 0xFFFFu);
            hi -= widen<T>(part[k] >> 16);
        }
    } else {
        part[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(lo, hi));
        part[1] = narrow2<T>((lo - widen<T>(part[0] & 0xFFFFu)) * kRest, (hi - widen<T>(part[0] >> 16)) * kRest);
    }
}

// O^T += V^T P^T over the 16 (binary16 only) or 32 tokens of a step (NT = 1, 2): operands of two words per 16 tokens.
template <typename T, int NT>
__device__ __forceinline__ f32x4 mfma_tokens(const uint32_t* v, const uint32_t* p, f32x4 o) {
    if constexpr (NT == 2) {
        return mfma_dense<T>(u32x4{v[0], v[1], v[2], v[3]}, u32x4{p[0], p[1], p[2], p[3]}, o);
    } else {
        typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
        return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(f16x4, uint2{v[0], v[1]}),
                                                     __builtin_bit_cast(f16x4, uint2{p[0], p[1]}), o, 0, 0, 0);
    }
}

// The same with the weights in their parts.  Of bfloat16's three on 16 tokens the first two share a product of 32 places,
// and the third takes such a one too: an accumulator that goes from the longer product straight into the shorter one is
// read before it is whole (the compiler leaves no wait there).
template <typename T, int NT>
__device__ __forceinline__ f32x4 mfma_weights(const uint32_t* v, const uint32_t (*p)[2 * NT], f32x4 o) {
    if constexpr (T::id == F16T::id) {
        const f32x4 rest = mfma_tokens<T, NT>(v, p[1], f32x4{0, 0, 0, 0});
        o = mfma_tokens<T, NT>(v, p[0], o);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = fmaf(rest[i], 1.0f / kRest, o[i]);
        return o;
    } else if constexpr (NT == 2) {
        return mfma_tokens<T, NT>(v, p[2], mfma_tokens<T, NT>(v, p[1], mfma_tokens<T, NT>(v, p[0], o)));
    } else {
        const u32x4 twice = {v[0], v[1], v[0], v[1]};
        return mfma_dense<T>(twice, u32x4{p[2][0], p[2][1], 0, 0},
                             mfma_dense<T>(twice, u32x4{p[0][0], p[0][1], p[1][0], p[1][1]}, o));
    }
}

// Tokens of request b: [start, len), counted from begin = start rounded down to a step of 32.
struct Span {
    uint32_t start, begin, len;
    __device__ __forceinline__ uint32_t steps() const { return max(1u, (len - begin + 31) / 32); }
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int32_t length) {
    Span s;
    s.len = min((uint32_t)max(length, 0), a.cap);
    s.start = a.window && s.len > a.window ? s.len - a.window : 0;
    s.begin = s.start & ~31u;
    return s;
}

// A workgroup's run of steps: from step `off` of request b on, `left` steps in all; per: a full run.
// The host has checked that all steps together are fewer than 2^31.
struct Run {
    int b;
    uint32_t off, left, per;
};
// Inclusive sum over the lanes of a wave, by row shifts and row broadcasts (no LDS round trip).
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
#define HTS_ROW(ctrl, rows) x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, rows, 0xF, false)
    HTS_ROW(0x111, 0xF);   // row_shr:1, 2, 4, 8
    HTS_ROW(0x112, 0xF);
    HTS_ROW(0x114, 0xF);
    HTS_ROW(0x118, 0xF);
    HTS_ROW(0x142, 0xA);   // row_bcast:15 into rows 1 and 3
    HTS_ROW(0x143, 0xC);   // row_bcast:31 into rows 2 and 3
#undef HTS_ROW
    return x;
}

// Lengths of the requests: in the lanes of every wave where there are at most 64, else in memory.
struct Lengths {
    const int32_t* p;
    int32_t mine;
    bool held;
    __device__ __forceinline__ int32_t operator[](int b) const {
        return held ? __builtin_amdgcn_readlane(mine, b) : scalar_load(p, b);
    }
};

__device__ __forceinline__ Run find_run(const AttnArgs& a, const Lengths& lengths, uint32_t x, int lane) {
    const int each = (a.B + 63) / 64, b0 = lane * each;
    uint32_t mine = 0;
    if (lengths.held) {
        if (lane < a.B) mine = span_of(a, lengths.mine).steps();
    } else {
        for (int i = 0; i < each; ++i)
            if (b0 + i < a.B) mine += span_of(a, a.lengths[b0 + i]).steps();
    }
    const uint32_t in = wave_scan(mine), total = __builtin_amdgcn_readlane(in, 63);
    Run r;
    // An even share, but where that is short a longer run, down to a third as many of them: each costs a start, an
    // end and its parts (one request of 4096 tokens, 32 heads: 19.8 us with runs of 6 steps, 18.4 with 16; 16 of up to
    // 300 in a table for 8192, 32/8 heads: 13.0 with 4, 14.8 with 8) -- and not longer for that than the requests are,
    // which cost as much each.
    const uint32_t few = min(min(max(3 * total / a.target, 4u), 16u), (total + a.B - 1) / a.B);
    r.per = max((total + gridDim.x - 1) / gridDim.x, few);
    const uint32_t pos = x * r.per;
    r.left = pos < total ? min(r.per, total - pos) : 0;
    if (!r.left) return r;
    const int owner = __builtin_ctzll(__ballot(in > pos));
    uint32_t at = __builtin_amdgcn_readlane(in - mine, owner);
    r.b = owner * each;
    while (!lengths.held) {                          // ends: the owner's requests hold step pos
        const uint32_t n = span_of(a, lengths[r.b]).steps();
        if (pos < at + n) break;
        at += n;
        ++r.b;
    }
    r.off = pos - at;
    return r;
}

// DP: the head size rounded up to 64, 128 or 256; FULL: it is the head size.  SPLIT: the workgroup takes a run of steps,
// else request blockIdx.x.  TOK: tokens of a step, 32 or 16.
template <typename T, bool C8, int DP, bool FULL, bool SPLIT, int TOK>
__global__ __launch_bounds__(64 * kWaves, DP == 256 ? 2 : TOK == 16 ? 4 : 3) void attn_kernel(AttnArgs a) {
    constexpr int NK = DP / 32;                 // 32-entry steps of q.k
    constexpr int VEC = DP == 64 ? 4 : 8;       // entries of V a lane holds per token and half
    constexpr int NH = DP == 256 ? 2 : 1;       // 128-entry halves of V
    constexpr int NT = TOK / 16;                // 16-token halves of a step
    constexpr int STRIDE = TOK * kWaves;
    constexpr int ES = C8 ? 1 : 2;
    constexpr int W = DP < 128 ? DP : 128;
    __shared__ float lds_o[kWaves][16][W + 4];
    __shared__ float lds_m[kWaves][16], lds_l[kWaves][16];

    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int wave = uniform(tid >> 6);
    const int y = blockIdx.y, hk = y / a.head_tiles, ht = y - hk * a.head_tiles;
    const int group = a.q_heads / a.k_heads;
    const int heads = min(16, group - ht * 16), head0 = hk * group + ht * 16;

    Run run{(int)blockIdx.x, 0, ~0u, ~0u};
    Lengths lengths{a.lengths, 0, SPLIT && a.B <= 64};
    if (lengths.held && lane < a.B) lengths.mine = a.lengths[lane];
    if (SPLIT) run = find_run(a, lengths, blockIdx.x, lane);
    const char* kbase = (const char*)a.kc + (int64_t)hk * a.head_stride * ES;
    const char* vbase = (const char*)a.vc + (int64_t)hk * a.head_stride * ES;
    // A half step is read through a buffer resource at its first token: a scalar base, one 32-bit offset per lane.
    // Entries past the head's end get an offset past the buffer's: they read as zero, and nothing is fetched.
    const uint32_t k_lane = ((uint32_t)c * (uint32_t)a.token_stride + 8 * g) * ES;
    const uint32_t v_lane = ((uint32_t)(4 * g) * (uint32_t)a.token_stride + VEC * c) * ES;
    const uint32_t v_step = (uint32_t)a.token_stride * ES, page_mask = (1u << a.page_shift) - 1;
    const uint32_t pages = (uint32_t)a.pages;   // below 2^31: an id below 0 is not below it
    const int64_t page_bytes = a.page_stride * ES;
    const float s_scale = a.scale * kLog2e * (C8 && a.k_scale ? a.k_scale[hk] : 1.0f);
    const float v_scale = C8 && a.v_scale ? a.v_scale[hk] : 1.0f;

    for (uint32_t slot = 2 * blockIdx.x; run.left; slot |= 1) {   // one request, or the part of it in this run
    const int b = run.b;
    const int32_t* table = a.table + b * a.ldt;
    const uint32_t last_page = (a.cap - 1) >> a.page_shift;   // ids past it are asked for, but never used
    const auto page_id = [&](uint32_t t) { return scalar_load(table, min(t >> a.page_shift, last_page)); };
    // a request of its own starts at its first token, unless a window cuts it: its first pages are asked for together
    // with its length
    int32_t early[2 * NT];
    const bool known = !SPLIT && !a.window;
    if (known)
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) early[i] = page_id(TOK * wave + 16 * (i % NT) + STRIDE * (i / NT));
    const Span sp = span_of(a, lengths[b]);
    const uint32_t steps = sp.steps(), n_steps = min(steps - run.off, run.left);
    const bool whole_request = n_steps == steps;
    const uint32_t first = sp.begin + 32 * run.off;
    const uint32_t last = min(sp.len, first + 32 * n_steps);
    if (SPLIT) {
        if (run.off == 0 && y == 0 && tid == 0)
            a.plan[b] = uint2{slot, 1 + (steps - n_steps + run.per - 1) / run.per};
        run.left -= n_steps;
        run.off = 0;
        ++run.b;
    } else {
        run.left = 0;
    }

    u32x4 q[NK];
    {
        const uint16_t* row = a.Q + b * a.ldq + (int64_t)(head0 + c) * a.dim;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            const int d = 32 * k + 8 * g;
            q[k] = c < heads && (FULL || d < a.dim) ? ld16(row + d) : u32x4{0, 0, 0, 0};
        }
    }

    // the 16-token halves of the step at t: the page's id (requested a step ahead), then the byte offset of
    // the half's first token and whether a page holds it
    struct Half {
        int64_t off;
        bool ok;
    };
    const auto half = [&](uint32_t t, int32_t id) {
        Half h;
        h.ok = (uint32_t)id < pages;
        h.off = (h.ok ? id : 0) * page_bytes + (uint64_t)(t & page_mask) * v_step;
        return h;
    };
    Raw<C8, 8> kr[NT][NK];
    Raw<C8, VEC> vr[NH][4 * NT];
    const auto resource = [&](const char* base, int64_t off) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base) + off, (short)0, (int)kBufferEnd,
                                                 0x00020000);
    };
    const auto load_k = [&](const Half* h) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const auto from = resource(kbase, h[j].off);
#pragma unroll
            for (int k = 0; k < NK; ++k)
                kr[j][k].load(from, FULL || 32 * k + 8 * g < a.dim ? k_lane : kBufferEnd, 32 * k * ES);
        }
    };
    const auto load_v = [&](const Half* h) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const auto from = resource(vbase, h[j].off);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < NH; ++n)
                    vr[n][4 * j + i].load(from, FULL || 128 * n + VEC * c < a.dim ? v_lane : kBufferEnd,
                                          i * v_step + 128 * n * ES);
        }
    };

    f32x4 o[NH][VEC];
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[n][j] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, ref = 0.0f, l = 0.0f;   // of head c; l: this lane's tokens only

    uint32_t t = first + TOK * wave;
    Half now[NT];
    int32_t ahead[NT];
    // one step; MORE: the wave has another step, whose loads are issued on the way.  (The last step is
    // a copy of its own: behind a branch around the loads the compiler would wait for V where K is used.)
    const auto step = [&](auto more) {
        constexpr bool MORE = decltype(more)::value;
        Half next[NT];
        const uint32_t tn = t + STRIDE;
        if (MORE)
#pragma unroll
            for (int j = 0; j < NT; ++j) next[j] = half(tn + 16 * j, ahead[j]);
        f32x4 s[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            s[j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                const u32x4 x = {kr[j][k].template pair<T>(0), kr[j][k].template pair<T>(1),
                                 kr[j][k].template pair<T>(2), kr[j][k].template pair<T>(3)};
                s[j] = mfma_dense<T>(x, q[k], s[j]);
            }
        }
        if (MORE) {
            load_k(next);
#pragma unroll
            for (int j = 0; j < NT; ++j) ahead[j] = page_id(tn + STRIDE + 16 * j);
        }
        // outside the span, or in no page: no weight (and no value: 0 * NaN is NaN)
        const bool whole = t >= sp.start && t + TOK <= last && t + TOK > t && now[0].ok && now[NT - 1].ok;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] *= s_scale;
        if (!whole) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
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
        float top = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3]));
        if (NT == 2) top = fmaxf(top, fmaxf(fmaxf(s[NT - 1][0], s[NT - 1][1]), fmaxf(s[NT - 1][2], s[NT - 1][3])));
        if (__any(top > m + 8.0f)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            top = fmaxf(top, m);
            const float f = exp2f(m - (top == -INFINITY ? 0.0f : top));
            m = top;
            ref = top == -INFINITY ? 0.0f : top - kShift;
            l *= f;
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int j = 0; j < VEC; ++j) o[n][j] *= f;
        }
        uint32_t p[kParts<T>][2 * NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float p0 = __builtin_amdgcn_exp2f(s[j][2 * i] - ref);
                const float p1 = __builtin_amdgcn_exp2f(s[j][2 * i + 1] - ref);
                l += p0 + p1;
                uint32_t part[kParts<T>];
                split2<T>(p0, p1, part);
#pragma unroll
                for (int k = 0; k < kParts<T>; ++k) p[k][2 * j + i] = part[k];
            }
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int w = 0; w < VEC / 2; ++w) {
                uint32_t x[4 * NT], even[2 * NT], odd[2 * NT];
#pragma unroll
                for (int i = 0; i < 4 * NT; ++i) x[i] = vr[n][i].template pair<T>(w);
#pragma unroll
                for (int i = 0; i < 2 * NT; ++i) {
                    even[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x05040100);
                    odd[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x07060302);
                }
                o[n][2 * w] = mfma_weights<T, NT>(even, p, o[n][2 * w]);
                o[n][2 * w + 1] = mfma_weights<T, NT>(odd, p, o[n][2 * w + 1]);
            }
        if (MORE) {
            load_v(next);
#pragma unroll
            for (int j = 0; j < NT; ++j) now[j] = next[j];
            t = tn;
        }
    };
    if (t < last) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            now[j] = half(t + 16 * j, known ? early[j] : page_id(t + 16 * j));
            ahead[j] = known ? early[NT + j] : page_id(t + STRIDE + 16 * j);
        }
        load_k(now);
        load_v(now);
        while (last - t > STRIDE) step(std::true_type());
        step(std::false_type());
    }

    // the four waves' parts of each head, weighted by their maxima and summed in order
    // (its places are worked out here: kept through the loop they would take registers that it does not have)
    int late = tid;
    asm volatile("" : "+v"(late));
    const int lc = late & 15, lg = (late & 63) >> 4;
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (lg == 0) {
        lds_m[wave][lc] = m;
        lds_l[wave][lc] = l;
    }
    const int64_t part = ((int64_t)slot * gridDim.y + y) * a.tile_heads;
#pragma unroll
    for (int n = 0; n < NH; ++n) {
        if (n) __syncthreads();
        // lane (c, g) holds 4 VEC entries of head c in a row, from 4 VEC g on in its half
        if (lc < heads)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < VEC; j += 4)
                    *reinterpret_cast<f32x4*>(&lds_o[wave][lc][4 * VEC * lg + VEC * i + j]) =
                        f32x4{o[n][j][i], o[n][j + 1][i], o[n][j + 2][i], o[n][j + 3][i]};
        __syncthreads();
        for (int it = late; it < heads * (W / 4); it += 64 * kWaves) {
            const int h = it / (W / 4), d = (it & (W / 4 - 1)) * 4, at = 128 * n + d;
            if (!FULL && at >= a.dim) continue;
            f32x4 sum = {0, 0, 0, 0};
            float top = -INFINITY, den = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) top = fmaxf(top, lds_m[w][h]);
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float f = lds_m[w][h] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(lds_m[w][h] - top);
                sum += *reinterpret_cast<const f32x4*>(&lds_o[w][h][d]) * f;
                den = fmaf(lds_l[w][h], f, den);
            }
            if (!whole_request) {
                *reinterpret_cast<f32x4*>(a.part_o + (part + h) * a.dim + at) = sum;
                if (at == 0) a.part_ml[part + h] = float2{top, den};
            } else {
                const float inv = den == 0.0f ? 0.0f : v_scale / den;
                uint16_t* out = a.O + b * a.ldo + (int64_t)(head0 + h) * a.dim + at;
                *reinterpret_cast<uint2*>(out) = uint2{narrow2<T>(sum[0] * inv, sum[1] * inv),
                                                       narrow2<T>(sum[2] * inv, sum[3] * inv)};
                if (at == 0 && a.lse)
                    a.lse[(int64_t)b * a.q_heads + head0 + h] = den == 0.0f ? -INFINITY : (top - kShift + log2f(den)) * kLn2;
            }
        }
    }
    if (run.left) __syncthreads();       // the next request's parts go to the same LDS
    }
}

// The place of part i of request b's head h (query head) in the workspace: the first part's slot, then the first
// slot of each run after it.
struct Parts {
    uint32_t first;
    int64_t rows, at, heads;
    __device__ __forceinline__ Parts(const AttnArgs& a, uint2 plan, int h) {
        const int group = a.q_heads / a.k_heads, hk = h / group, gh = h - hk * group;
        first = plan.x;
        rows = (int64_t)a.k_heads * a.head_tiles;
        at = (int64_t)(hk * a.head_tiles + gh / 16) * a.tile_heads + (gh & 15);
        heads = rows * a.tile_heads;
    }
    __device__ __forceinline__ int64_t operator()(int i) const {
        return (int64_t)(i ? 2 * (first / 2 + i) : first) * heads + at;
    }
};
template <typename T>
__device__ __forceinline__ void write_joined(const AttnArgs& a, int b, int h, int d, f32x4 sum, float l, float top) {
    const float inv = l == 0.0f ? 0.0f : (a.v_scale ? a.v_scale[h / (a.q_heads / a.k_heads)] : 1.0f) / l;
    *reinterpret_cast<uint2*>(a.O + b * a.ldo + (int64_t)h * a.dim + d) =
        uint2{narrow2<T>(sum[0] * inv, sum[1] * inv), narrow2<T>(sum[2] * inv, sum[3] * inv)};
    if (d == 0 && a.lse) a.lse[(int64_t)b * a.q_heads + h] = l == 0.0f ? -INFINITY : (top - kShift + log2f(l)) * kLn2;
}

// Join of many heads of few parts: a thread takes four entries of one head through all its parts, in order, with a
// running maximum; nothing is shared.
constexpr int kFlatThreads = 256, kFlatParts = 4;
template <typename T>
__global__ __launch_bounds__(kFlatThreads) void join_flat_kernel(AttnArgs a) {
    const int quads = a.dim / 4, per = kFlatThreads / quads, row = threadIdx.x / quads;
    const int64_t i = (blockIdx.y * kGridX + blockIdx.x) * per + row;
    if (row >= per || i >= (int64_t)a.B * a.q_heads) return;
    const int b = (int)(i / a.q_heads), h = (int)(i - (int64_t)b * a.q_heads), d = (threadIdx.x - row * quads) * 4;
    const uint2 plan = a.plan[b];
    if (plan.y <= 1) return;
    const Parts part(a, plan, h);
    float top = -INFINITY, l = 0.0f;
    f32x4 sum = {0, 0, 0, 0};
    for (int base = 0; base < (int)plan.y; base += kFlatParts) {
        f32x4 x[kFlatParts];
        float2 ml[kFlatParts];
#pragma unroll
        for (int k = 0; k < kFlatParts; ++k) {
            x[k] = f32x4{0, 0, 0, 0};
            ml[k] = float2{-INFINITY, 0.0f};
            if (base + k < (int)plan.y) {
                x[k] = *reinterpret_cast<const f32x4*>(a.part_o + part(base + k) * a.dim + d);
                ml[k] = a.part_ml[part(base + k)];
            }
        }
        const float was = top;
#pragma unroll
        for (int k = 0; k < kFlatParts; ++k) top = fmaxf(top, ml[k].x);
        const float f = was == -INFINITY ? 0.0f : exp2f(was - top);
        sum *= f;
        l *= f;
#pragma unroll
        for (int k = 0; k < kFlatParts; ++k) {
            const float w = ml[k].x == -INFINITY ? 0.0f : exp2f(ml[k].x - top);
            sum += x[k] * w;
            l += ml[k].y * w;
        }
    }
    write_joined<T>(a, b, h, d, sum, l, top);
}

// Join of few heads, which may have many parts each: one workgroup per request and query head.  Row r of dim / 4
// lanes takes parts r, r + rows, ..., 8 at a time (the first ones' loads do not wait for the weights); the rows' sums
// are added in order.
constexpr int kJoinThreads = 256, kJoinParts = 8;
template <typename T>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(AttnArgs a) {
    __shared__ f32x4 lds[kJoinThreads];
    __shared__ float lds_m[kJoinThreads / 64], lds_l[kJoinThreads / 64];
    constexpr int threads = kJoinThreads, waves = threads / 64;
    const int b = blockIdx.x, h = blockIdx.y;
    const uint2 plan = a.plan[b];
    const int parts = (int)plan.y;
    if (parts <= 1) return;
    const Parts part(a, plan, h);
    const int tid = threadIdx.x, lane = tid & 63;
    const int quads = a.dim / 4, rows = threads / quads, row = tid / quads, d = (tid - row * quads) * 4;
    f32x4 x[kJoinParts];
    float m[kJoinParts];
    const auto load = [&](int base) {
#pragma unroll
        for (int k = 0; k < kJoinParts; ++k) {
            const int i = base + k * rows;
            x[k] = f32x4{0, 0, 0, 0};
            m[k] = -INFINITY;
            if (row < rows && i < parts) {
                x[k] = *reinterpret_cast<const f32x4*>(a.part_o + part(i) * a.dim + d);
                m[k] = a.part_ml[part(i)].x;
            }
        }
    };
    load(row);
    float2 ml = {-INFINITY, 0.0f};       // this thread's part of the maximum and the sum
    if (tid < parts) ml = a.part_ml[part(tid)];
    float top = ml.x;
    for (int i = tid + threads; i < parts; i += threads) top = fmaxf(top, a.part_ml[part(i)].x);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    if (lane == 0) lds_m[tid >> 6] = top;
    __syncthreads();
    for (int w = 0; w < waves; ++w) top = fmaxf(top, lds_m[w]);
    const auto weight = [&](float v) { return v == -INFINITY ? 0.0f : exp2f(v - top); };
    f32x4 sum = {0, 0, 0, 0};
    for (int base = row;;) {
#pragma unroll
        for (int k = 0; k < kJoinParts; ++k) sum += x[k] * weight(m[k]);
        base += kJoinParts * rows;
        if (row >= rows || base >= parts) break;
        load(base);
    }
    lds[tid] = sum;
    float l = ml.y * weight(ml.x);
    for (int i = tid + threads; i < parts; i += threads) {
        const float2 v = a.part_ml[part(i)];
        l += v.y * weight(v.x);
    }
    l = wave_sum(l);
    if (lane == 0) lds_l[tid >> 6] = l;
    __syncthreads();
    if (row) return;
    l = 0.0f;
    for (int w = 0; w < waves; ++w) l += lds_l[w];
    sum = f32x4{0, 0, 0, 0};
    for (int r = 0; r < rows; ++r) sum += lds[r * quads + tid];
    write_joined<T>(a, b, h, d, sum, l, top);
}

// Tokens of a step.  16 leave room for more waves, or for heads above 128 entries without spills (16 requests up to
// 8192, 16/4 heads of 256: 57.7 us against 71.1; 32/8 heads of 64: 34.5 against 35.9; 64 up to 8191 on an 8-bit cache:
// 102.5 against 104.3; there of 64: 143 up to 1500, 10/10 heads 47.7 against 49.4, 64 up to 4096, 32/8 36.8 against 38.2);
// 32 keep more of a long 16-bit cache of 128-entry heads in flight per wave (4 requests up to
// 131072: 236.8 against 241.7, 32 up to 4096: 58.4 against 59.8), and halve the steps of a request that is not cut.
template <bool C8, int DP, bool FULL, bool SPLIT>
constexpr int kTok = DP == 256 || (SPLIT && !(DP == 128 && FULL && !C8)) ? 16 : 32;
template <typename T, bool C8, bool SPLIT>
void launch_runs(const AttnArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(SPLIT ? a.runs : a.B), (unsigned)(a.k_heads * a.head_tiles)), block(64 * kWaves);
    if (a.dim == 64) attn_kernel<T, C8, 64, true, SPLIT, kTok<C8, 64, true, SPLIT>><<<grid, block, 0, s>>>(a);
    else if (a.dim < 64) attn_kernel<T, C8, 64, false, SPLIT, kTok<C8, 64, false, SPLIT>><<<grid, block, 0, s>>>(a);
    else if (a.dim == 128) attn_kernel<T, C8, 128, true, SPLIT, kTok<C8, 128, true, SPLIT>><<<grid, block, 0, s>>>(a);
    else if (a.dim < 128) attn_kernel<T, C8, 128, false, SPLIT, kTok<C8, 128, false, SPLIT>><<<grid, block, 0, s>>>(a);
    else if (a.dim == 256) attn_kernel<T, C8, 256, true, SPLIT, kTok<C8, 256, true, SPLIT>><<<grid, block, 0, s>>>(a);
    else attn_kernel<T, C8, 256, false, SPLIT, kTok<C8, 256, false, SPLIT>><<<grid, block, 0, s>>>(a);
}

template <typename T, bool C8>
hipError_t launch(const AttnArgs& a, hipStream_t s) {
    if (a.part_o) launch_runs<T, C8, true>(a, s);
    else launch_runs<T, C8, false>(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part_o) return e;
    // (64 requests up to 8191, 40 heads: 6.9 us with a workgroup per head, 4.9 flat; 4 requests up to 131072, 64 heads,
    // 33 to 43 parts each: 5.2 us with a workgroup per head)
    const int64_t heads = (int64_t)a.B * a.q_heads;
    if (heads <= 512) {
        join_kernel<T><<<dim3((unsigned)a.B, (unsigned)a.q_heads), dim3(kJoinThreads), 0, s>>>(a);
    } else {
        const int64_t per = kFlatThreads / (a.dim / 4);
        const WideGrid wide = wide_grid((heads + per - 1) / per);
        join_flat_kernel<T><<<dim3(wide.x, wide.rest), dim3(kFlatThreads), 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, hipStream_t s) {
    if (a.dtype == HTS_BF16) return a.cache8 ? launch<BF16T, true>(a, s) : launch<BF16T, false>(a, s);
    return a.cache8 ? launch<F16T, true>(a, s) : launch<F16T, false>(a, s);
}

}  // namespace hts
