// C ABI of the steps around the products: page step, rotary positions, paged attention, residual
// norm.  Argument checks and kernel launches; every check happens before anything is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "api_checks.h"
#include "hts.h"
#include "serve_internal.h"

namespace {

using namespace hts::api;

constexpr int64_t kInt32 = int64_t(1) << 31;

hts_status check_aligned(const void* p, size_t bytes, const char* name) {
    if (!p) return fail(HTS_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) & (bytes - 1))
        return fail(HTS_ERR_ALIGN, "%s is not %zu-byte aligned", name, bytes);
    return HTS_OK;
}

hts_status check_page(int32_t page) {
    if (page < 16 || page > 1024 || (page & (page - 1)))
        return fail(HTS_ERR_UNSUPPORTED, "page=%d is not a power of two from 16 to 1024", page);
    return HTS_OK;
}

hts_status check_heads(int32_t dtype, int32_t dim) {
    if (!is16bit(dtype)) return fail(HTS_ERR_DTYPE, "dtype %d is not HTS_F16 or HTS_BF16", dtype);
    if (dim < 8 || dim > 256 || dim % 8)
        return fail(HTS_ERR_UNSUPPORTED, "head size %d is not a multiple of 8 from 8 to 256", dim);
    return HTS_OK;
}

// The cache's description against the type it is used with; *elements: where its last one ends.
hts_status check_kv(const hts_kv_desc* kv, int32_t dtype, const float* k_scale, const float* v_scale,
                    uint64_t* elements) {
    if (!kv) return fail(HTS_ERR_INVALID_ARG, "cache descriptor is NULL");
    if (kv->dtype != HTS_FP8_E4M3 && !is16bit(kv->dtype))
        return fail(HTS_ERR_DTYPE, "cache dtype %d is not HTS_F16, HTS_BF16 or HTS_FP8_E4M3", kv->dtype);
    hts_status st;
    if ((st = check_heads(dtype, kv->dim)) || (st = check_page(kv->page))) return st;
    if (kv->dtype != dtype && kv->dtype != HTS_FP8_E4M3)
        return fail(HTS_ERR_DTYPE, "a 16-bit cache must have the type of the inputs");
    if (kv->dtype != HTS_FP8_E4M3 && (k_scale || v_scale))
        return fail(HTS_ERR_INVALID_ARG, "k_scale and v_scale belong to 8-bit caches");
    if (k_scale && (st = check_aligned(k_scale, 4, "k_scale"))) return st;
    if (v_scale && (st = check_aligned(v_scale, 4, "v_scale"))) return st;
    if (kv->pages < 1 || kv->pages >= kInt32)
        return fail(HTS_ERR_SHAPE, "pages=%lld is not from 1 to 2^31 - 1", (long long)kv->pages);
    if (kv->heads < 1 || kv->heads > 65535) return fail(HTS_ERR_SHAPE, "heads=%d is not from 1 to 65535", kv->heads);
    struct Axis {
        int64_t n, stride;
        const char* name;
    } ax[3] = {{kv->pages, kv->page_stride, "page_stride"},
               {kv->page, kv->token_stride, "token_stride"},
               {kv->heads, kv->head_stride, "head_stride"}};
    for (auto& x : ax) {
        if (x.n == 1) x.stride = int64_t(1) << 61;   // not used; sorts last
        else if (&x == &ax[1] && x.stride >= (int64_t(1) << 26))
            return fail(HTS_ERR_UNSUPPORTED, "token_stride=%lld is not below 2^26", (long long)x.stride);
        else if (x.stride <= 0 || x.stride >= (int64_t(1) << 48))
            return fail(HTS_ERR_SHAPE, "%s=%lld is not positive (below 2^48)", x.name, (long long)x.stride);
        else if (x.stride % 8)
            return fail(HTS_ERR_ALIGN, "%s=%lld is not a multiple of 8", x.name, (long long)x.stride);
    }
    std::sort(ax, ax + 3, [](const Axis& p, const Axis& q) { return p.stride < q.stride; });
    __int128 end = kv->dim;
    for (const auto& x : ax) {
        if (x.n == 1) continue;
        if (x.stride < end)
            return fail(HTS_ERR_SHAPE, "%s=%lld lets elements of the cache share a place", x.name, (long long)x.stride);
        end += (__int128)(x.n - 1) * x.stride;
        if (end >= ((__int128)1 << 60)) return fail(HTS_ERR_SHAPE, "the cache spans more than 2^60 elements");
    }
    if (elements) *elements = (uint64_t)end;
    return HTS_OK;
}

int kv_bytes(const hts_kv_desc* kv) { return kv->dtype == HTS_FP8_E4M3 ? 1 : 2; }
int log2i(int32_t x) { return 31 - __builtin_clz((unsigned)x); }
bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na && nb && x < y + nb && y < x + na;
}

hts_status check_table(const int32_t* table, int64_t B, int64_t ldt, int64_t width) {
    if (width < 1 || width >= kInt32) return fail(HTS_ERR_SHAPE, "width=%lld is not from 1 to 2^31 - 1", (long long)width);
    if (ldt < width || ldt >= kInt32)
        return fail(HTS_ERR_SHAPE, "ldt=%lld is not from width=%lld to 2^31 - 1", (long long)ldt, (long long)width);
    return B ? check_aligned(table, 4, "block_table") : HTS_OK;
}

// How hts_paged_attn divides its work: runs per cache head and tile of 16 query heads, as many as the chip
// holds workgroups of them at once.
struct AttnPlan {
    int32_t head_tiles, tile_heads, runs, target;
    uint32_t cap, window;
    bool split;
    uint64_t plan_bytes, ml_bytes, bytes;
};
AttnPlan attn_plan(int64_t B, int32_t q_heads, const hts_kv_desc* kv, int64_t width, int64_t window) {
    AttnPlan p{};
    const int32_t group = q_heads / kv->heads;
    p.head_tiles = (group + 15) / 16;
    p.tile_heads = std::min(group, 16);
    p.cap = (uint32_t)std::min<int64_t>(width * kv->page, kInt32 - 1);
    p.window = (uint32_t)std::min<int64_t>(window, kInt32 - 1);
    const int64_t rows = (int64_t)kv->heads * p.head_tiles;
    const uint64_t most = window ? std::min<uint64_t>(p.cap, (uint64_t)p.window + 31) : p.cap;
    const uint64_t steps = (uint64_t)B * ((most + 31) / 32);
    // 256 CUs hold three or four workgroups each, two of those for heads above 128 entries.  Four pay for smaller heads
    // of 16 bits (16 requests up to 4096, 16/4 heads of 96: 17.0 us with 1024 runs, 18.3 with 768; 64 requests up to 8191
    // on an 8-bit cache: 113.9 and 112.4).  Fewer stream as fast where each has long stretches to itself, and leave
    // fewer parts: one a CU for heads above 128 (16 requests up to 8192, 16/4 heads of 256: 58.2 us with 256 runs, 59.7
    // with 512; of 192 46.5 and 48.1; on an 8-bit cache 37.1 and 37.3, of 192 33.5 and 32.9; 30 up to 1142 there, 5/5 of
    // 192: 22.1 and 26.2; 64 up to 2048, 8/8 of 160: 71.3 and 70.7), two where a page holds a head's tokens one after another (256 requests up to 2048, 32/8 heads, pages
    // of 64: 200 us with 512, 206 with 768; with the heads of a token together, 221 and 209), as it does where there is one
    // head, whose stride is not used (64 up to 8191, 16/1 heads: 36.1 us with 512, 40.1 with 768; 4 up to 131072, 8/1: 39.9
    // and 42.0; 32 up to 4096, 4/1: 14.8 and 14.7).
    const bool in_a_row = kv->heads == 1 || kv->head_stride > kv->token_stride;
    const int64_t runs = kv->dim > 128 ? 256
                         : in_a_row    ? 512
                         : kv->dim < 128 && kv->dtype != HTS_FP8_E4M3 ? 1024
                                                                      : 768;
    p.target = (int32_t)std::max<int64_t>(1, runs / rows);
    const uint64_t least = std::min<uint64_t>(std::max<uint64_t>(3 * steps / p.target, 4), 16);   // as in the kernel
    p.runs = (int32_t)std::min<uint64_t>(p.target, std::max<uint64_t>(B, (steps + least - 1) / least));
    p.split = B >= 1 && B <= hts::kMaxSplitRequests && most > hts::kAttnWholeTokens && steps < (uint64_t)kInt32;
    if (p.split) {
        const uint64_t parts = 2 * (uint64_t)p.runs * rows * p.tile_heads;
        p.plan_bytes = (8 * (uint64_t)B + 255) & ~uint64_t(255);
        p.ml_bytes = (8 * parts + 255) & ~uint64_t(255);
        p.bytes = p.plan_bytes + p.ml_bytes + 4 * parts * kv->dim;
    }
    return p;
}

hts_status check_rope(const hts_rope_desc* d, const double* turns, int64_t T, const int32_t* positions) {
    if (!d) return fail(HTS_ERR_INVALID_ARG, "descriptor is NULL");
    if (d->reserved != 0) return fail(HTS_ERR_INVALID_ARG, "descriptor reserved field must be 0");
    hts_status st = check_heads(d->dtype, d->dim);
    if (st) return st;
    if (d->layout != HTS_ROPE_HALF && d->layout != HTS_ROPE_INTERLEAVED)
        return fail(HTS_ERR_INVALID_ARG, "layout %d is not HTS_ROPE_HALF or HTS_ROPE_INTERLEAVED", d->layout);
    if (d->rot < 8 || d->rot > d->dim || d->rot % 8)
        return fail(HTS_ERR_UNSUPPORTED, "rot=%d is not a multiple of 8 from 8 to the head size %d", d->rot, d->dim);
    if (d->q_heads < 0 || d->k_heads < 0 || d->q_heads > 65535 || d->k_heads > 65535)
        return fail(HTS_ERR_SHAPE, "q_heads=%d k_heads=%d are not from 0 to 65535", d->q_heads, d->k_heads);
    if (!std::isfinite(d->magnitude)) return fail(HTS_ERR_INVALID_ARG, "magnitude is not finite");
    if (T < 0 || T >= kInt32) return fail(HTS_ERR_SHAPE, "T=%lld is not from 0 to 2^31 - 1", (long long)T);
    if (T == 0) return HTS_OK;
    if ((st = check_aligned(turns, 8, "turns")) || (st = check_aligned(positions, 4, "positions"))) return st;
    return HTS_OK;
}

// One matrix [T, heads*dim]; nothing to check where there are no heads.
hts_status check_matrix(const void* p, int64_t ld, int64_t cols, const char* name, const char* ld_name) {
    if (!cols) return HTS_OK;
    hts_status st = check_ptr(p, name);
    return st ? st : check_ld(ld, cols, 8, ld_name);
}

hts::RopeArgs rope_args(const hts_rope_desc* d, const double* turns, int64_t T, const int32_t* positions) {
    hts::RopeArgs a{};
    a.dtype = d->dtype;
    a.layout = d->layout;
    a.dim = d->dim;
    a.rot = d->rot;
    a.q_heads = d->q_heads;
    a.k_heads = d->k_heads;
    a.magnitude = d->magnitude;
    a.T = T;
    a.turns = turns;
    a.positions = positions;
    return a;
}

// hts_rope_cache of T tokens, or with `starts` of T requests whose tokens lie among `tokens`.
hts_status rope_cache(const hts_rope_desc* d, const double* turns, int64_t T, const int32_t* starts, int64_t tokens,
                      const int32_t* positions, const int64_t* slots, const void* Q, int64_t ldq, void* Q_out, int64_t ldqo,
                      const void* K, int64_t ldk, const void* V, int64_t ldv, const hts_kv_desc* kv, void* k_cache,
                      void* v_cache, const float* k_scale, const float* v_scale, void* stream) {
    hts_status st = check_rope(d, turns, T, positions);
    if (st) return st;
    uint64_t span = 0;
    if ((st = check_kv(kv, d->dtype, k_scale, v_scale, &span))) return st;
    if (kv->dim != d->dim || kv->heads != d->k_heads)
        return fail(HTS_ERR_SHAPE, "the cache holds %d heads of %d, the step %d of %d", kv->heads, kv->dim, d->k_heads,
                    d->dim);
    if (T == 0) return ok();
    const int64_t nq = (int64_t)d->q_heads * d->dim, nk = (int64_t)d->k_heads * d->dim;
    if ((st = check_matrix(Q, ldq, nq, "Q", "ldq")) || (st = check_matrix(Q_out, ldqo, nq, "Q_out", "ldqo")) ||
        (st = check_matrix(K, ldk, nk, "K", "ldk")) || (st = check_matrix(V, ldv, nk, "V", "ldv")) ||
        (st = check_ptr(k_cache, "k_cache")) || (st = check_ptr(v_cache, "v_cache")) ||
        (st = check_aligned(slots, 8, "slots")))
        return st;
    if (k_cache == v_cache) return fail(HTS_ERR_INVALID_ARG, "k_cache and v_cache are one buffer");
    if (nq && Q_out == Q && ldqo != ldq)
        return fail(HTS_ERR_INVALID_ARG, "in place, input and output have one leading dimension");
    const int es = kv_bytes(kv);
    if (debug_mode() &&
        ((st = debug_range(turns, 4 * (uint64_t)d->rot, "turns")) ||
         (st = debug_range(positions, 4 * (uint64_t)tokens, "positions")) ||
         (st = debug_range(slots, 8 * (uint64_t)tokens, "slots")) ||
         (starts && (st = debug_range(starts, 4 * ((uint64_t)T + 1), "starts"))) ||
         (nq && ((st = debug_range(Q, block_bytes(T, nq, ldq, 2), "Q")) ||
                 (st = debug_range(Q_out, block_bytes(T, nq, ldqo, 2), "Q_out")))) ||
         (st = debug_range(K, block_bytes(T, nk, ldk, 2), "K")) || (st = debug_range(V, block_bytes(T, nk, ldv, 2), "V")) ||
         (st = debug_range(k_cache, span * es, "k_cache")) || (st = debug_range(v_cache, span * es, "v_cache")) ||
         (st = debug_range(k_scale, 4 * (uint64_t)kv->heads, "k_scale")) ||
         (st = debug_range(v_scale, 4 * (uint64_t)kv->heads, "v_scale"))))
        return st;
    hts::RopeArgs a = rope_args(d, turns, T, positions);
    a.Q = static_cast<const uint16_t*>(Q);
    a.ldq = ldq;
    a.Qo = static_cast<uint16_t*>(Q_out);
    a.ldqo = ldqo;
    a.K = static_cast<const uint16_t*>(K);
    a.ldk = ldk;
    a.V = static_cast<const uint16_t*>(V);
    a.ldv = ldv;
    a.slots = slots;
    a.starts = starts;
    a.tokens = tokens;
    a.kc = k_cache;
    a.vc = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.n_slots = kv->pages * kv->page;
    a.cache8 = kv->dtype == HTS_FP8_E4M3;
    a.page_shift = log2i(kv->page);
    a.page_stride = kv->page_stride;
    a.token_stride = kv->token_stride;
    a.head_stride = kv->head_stride;
    return hip_status(hts::launch_rope(a, static_cast<hipStream_t>(stream)), "rotary kernel launch");
}

}  // namespace

extern "C" {

hts_status hts_kv_step(int64_t B, const int32_t* cached, const int32_t* added, int32_t page,
                       const int32_t* free_pages, int64_t n_free, const int32_t* free_head, int32_t* block_table,
                       int64_t ldt, int64_t width, int64_t tokens, int32_t* lengths, int32_t* starts, int64_t* slots,
                       int32_t* positions, int32_t* head_out, void* stream) {
    hts_status st = check_page(page);
    if (st) return st;
    if (B < 0) return fail(HTS_ERR_SHAPE, "B=%lld is negative", (long long)B);
    if (B > hts::kMaxStepRequests)
        return fail(HTS_ERR_UNSUPPORTED, "B=%lld requests exceed %d", (long long)B, hts::kMaxStepRequests);
    if (n_free < 0 || n_free >= kInt32 || tokens < 0 || tokens >= kInt32)
        return fail(HTS_ERR_SHAPE, "n_free=%lld tokens=%lld are not from 0 to 2^31 - 1", (long long)n_free,
                    (long long)tokens);
    if ((st = check_table(block_table, B, ldt, width))) return st;
    if (B * width >= kInt32) return fail(HTS_ERR_SHAPE, "B * width must be below 2^31");
    if (B && ((st = check_aligned(cached, 4, "cached")) || (st = check_aligned(added, 4, "added")) ||
              (st = check_aligned(lengths, 4, "lengths"))))
        return st;
    if (n_free && (st = check_aligned(free_pages, 4, "free_pages"))) return st;
    if (free_head && (st = check_aligned(free_head, 4, "free_head"))) return st;
    if ((st = check_aligned(starts, 4, "starts")) || (st = check_aligned(head_out, 4, "head_out"))) return st;
    if (tokens && ((st = check_aligned(slots, 8, "slots")) || (st = check_aligned(positions, 4, "positions")))) return st;
    // every workgroup reads the inputs, so nothing may be written over them
    const uint64_t rows = 4 * (uint64_t)B, table_bytes = block_bytes(B, width, ldt, 4);
    const struct {
        const void* p;
        uint64_t n;
    } in[4] = {{cached, rows}, {added, rows}, {free_pages, 4 * (uint64_t)n_free}, {free_head, free_head ? 4u : 0u}},
      out[6] = {{lengths, rows},   {starts, rows + 4},       {slots, 8 * (uint64_t)tokens}, {positions, 4 * (uint64_t)tokens},
                {head_out, 4}, {block_table, table_bytes}};
    for (int i = 0; i < 6; ++i) {
        for (const auto& x : in)
            if (overlap(x.p, x.n, out[i].p, out[i].n))
                return fail(HTS_ERR_INVALID_ARG, "an output of the step overlaps an input");
        for (int j = 0; j < i; ++j)
            if (overlap(out[j].p, out[j].n, out[i].p, out[i].n))
                return fail(HTS_ERR_INVALID_ARG, "two outputs of the step overlap");
    }
    if (debug_mode() &&
        ((st = debug_range(cached, rows, "cached")) || (st = debug_range(added, rows, "added")) ||
         (st = debug_range(free_pages, 4 * (uint64_t)n_free, "free_pages")) ||
         (st = debug_range(free_head, 4, "free_head")) || (st = debug_range(block_table, table_bytes, "block_table")) ||
         (st = debug_range(lengths, rows, "lengths")) || (st = debug_range(starts, rows + 4, "starts")) ||
         (st = debug_range(slots, 8 * (uint64_t)tokens, "slots")) ||
         (st = debug_range(positions, 4 * (uint64_t)tokens, "positions")) || (st = debug_range(head_out, 4, "head_out"))))
        return st;
    hts::KvStepArgs a{};
    a.B = (int32_t)B;
    a.page_shift = log2i(page);
    a.cached = cached;
    a.added = added;
    a.free_pages = free_pages;
    a.n_free = n_free;
    a.free_head = free_head;
    a.table = block_table;
    a.ldt = ldt;
    a.width = width;
    a.tokens = tokens;
    a.lengths = lengths;
    a.starts = starts;
    a.slots = slots;
    a.positions = positions;
    a.head_out = head_out;
    return hip_status(hts::launch_kv_step(a, static_cast<hipStream_t>(stream)), "page-step kernel launch");
}

hts_status hts_rope_plan(const hts_rope_scaling* s, double* turns_host) {
    if (!s) return fail(HTS_ERR_INVALID_ARG, "scaling is NULL");
    if (!turns_host) return fail(HTS_ERR_INVALID_ARG, "turns_host is NULL");
    if (s->rot < 8 || s->rot > 256 || s->rot % 8)
        return fail(HTS_ERR_UNSUPPORTED, "rot=%d is not a multiple of 8 from 8 to 256", s->rot);
    if (s->rule < HTS_ROPE_PLAIN || s->rule > HTS_ROPE_RAMP_PAIRS)
        return fail(HTS_ERR_INVALID_ARG, "rule %d is not a scaling rule", s->rule);
    if (!(std::isfinite(s->theta) && s->theta > 1.0)) return fail(HTS_ERR_INVALID_ARG, "theta must be above 1");
    if (!(std::isfinite(s->factor) && s->factor >= 1.0)) return fail(HTS_ERR_INVALID_ARG, "factor must be at least 1");
    const bool ramp = s->rule == HTS_ROPE_RAMP || s->rule == HTS_ROPE_RAMP_PAIRS;
    if (ramp && !(std::isfinite(s->context) && s->context > 0.0 && s->low > 0.0 && s->high > s->low && std::isfinite(s->high)))
        return fail(HTS_ERR_INVALID_ARG, "a ramp takes context > 0 and 0 < low < high");
    const double two_pi = 6.283185307179586476925;
    const int R = s->rot;
    const double theta = s->rule == HTS_ROPE_BASE ? s->theta * std::pow(s->factor, R / (R - 2.0)) : s->theta;
    if (!std::isfinite(theta)) return fail(HTS_ERR_INVALID_ARG, "theta scaled by factor is not finite");
    // pair index with n turns over the context
    const auto pair = [&](double n) { return R * std::log(s->context / (two_pi * n)) / (2.0 * std::log(s->theta)); };
    double first = 0.0, last = 0.0;
    if (s->rule == HTS_ROPE_RAMP_PAIRS) {
        first = std::min(std::max(std::floor(pair(s->high)), 0.0), R - 1.0);
        last = std::min(std::max(std::ceil(pair(s->low)), 0.0), R - 1.0);
    }
    for (int i = 0; i < R / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / R);
        if (s->rule == HTS_ROPE_LINEAR) f /= s->factor;
        if (ramp) {
            double c = s->rule == HTS_ROPE_RAMP ? (s->context * f / two_pi - s->low) / (s->high - s->low)
                                                : 1.0 - (i - first) / std::max(last - first, 1e-3);
            c = std::min(std::max(c, 0.0), 1.0);
            f *= c + (1.0 - c) / s->factor;
        }
        turns_host[i] = f / two_pi;
    }
    return ok();
}

hts_status hts_rope(const hts_rope_desc* d, const double* turns, int64_t T, const int32_t* positions, const void* Q,
                    int64_t ldq, void* Q_out, int64_t ldqo, const void* K, int64_t ldk, void* K_out, int64_t ldko,
                    void* stream) {
    hts_status st = check_rope(d, turns, T, positions);
    if (st) return st;
    const int64_t nq = (int64_t)d->q_heads * d->dim, nk = (int64_t)d->k_heads * d->dim;
    if (T == 0 || (nq == 0 && nk == 0)) return ok();
    if ((st = check_matrix(Q, ldq, nq, "Q", "ldq")) || (st = check_matrix(Q_out, ldqo, nq, "Q_out", "ldqo")) ||
        (st = check_matrix(K, ldk, nk, "K", "ldk")) || (st = check_matrix(K_out, ldko, nk, "K_out", "ldko")))
        return st;
    if ((nq && Q_out == Q && ldqo != ldq) || (nk && K_out == K && ldko != ldk))
        return fail(HTS_ERR_INVALID_ARG, "in place, input and output have one leading dimension");
    if (debug_mode() &&
        ((st = debug_range(turns, 4 * (uint64_t)d->rot, "turns")) || (st = debug_range(positions, 4 * (uint64_t)T, "positions")) ||
         (nq && ((st = debug_range(Q, block_bytes(T, nq, ldq, 2), "Q")) ||
                 (st = debug_range(Q_out, block_bytes(T, nq, ldqo, 2), "Q_out")))) ||
         (nk && ((st = debug_range(K, block_bytes(T, nk, ldk, 2), "K")) ||
                 (st = debug_range(K_out, block_bytes(T, nk, ldko, 2), "K_out"))))))
        return st;
    hts::RopeArgs a = rope_args(d, turns, T, positions);
    a.Q = static_cast<const uint16_t*>(Q);
    a.ldq = ldq;
    a.Qo = static_cast<uint16_t*>(Q_out);
    a.ldqo = ldqo;
    a.K = static_cast<const uint16_t*>(K);
    a.ldk = ldk;
    a.Ko = static_cast<uint16_t*>(K_out);
    a.ldko = ldko;
    return hip_status(hts::launch_rope(a, static_cast<hipStream_t>(stream)), "rotary kernel launch");
}

hts_status hts_rope_cache(const hts_rope_desc* d, const double* turns, int64_t T, const int32_t* positions,
                          const int64_t* slots, const void* Q, int64_t ldq, void* Q_out, int64_t ldqo, const void* K,
                          int64_t ldk, const void* V, int64_t ldv, const hts_kv_desc* kv, void* k_cache, void* v_cache,
                          const float* k_scale, const float* v_scale, void* stream) {
    return rope_cache(d, turns, T, nullptr, T, positions, slots, Q, ldq, Q_out, ldqo, K, ldk, V, ldv, kv, k_cache, v_cache,
                      k_scale, v_scale, stream);
}

hts_status hts_rope_cache_rows(const hts_rope_desc* d, const double* turns, int64_t B, const int32_t* starts,
                               int64_t tokens, const int32_t* positions, const int64_t* slots, const void* Q, int64_t ldq,
                               void* Q_out, int64_t ldqo, const void* K, int64_t ldk, const void* V, int64_t ldv,
                               const hts_kv_desc* kv, void* k_cache, void* v_cache, const float* k_scale,
                               const float* v_scale, void* stream) {
    if (tokens < (B > 0) || tokens >= kInt32)
        return fail(HTS_ERR_SHAPE, "tokens=%lld is not from 1 to 2^31 - 1", (long long)tokens);
    if (B > 0) {
        const hts_status st = check_aligned(starts, 4, "starts");
        if (st) return st;
    }
    return rope_cache(d, turns, B, starts, tokens, positions, slots, Q, ldq, Q_out, ldqo, K, ldk, V, ldv, kv, k_cache,
                      v_cache, k_scale, v_scale, stream);
}

hts_status hts_paged_attn_workspace(int64_t B, int32_t q_heads, const hts_kv_desc* kv, int64_t width, int64_t window,
                                    size_t* bytes) {
    if (!bytes) return fail(HTS_ERR_INVALID_ARG, "bytes is NULL");
    if (B < 0 || B > 65535) return fail(HTS_ERR_SHAPE, "B=%lld is not from 0 to 65535", (long long)B);
    hts_status st = check_kv(kv, kv && kv->dtype == HTS_BF16 ? HTS_BF16 : HTS_F16, nullptr, nullptr, nullptr);
    if (st) return st;
    if (q_heads < 1 || q_heads > 65535 || q_heads % kv->heads)
        return fail(HTS_ERR_SHAPE, "q_heads=%d is not a multiple of the cache's %d heads (up to 65535)", q_heads, kv->heads);
    if (width < 1 || width >= kInt32) return fail(HTS_ERR_SHAPE, "width=%lld is not from 1 to 2^31 - 1", (long long)width);
    if (window < 0) return fail(HTS_ERR_SHAPE, "window=%lld is negative", (long long)window);
    *bytes = (size_t)attn_plan(B, q_heads, kv, width, window).bytes;
    return ok();
}

hts_status hts_paged_attn(int32_t dtype, int64_t B, int32_t q_heads, const hts_kv_desc* kv, const void* Q, int64_t ldq,
                          const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                          const int32_t* block_table, int64_t ldt, int64_t width, const int32_t* lengths, float scale,
                          int64_t window, void* O, int64_t ldo, float* lse, void* workspace, size_t workspace_bytes,
                          void* stream) {
    uint64_t span = 0;
    hts_status st = check_kv(kv, dtype, k_scale, v_scale, &span);
    if (st) return st;
    if (B < 0 || B > 65535) return fail(HTS_ERR_SHAPE, "B=%lld is not from 0 to 65535", (long long)B);
    if (q_heads < 1 || q_heads > 65535 || q_heads % kv->heads)
        return fail(HTS_ERR_SHAPE, "q_heads=%d is not a multiple of the cache's %d heads (up to 65535)", q_heads, kv->heads);
    if (!std::isfinite(scale)) return fail(HTS_ERR_INVALID_ARG, "scale is not finite");
    if (window < 0) return fail(HTS_ERR_SHAPE, "window=%lld is negative", (long long)window);
    const int64_t n = (int64_t)q_heads * kv->dim;
    if ((int64_t)kv->heads * ((q_heads / kv->heads + 15) / 16) > 65535)
        return fail(HTS_ERR_UNSUPPORTED, "cache heads times tiles of 16 query heads exceed 65535");
    if ((st = check_table(block_table, B, ldt, width)) || (st = check_ld(ldq, n, 8, "ldq")) ||
        (st = check_ld(ldo, n, 8, "ldo")))
        return st;
    if (B == 0) return ok();
    if ((st = check_ptr(Q, "Q")) || (st = check_ptr(O, "O")) || (st = check_ptr(k_cache, "k_cache")) ||
        (st = check_ptr(v_cache, "v_cache")) || (st = check_aligned(lengths, 4, "lengths")))
        return st;
    if (O == Q && ldo != ldq) return fail(HTS_ERR_INVALID_ARG, "in place, Q and O have one leading dimension");
    if (lse && (st = check_aligned(lse, 4, "lse"))) return st;
    if (workspace && !aligned16(workspace)) return fail(HTS_ERR_ALIGN, "workspace is not 16-byte aligned");
    const int es = kv_bytes(kv);
    if (debug_mode() &&
        ((st = debug_range(Q, block_bytes(B, n, ldq, 2), "Q")) || (st = debug_range(O, block_bytes(B, n, ldo, 2), "O")) ||
         (st = debug_range(k_cache, span * es, "k_cache")) || (st = debug_range(v_cache, span * es, "v_cache")) ||
         (st = debug_range(k_scale, 4 * (uint64_t)kv->heads, "k_scale")) ||
         (st = debug_range(v_scale, 4 * (uint64_t)kv->heads, "v_scale")) ||
         (st = debug_range(block_table, block_bytes(B, width, ldt, 4), "block_table")) ||
         (st = debug_range(lengths, 4 * (uint64_t)B, "lengths")) ||
         (st = debug_range(lse, 4 * (uint64_t)B * q_heads, "lse")) ||
         (st = debug_range(workspace, workspace_bytes, "workspace"))))
        return st;
    hts::AttnArgs a{};
    a.dtype = dtype;
    a.cache8 = kv->dtype == HTS_FP8_E4M3;
    a.B = (int32_t)B;
    a.q_heads = q_heads;
    a.k_heads = kv->heads;
    a.dim = kv->dim;
    a.page_shift = log2i(kv->page);
    a.pages = kv->pages;
    a.page_stride = kv->page_stride;
    a.token_stride = kv->token_stride;
    a.head_stride = kv->head_stride;
    a.Q = static_cast<const uint16_t*>(Q);
    a.ldq = ldq;
    a.kc = k_cache;
    a.vc = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.table = block_table;
    a.ldt = ldt;
    a.lengths = lengths;
    a.scale = scale;
    a.O = static_cast<uint16_t*>(O);
    a.ldo = ldo;
    a.lse = lse;
    const AttnPlan p = attn_plan(B, q_heads, kv, width, window);
    a.window = p.window;
    a.cap = p.cap;
    a.head_tiles = p.head_tiles;
    a.tile_heads = p.tile_heads;
    a.runs = p.runs;
    a.target = p.target;
    if (p.split && workspace && workspace_bytes >= p.bytes) {
        char* ws = static_cast<char*>(workspace);
        a.plan = reinterpret_cast<uint2*>(ws);
        a.part_ml = reinterpret_cast<float2*>(ws + p.plan_bytes);
        a.part_o = reinterpret_cast<float*>(ws + p.plan_bytes + p.ml_bytes);
    }
    return hip_status(hts::launch_attn(a, static_cast<hipStream_t>(stream)), "attention kernel launch");
}

hts_status hts_residual_norm(const hts_norm_desc* d, int64_t M, int64_t N, const void* block, int64_t ldb,
                             const void* post_weight, const void* post_bias, const void* gate, int64_t ldg,
                             const void* R, int64_t ldr, const void* pre_weight, const void* pre_bias, void* R_out,
                             int64_t ldro, void* Y, int64_t ldy, void* stream) {
    if (!d) return fail(HTS_ERR_INVALID_ARG, "descriptor is NULL");
    if (!is16bit(d->dtype)) return fail(HTS_ERR_DTYPE, "dtype %d is not HTS_F16 or HTS_BF16", d->dtype);
    if (d->r_dtype != d->dtype && d->r_dtype != HTS_F32)
        return fail(HTS_ERR_DTYPE, "r_dtype %d is neither dtype nor HTS_F32", d->r_dtype);
    const auto kind = [](int32_t k) { return k >= HTS_NORM_NONE && k <= HTS_NORM_LAYER; };
    if (!kind(d->post) || !kind(d->pre)) return fail(HTS_ERR_INVALID_ARG, "post=%d pre=%d: not a norm", d->post, d->pre);
    if (d->gate_act < HTS_GATE_PLAIN || d->gate_act > HTS_GATE_SILU)
        return fail(HTS_ERR_INVALID_ARG, "gate_act %d is not a gate", d->gate_act);
    if (!(std::isfinite(d->post_eps) && d->post_eps >= 0.0f && std::isfinite(d->pre_eps) && d->pre_eps >= 0.0f))
        return fail(HTS_ERR_INVALID_ARG, "post_eps and pre_eps must be finite and not negative");
    if (!std::isfinite(d->scale)) return fail(HTS_ERR_INVALID_ARG, "scale is not finite");
    if (M < 0 || M >= kInt32) return fail(HTS_ERR_SHAPE, "M=%lld is not from 0 to 2^31 - 1", (long long)M);
    if (N < 8 || N % 8) return fail(HTS_ERR_SHAPE, "N=%lld is not a positive multiple of 8", (long long)N);
    if (N > hts::kMaxNormWidth)
        return fail(HTS_ERR_UNSUPPORTED, "N=%lld exceeds the %lld entries of a row held in registers", (long long)N,
                    (long long)hts::kMaxNormWidth);
    if (M == 0) return ok();
    hts_status st;
    if (!block && !R) return fail(HTS_ERR_INVALID_ARG, "block and R are both NULL");
    if (!R_out && !Y) return fail(HTS_ERR_INVALID_ARG, "R_out and Y are both NULL");
    if (!block && (gate || d->post != HTS_NORM_NONE)) return fail(HTS_ERR_INVALID_ARG, "gate and post norm need block");
    if ((block && ((st = check_ptr(block, "block")) || (st = check_ld(ldb, N, 8, "ldb")))) ||
        (gate && ((st = check_ptr(gate, "gate")) || (ldg && (st = check_ld(ldg, N, 8, "ldg"))))) ||
        (R && ((st = check_ptr(R, "R")) || (st = check_ld(ldr, N, 8, "ldr")))) ||
        (R_out && ((st = check_ptr(R_out, "R_out")) || (st = check_ld(ldro, N, 8, "ldro")))) ||
        (Y && ((st = check_ptr(Y, "Y")) || (st = check_ld(ldy, N, 8, "ldy")))))
        return st;
    const struct {
        const void* p;
        const char* name;
    } vec[4] = {{post_weight, "post_weight"}, {post_bias, "post_bias"}, {pre_weight, "pre_weight"}, {pre_bias, "pre_bias"}};
    for (const auto& v : vec)
        if (v.p && (st = check_ptr(v.p, v.name))) return st;
    // in place: one leading dimension, one element size, and no second writer
    const int rs = d->r_dtype == HTS_F32 ? 4 : 2;
    if (Y && R_out && Y == R_out) return fail(HTS_ERR_INVALID_ARG, "R_out and Y are one buffer");
    if (R && ((R_out == R && ldro != ldr) || (Y == R && (ldy != ldr || rs != 2))))
        return fail(HTS_ERR_INVALID_ARG, "in place over R: another leading dimension or type");
    if (block && ((Y == block && ldy != ldb) || (R_out == block && (ldro != ldb || rs != 2))))
        return fail(HTS_ERR_INVALID_ARG, "in place over block: another leading dimension or type");
    if (gate && ((Y == gate && ldy != ldg) || (R_out == gate && (ldro != ldg || rs != 2))))
        return fail(HTS_ERR_INVALID_ARG, "in place over gate: another leading dimension or type");
    if (debug_mode()) {
        if ((st = debug_range(block, block_bytes(M, N, ldb, 2), "block")) ||
            (st = debug_range(gate, block_bytes(ldg ? M : 1, N, ldg, 2), "gate")) ||
            (st = debug_range(R, block_bytes(M, N, ldr, rs), "R")) ||
            (st = debug_range(R_out, block_bytes(M, N, ldro, rs), "R_out")) ||
            (st = debug_range(Y, block_bytes(M, N, ldy, 2), "Y")))
            return st;
        for (const auto& v : vec)
            if ((st = debug_range(v.p, 2 * (uint64_t)N, v.name))) return st;
    }
    hts::NormArgs a{};
    a.dtype = d->dtype;
    a.r32 = d->r_dtype == HTS_F32;
    a.post = d->post;
    a.pre = d->pre;
    a.gate_act = d->gate_act;
    a.post_eps = d->post_eps;
    a.pre_eps = d->pre_eps;
    a.scale = d->scale;
    a.M = M;
    a.N = (int32_t)N;
    a.block = static_cast<const uint16_t*>(block);
    a.ldb = ldb;
    a.post_w = static_cast<const uint16_t*>(post_weight);
    a.post_b = static_cast<const uint16_t*>(post_bias);
    a.gate = static_cast<const uint16_t*>(gate);
    a.ldg = ldg;
    a.R = R;
    a.ldr = ldr;
    a.pre_w = static_cast<const uint16_t*>(pre_weight);
    a.pre_b = static_cast<const uint16_t*>(pre_bias);
    a.R_out = R_out;
    a.ldro = ldro;
    a.Y = static_cast<uint16_t*>(Y);
    a.ldy = ldy;
    return hip_status(hts::launch_residual_norm(a, static_cast<hipStream_t>(stream)), "residual-norm kernel launch");
}

}  // extern "C"
