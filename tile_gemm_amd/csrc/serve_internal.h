// Internal declarations shared by the serving half of the C API and its gfx950 kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hts.h"

namespace hts {

// Workgroups of a launch in two grid axes, n below 2^31 or so: HIP takes fewer than 2^32 threads in one, that is 2^24 of 256
// or 2^22 of 1024.  Workgroup i is (i % kGridX, i / kGridX), and those past n return.
constexpr int64_t kGridX = int64_t(1) << 21;
struct WideGrid {
    unsigned x, rest;
};
inline WideGrid wide_grid(int64_t n) {
    return n <= kGridX ? WideGrid{(unsigned)n, 1u} : WideGrid{(unsigned)kGridX, (unsigned)((n + kGridX - 1) / kGridX)};
}

// hts_kv_step keeps one prefix-sum entry of each kind per request in LDS.
constexpr int kMaxStepRequests = 4096;
struct KvStepArgs {
    int32_t B;
    int32_t page_shift;
    const int32_t *cached, *added;
    const int32_t* free_pages;
    int64_t n_free;
    const int32_t* free_head;
    int32_t* table;
    int64_t ldt, width, tokens;
    int32_t *lengths, *starts;
    int64_t* slots;
    int32_t *positions, *head_out;
};
hipError_t launch_kv_step(const KvStepArgs& a, hipStream_t s);

struct RopeArgs {
    int32_t dtype, layout, dim, rot, q_heads, k_heads;
    float magnitude;
    int64_t T;
    const double* turns;
    const int32_t* positions;
    const uint16_t *Q, *K, *V;
    uint16_t *Qo, *Ko;         // Ko: nullptr where K goes to the cache
    int64_t ldq, ldqo, ldk, ldko, ldv;
    const int64_t* slots;      // nullptr: no cache
    const int32_t* starts;     // nullptr: row t is token t; else T + 1 entries: it is request t's, whose token is starts[t]
    int64_t tokens;            // entries of positions and slots
    void *kc, *vc;
    const float *k_scale, *v_scale;
    int64_t n_slots;
    int32_t cache8, page_shift;
    int64_t page_stride, token_stride, head_stride;
};
hipError_t launch_rope(const RopeArgs& a, hipStream_t s);

struct AttnArgs {
    int32_t dtype, cache8;
    int32_t B, q_heads, k_heads, dim, page_shift;
    int64_t pages, page_stride, token_stride, head_stride;
    const uint16_t* Q;
    int64_t ldq;
    const void *kc, *vc;
    const float *k_scale, *v_scale;
    const int32_t* table;
    int64_t ldt;
    const int32_t* lengths;
    float scale;
    uint32_t window;           // 0: none
    uint32_t cap;              // tokens a row of the table holds
    uint16_t* O;
    int64_t ldo;
    float* lse;
    int32_t head_tiles, tile_heads;   // tiles of 16 query heads to a cache head; heads of a tile (<= 16)
    // Split over the length (part_o not NULL): the steps of 32 tokens of all requests, cut into at most
    // `runs` equal runs; a run leaves at most two parts (of its first and its last request).
    uint32_t target;           // runs of a cache head that the chip holds at once
    int32_t runs;              // at most: fewer where the table's width bounds the steps
    uint2* plan;               // [B]: first part's slot, number of parts
    float2* part_ml;           // [2 runs][k_heads * head_tiles][tile_heads]
    float* part_o;             // the same, [dim]
};
// Requests whose runs every wave finds by one scan; more run unsplit.
constexpr int64_t kMaxSplitRequests = 4096;
// Where no request can be longer, each is one workgroup's (51 requests up to 455 tokens, 21/3 heads of 192: 12.5 us
// against 21.5 in runs with a join; 4 up to 512, 8/2 of 128: 7.9 and 9.2; 64 up to 512, 32/8: 16.6 and 21.1).  Up to
// 1000 tokens a small batch is faster in runs (4 requests, 8/2 of 128: 9.5 against 12.4), a large one slower (51, 21/3
// of 192: 24.5 against 20.2).
constexpr int kAttnWholeTokens = 512;
hipError_t launch_attn(const AttnArgs& a, hipStream_t s);

constexpr int64_t kMaxNormWidth = 32768;
struct NormArgs {
    int32_t dtype, r32, post, pre, gate_act;
    float post_eps, pre_eps, scale;
    int64_t M;
    int32_t N;
    const uint16_t* block;
    int64_t ldb;
    const uint16_t *post_w, *post_b;
    const uint16_t* gate;
    int64_t ldg;
    const void* R;
    int64_t ldr;
    const uint16_t *pre_w, *pre_b;
    void* R_out;
    int64_t ldro;
    uint16_t* Y;
    int64_t ldy;
};
hipError_t launch_residual_norm(const NormArgs& a, hipStream_t s);

}  // namespace hts
