// C ABI of the block-scaled 8-bit layers: argument checks, the choice of kernel and split, launches.  Every check
// happens before anything is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_checks.h"
#include "hts.h"
#include "scaled_internal.h"

namespace {

using namespace hts::api;
using hts::scale_blocks;

constexpr int64_t kInt32 = int64_t(1) << 31;
// A tile's rows are addressed by 32-bit byte offsets: 256 rows of this stay below 2^31.
constexpr int64_t kMaxLead = int64_t(1) << 22;
constexpr int64_t kMaxRows = int64_t(1) << 26, kMaxTiles = int64_t(1) << 22;

hts_status check_shape(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 1 || K < 1)
        return fail(HTS_ERR_SHAPE, "M=%lld N=%lld K=%lld (M >= 0, N and K positive)", (long long)M,
                    (long long)N, (long long)K);
    if (K % 16) return fail(HTS_ERR_SHAPE, "K=%lld is not a multiple of 16", (long long)K);
    if (K >= kMaxLead) return fail(HTS_ERR_UNSUPPORTED, "K=%lld is not below 2^22", (long long)K);
    // a launch takes fewer than 2^32 threads in an axis
    if (N >= kMaxRows || M >= kMaxRows || ((N + 127) / 128) * ((M + 127) / 128) >= kMaxTiles)
        return fail(HTS_ERR_UNSUPPORTED, "M=%lld N=%lld: below 2^26 each, ceil(M / 128) * ceil(N / 128) below 2^22", (long long)M, (long long)N);
    return HTS_OK;
}

hts_status check_lead(int64_t ld, int64_t least, int mult, const char* name) {
    hts_status st = check_ld(ld, least, mult, name);
    if (st) return st;
    if (ld >= kMaxLead) return fail(HTS_ERR_UNSUPPORTED, "%s=%lld is not below 2^22", name, (long long)ld);
    return HTS_OK;
}

hts_status check_scale(const float* p, int64_t ld, int64_t least, const char* name) {
    if (!p) return fail(HTS_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(HTS_ERR_ALIGN, "%s is not 4-byte aligned", name);
    if (ld < least || ld >= kInt32)
        return fail(HTS_ERR_SHAPE, "the leading dimension %lld of %s is not from %lld to 2^31 - 1", (long long)ld, name,
                    (long long)least);
    return HTS_OK;
}

uint64_t scale_bytes(int64_t rows, int64_t cols, int64_t ld) { return block_bytes(rows, cols, ld, 4); }

hts_status check_rows(const void* X, int64_t ldx, const float* xs, int64_t ldxs, int64_t M, int64_t K, const char* name,
                      const char* scale_name) {
    hts_status st;
    if ((st = check_ptr(X, name)) || (st = check_lead(ldx, K, 16, "ldx")) || (st = check_scale(xs, ldxs, M, scale_name)))
        return st;
    if (debug_mode() && ((st = debug_range(X, block_bytes(M, K, ldx, 1), name)) ||
                         (st = debug_range(xs, scale_bytes(scale_blocks(K), M, ldxs), scale_name))))
        return st;
    return HTS_OK;
}

hts_status check_weight(const hts_scaled_weight* w, int64_t N, int64_t K, const char* name) {
    if (!w) return fail(HTS_ERR_INVALID_ARG, "%s is NULL", name);
    hts_status st;
    if ((st = check_ptr(w->values, name)) || (st = check_lead(w->ld, K, 16, name)) ||
        (st = check_scale(w->scale, w->ld_scale, scale_blocks(K), name)))
        return st;
    if (debug_mode() && ((st = debug_range(w->values, block_bytes(N, K, w->ld, 1), name)) ||
                         (st = debug_range(w->scale, scale_bytes(scale_blocks(N), scale_blocks(K), w->ld_scale), name))))
        return st;
    return HTS_OK;
}

hts_status check_act(int32_t act) {
    if (act < HTS_ACT_SILU || act > HTS_ACT_GELU_TANH) return fail(HTS_ERR_INVALID_ARG, "act=%d is not an activation", act);
    return HTS_OK;
}

bool is_out(int32_t dt) { return dt == HTS_F32 || is16bit(dt); }
int out_bytes(int32_t dt) { return dt == HTS_F32 ? 4 : dt == HTS_FP8_E4M3 ? 1 : 2; }

// How a product runs: which kernel, over how many parts of K, with what workspace.
struct Plan {
    hts::ScaledKernel kernel;
    int32_t nsplit;
    int64_t ldp;
    uint64_t bytes;        // of the parts
    bool need;             // no run without them
};

// The kernel and split with the least estimated time.  A kernel's step (`blocks` of K on rows_n x rows_m) takes `step` us
// with one workgroup on each of some CUs, and no less than its weights take from memory; workgroups beyond a CU's each (two:
// TILE_128x128) wait for another round, and a round costs its start and end.  The steps are fitted to every kernel and
// split timed at 49 sizes of 16-bit outputs and 60 of whole sums, the weights from memory; over them the choice takes 1.03
// and 1.01 of the best one's time (geometric means).  Both sides of the choices that users meet most (us):
//   1 x 11008 x 4096 gated          ring 128x64 19.4, stream 20.6      8 rows          ring 128x64 19.2, stream 21.9
//   32 x 11008 x 4096 gated         ring 128x64 20.9, 64x32 25.8       16 x 11008 x 4096   ring 64x16 11.8, 64x32 12.1
//   48 x 13824 x 5120 gated         ring 128x64 32.6, 128x128 35.7     100 rows        ring 128x128 40.4, tile 128x128 44.7
//   64 x 11008 x 4096               ring 64x64 17.6, 128x64 in two 20.3    32 x 4096 x 11008   ring 32x16 16.0, 64x32 in four 15.9
//   128 x 11008 x 4096              ring 128x64 21.4, tile 128x128 in two 23.8
//   256 x 11008 x 4096              tile 128x128 26.4, ring 128x128 28.4
//   333 x 5504 x 4144 gated         tile 256x128 54.0, 128x128 45.4 (the farthest off)     512 x 11008 x 4096 gated  256x256 65.1, 128x128 67.9
//   2048 x 4096 x 11008             tile 256x128 96.0, 128x128 102, 256x256 128
//   8192 x 13824 x 5120             tile 256x256 519, 128x128 602, 256x128 612
// Whole sums (`whole` us a step), gated to E4M3 rows, the second launch of those that leave parts included:
//   1 x 11008 x 4096                stream 24.4, ring 64x16 25.4       1 x 13824 x 5120    ring 64x16 30.8, stream 35.5
//   64 x 11008 x 4096               ring 128x64 31.0, in two 37.7      100 rows        tile 128x128 in two 44.6, ring 128x128 49.7
//   200 x 11008 x 4096              tile 256x128 61.6, 128x128 in two 66.4     512 rows    128x128 111, 256x128 121
//   2048 x 11008 x 4096             tile 256x128 363, 128x128 380
struct Shape {
    int rows_n, rows_m, blocks;
    float step, whole;
};
constexpr Shape kShapes[hts::SCALED_KERNELS] = {
    {16, 32, 8, 0.0f, 0.0f},          // SCALED_STREAM (its own estimate)
    {32, 16, 8, 0.55f, 0.68f},        // RING_32x16
    {64, 16, 2, 0.22f, 0.38f},        // RING_64x16
    {32, 32, 4, 0.42f, 0.53f},        // RING_32x32
    {64, 32, 2, 0.31f, 0.50f},        // RING_64x32
    {64, 64, 2, 0.58f, 0.78f},        // RING_64x64
    {128, 64, 2, 0.92f, 1.22f},       // RING_128x64
    {128, 128, 1, 0.68f, 1.00f},      // RING_128x128
    {128, 128, 1, 0.60f, 1.02f},      // TILE_128x128
    {256, 128, 1, 0.75f, 1.60f},      // TILE_256x128
    {256, 256, 1, 1.05f, 0.0f},       // TILE_256x256 (no whole sums)
};

float estimate(hts::ScaledKernel k, int64_t M, int64_t N, int64_t KB, int weights, int split, bool whole) {
    if (k == hts::SCALED_STREAM)
        return 4.0f + std::max(weights * (float)N * KB * 128 / (whole ? 5.1e6f : 5.5e6f) * (1.0f + M / (whole ? 60.0f : 40.0f)),
                               0.35f * (weights + (M + 15) / 16) * ((KB + 7) / 8));     // a wave's loads, one block at a time
    const Shape& s = kShapes[k];
    const int64_t mb = (M + s.rows_m - 1) / s.rows_m;
    const int64_t tiles = (N * weights + s.rows_n - 1) / s.rows_n * mb * split;
    const int64_t steps = ((KB + split - 1) / split + s.blocks - 1) / s.blocks;
    const int at_once = k == hts::TILE_128x128 ? 512 : 256;
    float us = 1.0f;
    const int64_t full = tiles / at_once;
    for (int last = 0; last < 2; ++last) {
        const int64_t busy = last ? tiles % at_once : at_once, rounds = last ? (busy ? 1 : 0) : full;
        if (!rounds) continue;
        float step = whole ? s.whole : s.step;
        if (k == hts::TILE_128x128 && busy > 256) step = whole ? 1.8f : 1.2f;             // two on a CU
        if (k >= hts::TILE_256x128) step += (k == hts::TILE_256x256 ? 0.85f : 0.3f) * busy / 256;   // what clock and L2 leave
        if (k == hts::RING_128x128) step += 0.17f * busy / 256;
        // the tiles' two stages hold fewer bytes in flight, and so do three where whole sums make a step longer
        const float bytes_per_us = k >= hts::TILE_128x128 ? 4.0e6f : whole && k == hts::RING_128x64 ? 5.2e6f : 6.5e6f;
        const float wait = (float)busy / std::min(mb, busy) * s.rows_n * s.blocks * 128 / bytes_per_us;
        us += rounds * ((k < hts::RING_128x128 ? 4.5f : k < hts::TILE_128x128 ? 6.0f : 7.0f) + steps * std::max(step, wait));
    }
    return us;
}

// most: bytes that the parts may take.
Plan plan_of(int64_t M, int64_t N, int64_t K, bool gated, int32_t y_dtype, uint64_t most = ~uint64_t(0)) {
    const bool out8 = y_dtype == HTS_FP8_E4M3, whole = hts::whole_sums(y_dtype);
    Plan p{};
    p.ldp = (N + 3) / 4 * 4;
    const int64_t KB = scale_blocks(K);
    const int weights = gated ? 2 : 1;
    const float plane = (float)weights * M * p.ldp * 4 / 4.0e6f;           // a part written and read, us
    float best = 0.0f;
    for (int i = 0; i < hts::SCALED_KERNELS; ++i) {
        const auto k = (hts::ScaledKernel)i;
        if ((k == hts::SCALED_STREAM && M > hts::kScaledStreamRows) || (k == hts::TILE_256x256 && whole)) continue;
        for (int split = 1; split <= 8; split *= 2) {
            if (split > KB || (split > 1 && k == hts::SCALED_STREAM)) break;
            const bool parts = split > 1 || (out8 && !hts::writes_e4m3(k));
            const uint64_t bytes = parts ? (uint64_t)split * weights * M * p.ldp * 4 : 0;
            if (bytes > most) break;
            const float us = estimate(k, M, N, KB, weights, split, whole) + (parts ? 3.0f + split * plane : 0.0f);
            if (!p.nsplit || us < best) {
                best = us;
                p.kernel = k;
                p.nsplit = split;
                p.need = out8 && !hts::writes_e4m3(k);
                p.bytes = bytes;
            }
        }
    }
    return p;
}

hts_status run(hts::ScaledArgs& a, const Plan& p, void* workspace, size_t workspace_bytes, hipStream_t s) {
    if (p.bytes && workspace && workspace_bytes >= p.bytes) {
        a.part = static_cast<float*>(workspace);
        a.ldp = p.ldp;
        a.nsplit = p.nsplit;
    } else {
        a.nsplit = 1;
    }
    hipError_t e = p.kernel == hts::SCALED_STREAM     ? hts::launch_scaled_stream(a, s)
                   : p.kernel <= hts::RING_128x128 ? hts::launch_scaled_ring(a, p.kernel, s)
                                                  : hts::launch_scaled_tile(a, p.kernel, s);
    if (e == hipSuccess && a.part) e = hts::launch_scaled_sum(a, s);
    return hip_status(e, "scaled product kernel launch");
}

void set_rows(hts::ScaledArgs& a, const void* X, int64_t ldx, const float* xs, int64_t ldxs) {
    a.X = static_cast<const uint8_t*>(X);
    a.ldx = ldx;
    a.xs = xs;
    a.ldxs = ldxs;
}
void set_weight(hts::ScaledArgs& a, int i, const hts_scaled_weight& w) {
    a.W[i] = static_cast<const uint8_t*>(w.values);
    a.ldw[i] = w.ld;
    a.ws[i] = w.scale;
    a.ldws[i] = w.ld_scale;
}

hts_status quantize(int32_t dtype, int64_t M, int64_t K, const void* X, int64_t ldx, void* Q, int64_t ldq, float* scale,
                    int64_t lds, bool weight, void* stream) {
    if (!is_out(dtype)) return fail(HTS_ERR_DTYPE, "dtype %d is not HTS_F16, HTS_BF16 or HTS_F32", dtype);
    hts_status st = check_shape(M, 1, K);
    if (st) return st;
    if (M == 0) return ok();
    const int64_t KB = scale_blocks(K), rows = weight ? scale_blocks(M) : KB, cols = weight ? KB : M;
    if ((st = check_ptr(X, weight ? "W" : "X")) || (st = check_ld(ldx, K, 8, weight ? "ldw" : "ldx")) ||
        (st = check_ptr(Q, "Q")) || (st = check_ld(ldq, K, 16, "ldq")) || (st = check_scale(scale, lds, cols, "scale")))
        return st;
    if (debug_mode() && ((st = debug_range(X, block_bytes(M, K, ldx, out_bytes(dtype)), weight ? "W" : "X")) ||
                         (st = debug_range(Q, block_bytes(M, K, ldq, 1), "Q")) ||
                         (st = debug_range(scale, scale_bytes(rows, cols, lds), "scale"))))
        return st;
    const hts::QuantArgs a{dtype, M, K, X, ldx, static_cast<uint8_t*>(Q), ldq, scale, lds};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return hip_status(weight ? hts::launch_quantize_weight(a, s) : hts::launch_quantize_rows(a, s), "quantizer kernel launch");
}

uint64_t round256(uint64_t n) { return (n + 255) & ~uint64_t(255); }

// The workspace of a feed-forward part: the quantised rows and inner rows, then what the products take.
struct MlpPlan {
    bool made;             // two launches: each quantises its own input (then `parts` holds the 32-bit inner rows)
    Plan gated, down;
    int64_t lds;
    uint64_t xs, hq, hs, parts, bytes;       // offsets; the rows of X come first
};
MlpPlan mlp_plan(int64_t M, int64_t hidden, int64_t inner) {
    MlpPlan p{};
    p.gated = plan_of(M, inner, hidden, true, HTS_FP8_E4M3);
    p.down = plan_of(M, hidden, inner, false, HTS_BF16);
    p.lds = (M + 3) / 4 * 4;
    p.xs = round256((uint64_t)M * hidden);
    p.hq = p.xs + round256(4 * (uint64_t)p.lds * scale_blocks(hidden));
    p.hs = p.hq + round256((uint64_t)M * inner);
    p.parts = p.hs + round256(4 * (uint64_t)p.lds * scale_blocks(inner));
    p.bytes = p.parts + std::max(p.gated.bytes, p.down.bytes);
    // Two launches save the others' two or three.  Up to 4096 columns of X the first one keeps one block of loads ahead and
    // many waves, and they win by 2 to 9 us; beyond, every workgroup's making of the rows and its four blocks
    // ahead cost with every byte of weights.  us, two launches against the others (hidden x inner, rows): 4096 x 1024, 4
    // 12.8 : 15.3; 4096 x 11008, 1 34.6 : 42.1, 4 39.0 : 42.2; 4096 x 28672, 1 75.9 : 87.9; 1024 x 28672, 1 34.6 : 32.7; 5120 x
    // 2816, 4 19.9 : 26.3; 5120 x 8192, 1 35.8 : 36.1, 2 37.8 : 35.8; 5120 x 14336, 1 58.8 : 56.4; 8192 x 5632, 1 39.4 : 36.4.
    p.made = (hidden <= 4096 || 3.0 * hidden * inner * (0.022 + 0.01 * M) < 4.7e6) && M <= hts::kMadeRows &&
             M * std::max(scale_blocks(hidden), scale_blocks(inner)) <= hts::kMadeBlocks;
    if (p.made) {
        p.parts = 0;
        p.bytes = round256(4 * (uint64_t)M * inner);
    }
    return p;
}

}  // namespace

extern "C" {

hts_status hts_quantize_rows(int32_t dtype, int64_t M, int64_t K, const void* X, int64_t ldx, void* Q, int64_t ldq,
                             float* scale, int64_t lds, void* stream) {
    return quantize(dtype, M, K, X, ldx, Q, ldq, scale, lds, false, stream);
}

hts_status hts_quantize_weight(int32_t dtype, int64_t N, int64_t K, const void* W, int64_t ldw, void* Q, int64_t ldq,
                               float* scale, int64_t lds, void* stream) {
    return quantize(dtype, N, K, W, ldw, Q, ldq, scale, lds, true, stream);
}

hts_status hts_scaled_gemm(int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const float* x_scale,
                           int64_t ldxs, const hts_scaled_weight* W, void* Y, int64_t ldy, int32_t y_dtype,
                           void* workspace, size_t workspace_bytes, void* stream) {
    if (!is_out(y_dtype)) return fail(HTS_ERR_DTYPE, "y_dtype %d is not HTS_F32, HTS_F16 or HTS_BF16", y_dtype);
    hts_status st = check_shape(M, N, K);
    if (st) return st;
    if (M == 0) return ok();
    if ((st = check_rows(X, ldx, x_scale, ldxs, M, K, "X", "x_scale")) || (st = check_weight(W, N, K, "W")) ||
        (st = check_ptr(Y, "Y")) || (st = check_ld(ldy, N, 4, "ldy")))
        return st;
    if (workspace && !aligned16(workspace)) return fail(HTS_ERR_ALIGN, "workspace is not 16-byte aligned");
    if (debug_mode() && ((st = debug_range(Y, block_bytes(M, N, ldy, out_bytes(y_dtype)), "Y")) ||
                         (st = debug_range(workspace, workspace_bytes, "workspace"))))
        return st;
    hts::ScaledArgs a{};
    a.M = M;
    a.N = N;
    a.K = K;
    set_rows(a, X, ldx, x_scale, ldxs);
    set_weight(a, 0, *W);
    a.Y = Y;
    a.ldy = ldy;
    a.y_dtype = y_dtype;
    // one workspace for outputs of any type: what a 16-bit one takes
    const uint64_t most = y_dtype == HTS_F32 ? plan_of(M, N, K, false, HTS_BF16).bytes : ~uint64_t(0);
    return run(a, plan_of(M, N, K, false, y_dtype, most), workspace, workspace_bytes, static_cast<hipStream_t>(stream));
}

hts_status hts_scaled_gemm_workspace(int64_t M, int64_t N, int64_t K, size_t* bytes) {
    hts_status st = check_shape(M, N, K);
    if (st) return st;
    if (!bytes) return fail(HTS_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = (size_t)plan_of(M, N, K, false, HTS_BF16).bytes;
    return ok();
}

hts_status hts_scaled_gated(int32_t act, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
                            const float* x_scale, int64_t ldxs, const hts_scaled_weight* gate,
                            const hts_scaled_weight* up, void* H, int64_t ldh, int32_t h_dtype, float* h_scale,
                            int64_t ldhs, void* workspace, size_t workspace_bytes, void* stream) {
    const bool out8 = h_dtype == HTS_FP8_E4M3;
    if (!is_out(h_dtype) && !out8)
        return fail(HTS_ERR_DTYPE, "h_dtype %d is not HTS_F32, HTS_F16, HTS_BF16 or HTS_FP8_E4M3", h_dtype);
    hts_status st;
    if ((st = check_act(act)) || (st = check_shape(M, N, K))) return st;
    if (out8 && N % 16) return fail(HTS_ERR_SHAPE, "N=%lld is not a multiple of 16 (E4M3 rows)", (long long)N);
    if (M == 0) return ok();
    if ((st = check_rows(X, ldx, x_scale, ldxs, M, K, "X", "x_scale")) || (st = check_weight(gate, N, K, "gate")) ||
        (st = check_weight(up, N, K, "up")) || (st = check_ptr(H, "H")) || (st = check_ld(ldh, N, out8 ? 16 : 4, "ldh")))
        return st;
    if (out8 && (st = check_scale(h_scale, ldhs, M, "h_scale"))) return st;
    if (!out8 && h_scale) return fail(HTS_ERR_INVALID_ARG, "h_scale belongs to an E4M3 output");
    if (workspace && !aligned16(workspace)) return fail(HTS_ERR_ALIGN, "workspace is not 16-byte aligned");
    const Plan p = plan_of(M, N, K, true, h_dtype);
    if (p.need && (!workspace || workspace_bytes < p.bytes))
        return fail(HTS_ERR_WORKSPACE, "workspace of %zu bytes, hts_scaled_gated_workspace asks for %llu",
                    workspace ? workspace_bytes : (size_t)0, (unsigned long long)p.bytes);
    if (debug_mode() && ((st = debug_range(H, block_bytes(M, N, ldh, out_bytes(h_dtype)), "H")) ||
                         (out8 && (st = debug_range(h_scale, scale_bytes(scale_blocks(N), M, ldhs), "h_scale"))) ||
                         (st = debug_range(workspace, workspace_bytes, "workspace"))))
        return st;
    hts::ScaledArgs a{};
    a.M = M;
    a.N = N;
    a.K = K;
    set_rows(a, X, ldx, x_scale, ldxs);
    set_weight(a, 0, *gate);
    set_weight(a, 1, *up);
    a.act = act;
    a.gated = 1;
    a.Y = H;
    a.ldy = ldh;
    a.y_dtype = h_dtype;
    a.ys = h_scale;
    a.ldys = ldhs;
    return run(a, p, workspace, workspace_bytes, static_cast<hipStream_t>(stream));
}

hts_status hts_scaled_gated_workspace(int64_t M, int64_t N, int64_t K, int32_t h_dtype, size_t* bytes) {
    if (!is_out(h_dtype) && h_dtype != HTS_FP8_E4M3)
        return fail(HTS_ERR_DTYPE, "h_dtype %d is not HTS_F32, HTS_F16, HTS_BF16 or HTS_FP8_E4M3", h_dtype);
    hts_status st = check_shape(M, N, K);
    if (st) return st;
    if (!bytes) return fail(HTS_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = (size_t)plan_of(M, N, K, true, h_dtype).bytes;
    return ok();
}

hts_status hts_scaled_mlp(int32_t act, int32_t dtype, int64_t M, int64_t hidden, int64_t inner, const void* X,
                          int64_t ldx, const hts_scaled_weight* gate, const hts_scaled_weight* up,
                          const hts_scaled_weight* down, void* Y, int64_t ldy, void* workspace,
                          size_t workspace_bytes, void* stream) {
    if (!is16bit(dtype)) return fail(HTS_ERR_DTYPE, "dtype %d is not HTS_F16 or HTS_BF16", dtype);
    hts_status st;
    if ((st = check_act(act)) || (st = check_shape(M, inner, hidden)) || (st = check_shape(M, hidden, inner))) return st;
    if (M == 0) return ok();
    if ((st = check_ptr(X, "X")) || (st = check_ld(ldx, hidden, 8, "ldx")) || (st = check_ptr(Y, "Y")) ||
        (st = check_ld(ldy, hidden, 8, "ldy")) || (st = check_weight(gate, inner, hidden, "gate")) ||
        (st = check_weight(up, inner, hidden, "up")) || (st = check_weight(down, hidden, inner, "down")) ||
        (st = check_ptr(workspace, "workspace")))
        return st;
    if (X == Y && ldx != ldy) return fail(HTS_ERR_INVALID_ARG, "in place over X: another leading dimension");
    const MlpPlan p = mlp_plan(M, hidden, inner);
    if (workspace_bytes < p.bytes)
        return fail(HTS_ERR_WORKSPACE, "workspace of %zu bytes, hts_scaled_mlp_workspace asks for %llu", workspace_bytes,
                    (unsigned long long)p.bytes);
    if (debug_mode() && ((st = debug_range(X, block_bytes(M, hidden, ldx, 2), "X")) ||
                         (st = debug_range(Y, block_bytes(M, hidden, ldy, 2), "Y")) ||
                         (st = debug_range(workspace, workspace_bytes, "workspace"))))
        return st;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    float *xs = reinterpret_cast<float*>(w + p.xs), *hs = reinterpret_cast<float*>(w + p.hs);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hts::ScaledArgs a{};
    a.M = M;
    a.N = inner;
    a.K = hidden;
    set_weight(a, 0, *gate);
    set_weight(a, 1, *up);
    a.act = act;
    a.gated = 1;
    a.nsplit = 1;
    hts::ScaledArgs d{};
    d.M = M;
    d.N = hidden;
    d.K = inner;
    set_weight(d, 0, *down);
    d.Y = Y;
    d.ldy = ldy;
    d.y_dtype = dtype;
    d.nsplit = 1;
    if (p.made) {
        set_rows(a, X, ldx, nullptr, 0);
        a.Y = w;
        a.ldy = inner;
        a.y_dtype = HTS_F32;
        if ((st = hip_status(hts::launch_scaled_stream_made(a, dtype, s), "scaled product kernel launch"))) return st;
        set_rows(d, w, inner, nullptr, 0);
        return hip_status(hts::launch_scaled_stream_made(d, HTS_F32, s), "scaled product kernel launch");
    }
    const hts::QuantArgs q{dtype, M, hidden, X, ldx, w, hidden, xs, p.lds};
    if ((st = hip_status(hts::launch_quantize_rows(q, s), "quantizer kernel launch"))) return st;
    set_rows(a, w, hidden, xs, p.lds);
    a.Y = w + p.hq;
    a.ldy = inner;
    a.y_dtype = HTS_FP8_E4M3;
    a.ys = hs;
    a.ldys = p.lds;
    if ((st = run(a, p.gated, w + p.parts, p.gated.bytes, s))) return st;
    set_rows(d, w + p.hq, inner, hs, p.lds);
    return run(d, p.down, w + p.parts, p.down.bytes, s);
}

hts_status hts_scaled_mlp_workspace(int64_t M, int64_t hidden, int64_t inner, size_t* bytes) {
    hts_status st;
    if ((st = check_shape(M, inner, hidden)) || (st = check_shape(M, hidden, inner))) return st;
    if (!bytes) return fail(HTS_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = (size_t)mlp_plan(M, hidden, inner).bytes;
    return ok();
}

}  // extern "C"
