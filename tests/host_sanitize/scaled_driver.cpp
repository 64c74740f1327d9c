// Host-only driver of the block-scaled 8-bit half of the C API under AddressSanitizer / UndefinedBehaviorSanitizer: every
// entry point with valid, extreme and random sizes.  The launchers are stand-ins that check what the host code hands to
// the kernels: 32-bit byte offsets of a tile, grids below 2^32 threads in an axis, parts inside the caller's workspace.
// "--kernels M N K gated out8 .." prints the kernel and split of each size.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>

#include "hts.h"
#include "scaled_internal.h"

static int fails = 0, bad = 0, launches = 0, sums = 0, last_kernel = -1, last_split = 0;
static uintptr_t ws_lo = 0;
static size_t ws_size = 0;
static bool want_part = false;
#define EXPECT(cond, what)                                                                            \
    do {                                                                                              \
        if (!(cond)) {                                                                                \
            ++fails;                                                                                  \
            std::fprintf(stderr, "FAIL line %d: %s [%s]\n", __LINE__, what, hts_last_error());        \
        }                                                                                             \
    } while (0)
static void complain(const char* what) {
    ++bad;
    std::fprintf(stderr, "stub check failed: %s\n", what);
}

namespace hts {
static void look(const ScaledArgs& a, int kernel, int rows_n, int rows_m, int threads) {
    ++launches;
    last_kernel = kernel;
    last_split = a.nsplit;
    const int64_t tiles = (a.N * (a.gated ? 2 : 1) + rows_n - 1) / rows_n * ((a.M + rows_m - 1) / rows_m);
    if (a.M < 1 || a.N < 1 || a.K < 16 || a.K % 16 || !a.X || !a.W[0] || !a.ws[0] || !a.Y) complain("arguments");
    if (a.gated && (!a.W[1] || !a.ws[1] || a.act < 0 || a.act > 2)) complain("gated arguments");
    if ((tiles + 1) * threads >= (int64_t(1) << 32)) complain("grid");
    if (256 * a.ldw[0] + a.K >= (int64_t(1) << 31) || 256 * a.ldx + a.K >= (int64_t(1) << 31)) complain("32-bit offsets");
    if (a.nsplit < 1 || a.nsplit > 8 || a.nsplit > scale_blocks(a.K)) complain("split");
    if (a.nsplit > 1 && !a.part) complain("split without parts");
    if ((a.part != nullptr) != want_part) complain("parts or not");
    if (a.y_dtype == HTS_FP8_E4M3 && (!a.ys || a.N % 16 || (!a.part && !writes_e4m3((ScaledKernel)kernel)))) complain("E4M3 rows");
    if (a.part) {
        const uintptr_t p = (uintptr_t)a.part;
        if (a.ldp < a.N || a.ldp % 4 || p % 16 || p < ws_lo ||
            p + 4 * (uint64_t)a.nsplit * (a.gated ? 2 : 1) * a.M * a.ldp > ws_lo + ws_size)
            complain("parts outside the workspace");
    }
}
hipError_t launch_quantize_rows(const QuantArgs& a, hipStream_t) {
    ++launches;
    if (a.M < 1 || a.K < 16 || a.K % 16 || !a.X || !a.Q || !a.S || a.lds < a.M || a.ldq < a.K || a.ldx < a.K) complain("rows");
    return hipSuccess;
}
hipError_t launch_quantize_weight(const QuantArgs& a, hipStream_t) {
    ++launches;
    if (a.M < 1 || a.K < 16 || a.K % 16 || !a.X || !a.Q || !a.S || a.lds < scale_blocks(a.K)) complain("weight");
    return hipSuccess;
}
hipError_t launch_scaled_stream(const ScaledArgs& a, hipStream_t) {
    look(a, SCALED_STREAM, a.gated ? 32 : 16, 32, 512);
    if (a.M > kScaledStreamRows) complain("streamed rows");
    return hipSuccess;
}
hipError_t launch_scaled_stream_made(const ScaledArgs& a, int32_t x_dtype, hipStream_t) {
    want_part = false;
    look(a, -2, a.gated ? 32 : 16, 32, 512);
    if (a.M > kMadeRows || a.M * scale_blocks(a.K) > kMadeBlocks || a.y_dtype == HTS_FP8_E4M3 ||
        (a.gated ? x_dtype != HTS_F16 && x_dtype != HTS_BF16 : x_dtype != HTS_F32))
        complain("rows made in place");
    return hipSuccess;
}
hipError_t launch_scaled_ring(const ScaledArgs& a, ScaledKernel k, hipStream_t) {
    look(a, k, k <= RING_32x16 || k == RING_32x32 ? 32 : k == RING_128x64 || k == RING_128x128 ? 128 : 64, 16, 512);
    return hipSuccess;
}
hipError_t launch_scaled_tile(const ScaledArgs& a, ScaledKernel k, hipStream_t) {
    look(a, k, k == TILE_128x128 ? 128 : 256, k == TILE_256x256 ? 256 : 128, 512);
    return hipSuccess;
}
hipError_t launch_scaled_sum(const ScaledArgs& a, hipStream_t) {
    ++sums;
    if (!a.part) complain("sum of no parts");
    return hipSuccess;
}
}  // namespace hts

// Addresses that nothing reads.
static const void* at(uint64_t n) { return reinterpret_cast<const void*>(uintptr_t(n << 12)); }
static void* to(uint64_t n) { return reinterpret_cast<void*>(uintptr_t(n << 12)); }

static hts_scaled_weight weight(int64_t K) { return {at(0x100), (K + 15) / 16 * 16, (const float*)at(0x200), (K + 127) / 128}; }

static hts_status product(int64_t M, int64_t N, int64_t K, bool gated, bool out8, bool space) {
    hts_scaled_weight w = weight(K);
    size_t n = 0;
    hts_status st = gated ? hts_scaled_gated_workspace(M, N, K, out8 ? HTS_FP8_E4M3 : HTS_BF16, &n) : hts_scaled_gemm_workspace(M, N, K, &n);
    if (st) return st;
    ws_lo = (uintptr_t)at(0x900);
    ws_size = n;
    want_part = n > 0 && space;
    const int64_t ld = (N + 15) / 16 * 16;
    if (gated)
        return hts_scaled_gated(1, M, N, K, at(0x300), w.ld, (const float*)at(0x400), M, &w, &w, to(0x500), ld,
                                out8 ? HTS_FP8_E4M3 : HTS_BF16, out8 ? (float*)to(0x600) : nullptr, M,
                                space ? to(0x900) : nullptr, n, nullptr);
    return hts_scaled_gemm(M, N, K, at(0x300), w.ld, (const float*)at(0x400), M, &w, to(0x500), ld, HTS_F16,
                           space ? to(0x900) : nullptr, n, nullptr);
}

int main(int argc, char** argv) {
    if (argc > 1 && !std::strcmp(argv[1], "--kernels")) {
        for (int i = 2; i + 4 < argc; i += 5) {
            EXPECT(product(atoll(argv[i]), atoll(argv[i + 1]), atoll(argv[i + 2]), atoi(argv[i + 3]), atoi(argv[i + 4]), true) == HTS_OK, "sizes");
            std::printf("%d %d\n", last_kernel, last_split);
        }
        return fails || bad;
    }
    std::mt19937_64 g(7);
    auto size = [&](double most) { return (int64_t)std::exp(std::uniform_real_distribution<double>(0.0, std::log(most))(g)); };
    for (int n = 0; n < 20000; ++n) {
        const int64_t K = 16 * size(262143.0);
        const bool gated = g() % 2, out8 = gated && g() % 2, space = out8 || g() % 2;
        int64_t M = size(6.0e7), N = size(6.0e7);
        if (out8) N = 16 * ((N + 15) / 16);
        const hts_status st = product(M, N, K, gated, out8, space);
        EXPECT(st == HTS_OK || st == HTS_ERR_UNSUPPORTED, "random sizes");
        if (st == HTS_ERR_UNSUPPORTED) EXPECT(((N + 127) / 128) * ((M + 127) / 128) >= (1 << 22), "refused for its size alone");
    }
    const int64_t edge[] = {1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 4096, (1 << 26) - 1};
    for (int64_t M : edge)
        for (int64_t N : edge)
            for (int64_t K : {16, 112, 128, 144, 4096, (1 << 22) - 16}) {
                const hts_status st = product(M, N, K, false, false, true);
                EXPECT(st == HTS_OK || (st == HTS_ERR_UNSUPPORTED && M * N > (int64_t(1) << 35)), "edge sizes");
            }
    // feed-forward parts: the workspace's pieces in order and inside, whichever way they run
    for (int n = 0; n < 3000; ++n) {
        const int64_t M = size(20000.0), hidden = 16 * size(2000.0), inner = 16 * size(2000.0);
        hts_scaled_weight w = weight(hidden), d = weight(inner);
        size_t bytes = 0;
        EXPECT(hts_scaled_mlp_workspace(M, hidden, inner, &bytes) == HTS_OK && bytes > 0, "feed-forward workspace");
        ws_lo = (uintptr_t)at(0x900);
        ws_size = bytes;
        size_t gated = 0, down = 0;
        EXPECT(hts_scaled_gated_workspace(M, inner, hidden, HTS_FP8_E4M3, &gated) == HTS_OK, "gated");
        EXPECT(hts_scaled_gemm_workspace(M, hidden, inner, &down) == HTS_OK, "down");
        // (both products' parts or neither's: the stand-ins know one answer at a time)
        if ((gated > 0) != (down > 0)) continue;
        want_part = gated > 0;
        EXPECT(hts_scaled_mlp(0, HTS_F16, M, hidden, inner, at(0x300), (hidden + 7) / 8 * 8, &w, &w, &d, to(0x500),
                              (hidden + 7) / 8 * 8, to(0x900), bytes, nullptr) == HTS_OK, "feed-forward part");
        EXPECT(hts_scaled_mlp(0, HTS_F16, M, hidden, inner, at(0x300), (hidden + 7) / 8 * 8, &w, &w, &d, to(0x500),
                              (hidden + 7) / 8 * 8, to(0x900), bytes - 1, nullptr) == HTS_ERR_WORKSPACE, "short workspace");
    }
    std::printf("launches %d, sums %d, expectations failed: %d, stub checks failed: %d\n", launches, sums, fails, bad);
    return fails || bad;
}
