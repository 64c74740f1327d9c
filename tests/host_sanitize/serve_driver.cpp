// Host-only driver of the serving half of the C API under AddressSanitizer / UndefinedBehaviorSanitizer: every
// entry point with valid, extreme and invalid arguments.  The launchers are stand-ins that check what the host
// code hands to the kernels: workspace parts inside the caller's buffer, launch parameters in their ranges.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <memory>
#include <random>
#include <vector>

#include "hts.h"
#include "serve_internal.h"

static int fails = 0, bad = 0, launches = 0;
static const char* ws_lo = nullptr;
static size_t ws_size = 0;
static bool expect_split = false;
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
hipError_t launch_kv_step(const KvStepArgs& a, hipStream_t) {
    ++launches;
    if (a.B < 0 || a.B > kMaxStepRequests || a.page_shift < 4 || a.page_shift > 10 || !a.starts || !a.head_out ||
        a.ldt < a.width || (int64_t)a.B * a.width >= (int64_t(1) << 31) || a.tokens < 0)
        complain("page step arguments");
    return hipSuccess;
}
hipError_t launch_rope(const RopeArgs& a, hipStream_t) {
    ++launches;
    if (a.T <= 0 || a.rot < 8 || a.rot > a.dim || a.dim > 256 || a.rot % 8 || a.dim % 8 || !a.turns || !a.positions)
        complain("rotary arguments");
    if ((a.q_heads && (!a.Q || !a.Qo)) || (a.k_heads && !a.K)) complain("rotary matrices");
    if (a.slots ? (!a.kc || !a.vc || !a.V || a.n_slots < 16 || a.Ko) : (a.k_heads && !a.Ko)) complain("rotary cache");
    return hipSuccess;
}
hipError_t launch_attn(const AttnArgs& a, hipStream_t) {
    ++launches;
    if (a.B <= 0 || a.head_tiles < 1 || a.tile_heads < 1 || a.tile_heads > 16 || a.q_heads % a.k_heads || a.cap < 1 ||
        a.cap > 0x7FFFFFFFu || a.window > 0x7FFFFFFFu || a.page_shift < 4 || a.token_stride >= (int64_t(1) << 26))
        complain("attention arguments");
    const int64_t rows = (int64_t)a.k_heads * a.head_tiles;
    if (rows > 65535) complain("attention grid");
    if ((a.part_o != nullptr) != expect_split) complain("split or not");
    if (a.part_o) {
        const uint64_t parts = 2 * (uint64_t)a.runs * rows * a.tile_heads;
        const char *p = (const char*)a.plan, *m = (const char*)a.part_ml, *o = (const char*)a.part_o;
        if (a.runs < 1 || (uint32_t)a.runs > a.target || p < ws_lo || p + 8 * (int64_t)a.B > m || m + 8 * parts > o ||
            o + 4 * parts * a.dim > ws_lo + ws_size)
            complain("parts outside the workspace");
        // fewer than 2^31 steps, and every run of the kernel's rule fits the grid
        const uint64_t most = a.window ? std::min<uint64_t>(a.cap, (uint64_t)a.window + 31) : a.cap;
        const uint64_t steps = (uint64_t)a.B * ((most + 31) / 32);
        if (steps >= (uint64_t(1) << 31) || a.B > kMaxSplitRequests) complain("too many steps to split");
        for (uint64_t total : {steps, steps / 2 + 1, (uint64_t)a.B, (uint64_t)1}) {
            const uint64_t even = (total + a.runs - 1) / a.runs;
            const uint64_t few = std::min<uint64_t>(std::max<uint64_t>((uint32_t)(3 * total) / a.target, 4), 16);
            const uint64_t per = std::max(even, std::min<uint64_t>(few, (total + a.B - 1) / a.B));
            if ((total + per - 1) / per > (uint64_t)a.runs) complain("more runs than workgroups");
        }
    }
    return hipSuccess;
}
hipError_t launch_residual_norm(const NormArgs& a, hipStream_t) {
    ++launches;
    if (a.M <= 0 || a.N < 8 || a.N % 8 || a.N > kMaxNormWidth || (!a.block && !a.R) || (!a.R_out && !a.Y))
        complain("norm arguments");
    return hipSuccess;
}
}  // namespace hts

alignas(256) static unsigned char fake[4096];
static void* dev(size_t off = 0) { return fake + off; }

static hts_kv_desc cache(int64_t pages, int page, int heads, int dim, int dt, bool head_order) {
    const int64_t n = (int64_t)heads * dim * page;
    return head_order ? hts_kv_desc{pages, page, heads, dim, dt, n, dim, (int64_t)page * dim}
                      : hts_kv_desc{pages, page, heads, dim, dt, n, (int64_t)heads * dim, dim};
}

static void test_attention(std::mt19937& rng) {
    const int dims[] = {8, 64, 72, 128, 200, 256}, heads[] = {1, 2, 8, 40, 1000}, groups[] = {1, 4, 16, 17, 40};
    const int64_t batches[] = {1, 2, 64, 65, 4096, 4097, 65535}, widths[] = {1, 31, 33, 1000, 1 << 20, (1u << 31) - 1};
    const int64_t windows[] = {0, 1, 4096, int64_t(1) << 40};
    for (int dim : dims)
        for (int hk : heads)
            for (int gr : groups)
                for (int64_t B : batches)
                    for (int64_t width : widths)
                        for (int64_t window : windows) {
                            const int page = 16 << (rng() % 7);
                            const hts_kv_desc kv = cache(100, page, hk, dim, HTS_BF16, rng() & 1);
                            size_t bytes = 1;
                            if ((int64_t)hk * gr > 65535) continue;
                            EXPECT(hts_paged_attn_workspace(B, hk * gr, &kv, width, window, &bytes) == HTS_OK, "workspace");
                            ws_lo = (const char*)0x100000000;   // addresses are only compared
                            ws_size = bytes;
                            const int64_t n = (int64_t)hk * gr * dim;
                            for (int fits = 0; fits < 2; ++fits) {
                                expect_split = fits && bytes > 0;
                                const hts_status st = hts_paged_attn(HTS_BF16, B, hk * gr, &kv, dev(), n, dev(), dev(), nullptr,
                                                                     nullptr, (const int32_t*)dev(), width, width, (const int32_t*)dev(),
                                                                     0.1f, window, dev(), n, nullptr, (void*)ws_lo,
                                                                     fits ? bytes : (bytes ? bytes - 1 : 0), nullptr);
                                EXPECT(st == HTS_OK, "attention");
                            }
                        }
}

static void test_cache_descriptions(std::mt19937& rng) {
    // random descriptions: a taken one has no two elements at one place (checked by marking a small cache)
    int taken = 0;
    for (int trial = 0; trial < 20000; ++trial) {
        const int pages = 1 + rng() % 3, page = 16, heads = 1 + rng() % 3, dim = 8;
        auto stride = [&] { return (int64_t)(8 * (rng() % 60)); };
        hts_kv_desc kv{pages, page, heads, dim, HTS_F16, stride(), stride(), stride()};
        size_t bytes;
        if (hts_paged_attn_workspace(1, heads, &kv, 1, 0, &bytes) != HTS_OK) continue;
        ++taken;
        std::vector<char> seen(1 << 14, 0);
        bool clash = false;
        for (int p = 0; p < pages; ++p)
            for (int t = 0; t < page; ++t)
                for (int h = 0; h < heads; ++h) {
                    const int64_t at = (pages > 1 ? p * kv.page_stride : 0) + t * kv.token_stride + (heads > 1 ? h * kv.head_stride : 0);
                    clash = clash || seen.at((size_t)at / 8);
                    seen.at((size_t)at / 8) = 1;
                }
        EXPECT(!clash, "a cache with shared places was taken");
    }
    EXPECT(taken > 100, "too few descriptions were taken");
}

static void test_rope_plans(std::mt19937& rng) {
    for (int trial = 0; trial < 3000; ++trial) {
        const int rot = 8 * (1 + rng() % 32);
        hts_rope_scaling s{rot, (int)(rng() % 5), std::exp((rng() % 2000) / 100.0 + 0.01), 1.0 + (rng() % 100) / 3.0,
                           1.0 + rng() % 100000, 0.5 + (rng() % 10), 11.0 + (rng() % 50)};
        std::unique_ptr<double[]> turns(new double[rot / 2]);   // exactly as many as the plan writes
        EXPECT(hts_rope_plan(&s, turns.get()) == HTS_OK, "plan");
        for (int i = 0; i < rot / 2; ++i) EXPECT(turns[i] > 0.0 && turns[i] <= 0.16, "turns in range");
    }
}

static void test_others() {
    int32_t* i32 = (int32_t*)dev();
    // extreme but valid sizes: no overflow in the checks
    EXPECT(hts_kv_step(4096, (int32_t*)0x100000000, (int32_t*)0x200000000, 1024, (int32_t*)0x300000000, (1ll << 31) - 1, nullptr,
                       (int32_t*)0x4000000000, (1ll << 31) - 1, (1 << 19) - 1, (1ll << 31) - 1, (int32_t*)0x500000000,
                       (int32_t*)0x600000000, (int64_t*)0x700000000000, (int32_t*)0x800000000000, (int32_t*)0x900000000,
                       nullptr) == HTS_OK, "large page step");
    EXPECT(hts_kv_step(0, nullptr, nullptr, 16, nullptr, 0, nullptr, nullptr, 1, 1, 0, nullptr, i32, nullptr, nullptr, i32 + 1,
                       nullptr) == HTS_OK, "empty page step");
    EXPECT(hts_kv_step(1, i32, i32 + 4, 16, nullptr, 0, nullptr, i32 + 8, 1, 1, 0, i32, i32 + 16, nullptr, nullptr, i32 + 20,
                       nullptr) == HTS_ERR_INVALID_ARG, "lengths over cached");
    hts_rope_desc r{HTS_F16, HTS_ROPE_HALF, 128, 128, 65535, 65535, 1.0f, 0};
    EXPECT(hts_rope(&r, (double*)dev(), (1ll << 31) - 1, i32, dev(), 1ll << 40, dev(), 1ll << 40, dev(), 1ll << 40, dev(),
                    1ll << 40, nullptr) == HTS_OK, "large rotary step");
    hts_norm_desc n{HTS_F16, HTS_F32, HTS_NORM_RMS, HTS_NORM_LAYER, 0.0f, 0.0f, 1.0f, HTS_GATE_SILU};
    EXPECT(hts_residual_norm(&n, (1ll << 31) - 1, 32768, dev(), 1ll << 40, nullptr, nullptr, dev(512), 0, dev(1024), 1ll << 40, nullptr,
                             nullptr, dev(1024), 1ll << 40, dev(256), 1ll << 40, nullptr) == HTS_OK, "large norm");
    EXPECT(hts_residual_norm(nullptr, 1, 8, dev(), 8, nullptr, nullptr, nullptr, 0, nullptr, 0, nullptr, nullptr, dev(), 8, nullptr,
                             0, nullptr) == HTS_ERR_INVALID_ARG, "no descriptor");
    // debug mode on host memory: refused, nothing launched
    setenv("HTS_DEBUG", "1", 1);
    const int before = launches;
    EXPECT(hts_residual_norm(&n, 2, 64, dev(), 64, nullptr, nullptr, nullptr, 0, dev(), 64, nullptr, nullptr, dev(256), 64, nullptr,
                             0, nullptr) == HTS_ERR_INVALID_ARG, "debug norm");
    EXPECT(std::strstr(hts_last_error(), "not device memory") != nullptr, "debug message");
    EXPECT(hts_rope(&r, (double*)dev(), 1, i32, dev(), 65535 * 128, dev(), 65535 * 128, dev(), 65535 * 128, dev(), 65535 * 128,
                    nullptr) == HTS_ERR_INVALID_ARG, "debug rotary");
    EXPECT(hts_kv_step(1, i32, i32 + 4, 16, nullptr, 0, nullptr, i32 + 8, 1, 1, 0, i32 + 12, i32 + 16, nullptr, nullptr, i32 + 20,
                       nullptr) == HTS_ERR_INVALID_ARG, "debug page step");
    EXPECT(launches == before, "nothing launched in refused debug calls");
    unsetenv("HTS_DEBUG");
}

int main() {
    std::mt19937 rng(4242);
    test_attention(rng);
    test_cache_descriptions(rng);
    test_rope_plans(rng);
    test_others();
    std::printf("expectations failed: %d, stub checks failed: %d, launches: %d\n", fails, bad, launches);
    return fails || bad;
}
