// The block-scaled products with 32-bit outputs under the same stand-ins and sanitizers as the other types.
// "--kernels M N K gated .." prints the kernel and split of each size.
#define main scaled_driver_main
#include "scaled_driver.cpp"
#undef main

static hts_status product32(int64_t M, int64_t N, int64_t K, bool gated, bool space) {
    hts_scaled_weight w = weight(K);
    size_t n = 0;
    hts_status st = gated ? hts_scaled_gated_workspace(M, N, K, HTS_F32, &n) : hts_scaled_gemm_workspace(M, N, K, &n);
    if (st) return st;
    ws_lo = (uintptr_t)at(0x900);
    ws_size = n;
    const int64_t ld = (N + 15) / 16 * 16;
    // whether a plain product takes parts is its own affair: any that it takes lie in the workspace
    for (int parts = 0; parts < 2; ++parts) {
        want_part = parts && n > 0 && space;
        const int before = bad;
        st = gated ? hts_scaled_gated(1, M, N, K, at(0x300), w.ld, (const float*)at(0x400), M, &w, &w, to(0x500), ld, HTS_F32,
                                      nullptr, 0, space ? to(0x900) : nullptr, n, nullptr)
                   : hts_scaled_gemm(M, N, K, at(0x300), w.ld, (const float*)at(0x400), M, &w, to(0x500), ld, HTS_F32,
                                     space ? to(0x900) : nullptr, n, nullptr);
        if (st || bad == before) return st;
        if (!parts && n > 0 && space && bad == before + 1) bad = before;      // it took parts
    }
    return st;
}

int main(int argc, char** argv) {
    if (argc > 1 && !std::strcmp(argv[1], "--kernels")) {
        for (int i = 2; i + 3 < argc; i += 4) {
            EXPECT(product32(atoll(argv[i]), atoll(argv[i + 1]), atoll(argv[i + 2]), atoi(argv[i + 3]), true) == HTS_OK, "sizes");
            std::printf("%d %d\n", last_kernel, last_split);
        }
        return fails || bad;
    }
    std::mt19937_64 g(11);
    auto size = [&](double most) { return (int64_t)std::exp(std::uniform_real_distribution<double>(0.0, std::log(most))(g)); };
    for (int n = 0; n < 20000; ++n) {
        const int64_t K = 16 * size(262143.0), M = size(6.0e7), N = size(6.0e7);
        const hts_status st = product32(M, N, K, g() % 2, g() % 2);
        EXPECT(st == HTS_OK || st == HTS_ERR_UNSUPPORTED, "random sizes");
        EXPECT(last_kernel != hts::TILE_256x256 || st, "a tile without whole sums");
    }
    std::printf("launches %d, sums %d, expectations failed: %d, stub checks failed: %d\n", launches, sums, fails, bad);
    return fails || bad;
}
