// Block-scaled 8-bit product for larger M: the matrix-core-bound tiled path, and its gated form.
//
//   Y[m][n] = sum_b xs[b][m] ws[n / 128][b] sum_{k in block b} X[m][k] W[n][k]
//
// A workgroup owns 64 WN rows of W and BM rows of X (the gated form: 32 WN gate rows and the same up rows), and walks K
// in its blocks of 128.  One 16x16x128 instruction makes a 16 x 16 piece of a block's sum; the piece is multiplied by
// both scales and added to its 32-bit accumulator on the vector units, while the matrix cores make the next ones.
#include "scaled_device.h"

namespace hts {
namespace {

typedef __attribute__((address_space(3))) void lds_t;
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __amdgpu_buffer_rsrc_t rsrc_t;

extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ void copy16(rsrc_t r, uint32_t lds_off, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_t*)((lds_u8*)smem + lds_off), 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void copy4(const void* g, uint32_t lds_off) {
    __builtin_amdgcn_global_load_lds(g, (lds_t*)((lds_u8*)smem + lds_off), 4, 0, 0);
}
// Past every buffer's end (their bytes stay below 2^31): such a lane reads zeros.
constexpr uint32_t kOutside = 0x80000000u;

template <int WN, int WM, int BM>
struct TileShape {
    static constexpr int NW = WN * WM, BN = 64 * WN, WTM = BM / WM, NBJ = WTM / 16;
    static constexpr int WJ = BN / (8 * NW), XJ = BM / (8 * NW);      // copies of 1 KB per wave and block
    static constexpr int XOFF = BN * 128, SOFF = XOFF + BM * 128, STAGE = SOFF + BM * 4;
    static constexpr int TOTAL = 2 * STAGE;
    static_assert(BM % (8 * NW) == 0 && BM / 64 <= NW, "copies");
    static_assert(WN * BM * 4 <= STAGE, "the blocks' largest values fit");
};

template <bool GATED, int WN, int WM, int BM>
__global__ __launch_bounds__(64 * WN * WM, 2) void scaled_tile_kernel(const ScaledArgs a, int NB, int MB) {
    using T = TileShape<WN, WM, BM>;
    constexpr int NW = T::NW, NBJ = T::NBJ, BNO = GATED ? T::BN / 2 : T::BN, RW = GATED ? 32 : 64;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN, wm = wave / WN;
    const int nb = blockIdx.x % NB, mb = blockIdx.x / NB;
    const int64_t n0 = (int64_t)nb * BNO, m0 = (int64_t)mb * BM;
    const int KB = (int)((a.K + 127) / 128);
    const int split = blockIdx.y;
    const int kb0 = (int)((int64_t)split * KB / a.nsplit), kb1 = (int)((int64_t)(split + 1) * KB / a.nsplit);

    // copies: a lane takes chunk `ch` of a row; LDS chunk position = chunk ^ ((row / 2) & 7)
    const int ch = (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7);
    const int rows_n = (int)(a.N - n0 < BNO ? a.N - n0 : BNO), rows_m = (int)(a.M - m0 < BM ? a.M - m0 : BM);
    const rsrc_t xr = make_rsrc(a.X + m0 * a.ldx, (uint32_t)((rows_m - 1) * a.ldx + a.K));
    rsrc_t wr[2];
    wr[0] = make_rsrc(a.W[0] + n0 * a.ldw[0], (uint32_t)((rows_n - 1) * a.ldw[0] + a.K));
    wr[1] = GATED ? make_rsrc(a.W[1] + n0 * a.ldw[1], (uint32_t)((rows_n - 1) * a.ldw[1] + a.K)) : wr[0];
    uint32_t wvo[T::WJ], xvo[T::XJ];
#pragma unroll
    for (int v = 0; v < T::WJ; ++v) {
        const int job = wave + NW * v, r = 8 * job + (lane >> 3);     // LDS row: wave r / 64's row r % 64
        const int src = GATED ? (job >> 2) & 1 : 0;
        int n = GATED ? 32 * (r >> 6) + (r & 31) : r;
        n = n < rows_n ? n : rows_n - 1;                              // rows past N feed outputs that are not stored
        wvo[v] = (uint32_t)(n * a.ldw[src]) + 16 * ch;
    }
#pragma unroll
    for (int v = 0; v < T::XJ; ++v) {
        // column j of a wave's block bj is its row NBJ j + bj, so that a lane's scales are consecutive
        const int r = 8 * (wave + NW * v) + (lane >> 3);
        const int t = r % T::WTM;
        int m = r / T::WTM * T::WTM + NBJ * (t & 15) + (t >> 4);
        m = m < rows_m ? m : rows_m - 1;
        xvo[v] = (uint32_t)(m * a.ldx) + 16 * ch;
    }
    const int sm = 64 * wave + lane;
    const float* xs = a.xs + m0 + (sm < rows_m ? sm : rows_m - 1);
    const int tail = (int)(a.K - (int64_t)128 * (KB - 1));            // columns of the last block

    auto issue = [&](int kb) {
        const uint32_t st = (kb & 1) * T::STAGE, so = 128u * kb;
        const bool cut = kb == KB - 1 && 16 * ch >= tail;
#pragma unroll
        for (int v = 0; v < T::WJ; ++v) {
            const int job = wave + NW * v;
            copy16(wr[GATED ? (job >> 2) & 1 : 0], st + 1024 * job, cut ? kOutside : wvo[v], so);
        }
#pragma unroll
        for (int v = 0; v < T::XJ; ++v) copy16(xr, st + T::XOFF + 1024 * (wave + NW * v), cut ? kOutside : xvo[v], so);
        if (wave < BM / 64) copy4(xs + (int64_t)kb * a.ldxs, st + T::SOFF + 256 * wave);
    };

    f32x4 acc[4][NBJ];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int bj = 0; bj < NBJ; ++bj) acc[b][bj] = f32x4{0.f, 0.f, 0.f, 0.f};

    // the weights' scales of 64 blocks, one per lane
    const int64_t nr = n0 + RW * wn;
    const int64_t srow = (nr < a.N ? nr : a.N - 1) / 128;
    float wsv[2] = {0.f, 0.f};
    auto load_ws = [&](int kb) {
        const int k = kb + lane < KB ? kb + lane : KB - 1;
        wsv[0] = a.ws[0][srow * a.ldws[0] + k];
        if (GATED) wsv[1] = a.ws[1][srow * a.ldws[1] + k];
    };
    const int i = lane & 15, g = lane >> 4;
    const int c0 = 16 * (g ^ ((i >> 1) & 7)), c1 = 16 * ((4 + g) ^ ((i >> 1) & 7));
    const uint32_t abase = wn * 8192 + i * 128, bbase = T::XOFF + wm * T::WTM * 128 + i * 128;
    const uint32_t sbase = T::SOFF + 4 * (wm * T::WTM + NBJ * i);

    if (kb0 < kb1) issue(kb0);
    for (int kb = kb0; kb < kb1; ++kb) {
        if (((kb - kb0) & 63) == 0) load_ws(kb);
        __syncthreads();               // this block's copies have landed, and the other stage is free
        if (kb + 1 < kb1) issue(kb + 1);
        const uint8_t* st = smem + (kb & 1) * T::STAGE;
        const int l = (kb - kb0) & 63;
        const float w0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wsv[0]), l));
        const float w1 = GATED ? __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wsv[1]), l)) : w0;
        float sx[NBJ];
#pragma unroll
        for (int bj = 0; bj < NBJ; ++bj) sx[bj] = *reinterpret_cast<const float*>(st + sbase + 4 * bj);
        u32x8 A[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) A[b] = cat8(ld16(st + abase + 2048 * b + c0), ld16(st + abase + 2048 * b + c1));
#pragma unroll
        for (int bj = 0; bj < NBJ; ++bj) {
            const u32x8 B = cat8(ld16(st + bbase + 2048 * bj + c0), ld16(st + bbase + 2048 * bj + c1));
            const float s0 = sx[bj] * w0, s1 = GATED ? sx[bj] * w1 : s0;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const f32x4 p = mfma_block(A[b], B);
                const float s = (GATED && b >= 2) ? s1 : s0;
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[b][bj][e] = __builtin_fmaf(p[e], s, acc[b][bj][e]);
            }
        }
    }

    // lane (j + 16 q) holds rows 4 q .. 4 q + 3 of block b for row NBJ j + bj of X
    const int64_t m1 = m0 + wm * T::WTM + NBJ * i;
    if (a.nsplit > 1) {
        const int64_t plane = a.M * a.ldp;
        float* part = a.part + (int64_t)split * (GATED ? 2 : 1) * plane;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int64_t n = nr + 16 * (GATED ? b & 1 : b) + 4 * g;
            float* to = part + (GATED && b >= 2 ? plane : 0);
#pragma unroll
            for (int bj = 0; bj < NBJ; ++bj)
                if (m1 + bj < a.M && n < a.ldp) *reinterpret_cast<f32x4*>(to + (m1 + bj) * a.ldp + n) = acc[b][bj];
        }
        return;
    }
    if constexpr (GATED) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int bj = 0; bj < NBJ; ++bj)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float h = act_value(a.act, acc[b][bj][e]) * acc[b + 2][bj][e];
                    acc[b][bj][e] = nr + 16 * b + 4 * g + e < a.N ? h : 0.f;
                }
        if constexpr (BNO == 128) {
            if (a.y_dtype == HTS_FP8_E4M3) {
                __syncthreads();       // the last block's reads are done: its memory takes the largest values
                float* tops = reinterpret_cast<float*>(smem);
                float t[NBJ];
#pragma unroll
                for (int bj = 0; bj < NBJ; ++bj) {
                    t[bj] = 0.f;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) t[bj] = fmaxf(t[bj], fabsf(acc[b][bj][e]));
                    t[bj] = fmaxf(t[bj], __shfl_xor(t[bj], 16));
                    t[bj] = fmaxf(t[bj], __shfl_xor(t[bj], 32));
                    if (g == 0) tops[wn * BM + wm * T::WTM + NBJ * i + bj] = t[bj];
                }
                __syncthreads();
                uint8_t* Y = static_cast<uint8_t*>(a.Y);
#pragma unroll
                for (int bj = 0; bj < NBJ; ++bj) {
                    const int at = wm * T::WTM + NBJ * i + bj;
                    float top = kLeastTop;
#pragma unroll
                    for (int w = 0; w < WN; ++w) top = fmaxf(top, tops[w * BM + at]);
                    const float r = kE4m3Max / top;
                    if (m1 + bj >= a.M) continue;
                    if (wn == 0 && g == 0) a.ys[nb * a.ldys + m1 + bj] = top / kE4m3Max;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int64_t n = nr + 16 * b + 4 * g;
                        float f[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[e] = acc[b][bj][e] * r;
                        if (n < a.N) *reinterpret_cast<uint32_t*>(Y + (m1 + bj) * a.ldy + n) = narrow4_e4m3(f);
                    }
                }
                return;
            }
        }
    }
#pragma unroll
    for (int b = 0; b < (GATED ? 2 : 4); ++b) {
        const int64_t n = nr + 16 * b + 4 * g;
#pragma unroll
        for (int bj = 0; bj < NBJ; ++bj)
            if (m1 + bj < a.M && n < a.N) store_upto4(a.Y, (m1 + bj) * a.ldy + n, a.N - n, a.y_dtype, acc[b][bj]);
    }
}

template <bool GATED, int WN, int WM, int BM>
hipError_t launch_shape(const ScaledArgs& a, hipStream_t s) {
    using T = TileShape<WN, WM, BM>;
    auto kern = scaled_tile_kernel<GATED, WN, WM, BM>;
    static DeviceOnce lds_limit;
    hipError_t e = lds_limit.run([&] {
        return hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, T::TOTAL);
    });
    if (e != hipSuccess) return e;
    constexpr int BNO = GATED ? T::BN / 2 : T::BN;
    const int NB = (int)((a.N + BNO - 1) / BNO), MB = (int)((a.M + BM - 1) / BM);
    kern<<<dim3((unsigned)NB * MB, (unsigned)a.nsplit), dim3(64 * T::NW), T::TOTAL, s>>>(a, NB, MB);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scaled_tile(const ScaledArgs& a, ScaledTile shape, hipStream_t s) {
    if (shape == TILE_256x256) return a.gated ? launch_shape<true, 4, 2, 256>(a, s) : launch_shape<false, 4, 2, 256>(a, s);
    if (shape == TILE_256x128) return a.gated ? launch_shape<true, 4, 2, 128>(a, s) : launch_shape<false, 4, 2, 128>(a, s);
    return a.gated ? launch_shape<true, 2, 2, 128>(a, s) : launch_shape<false, 2, 2, 128>(a, s);
}

}  // namespace hts
