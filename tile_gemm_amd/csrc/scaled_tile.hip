// Block-scaled 8-bit product for larger M: the matrix-core-bound tiled path, and its gated form.
//
//   Y[m][n] = sum_b xs[b][m] ws[n / 128][b] sum_{k in block b} X[m][k] W[n][k]
//
// A workgroup owns 64 WN rows of W and BM rows of X (the gated form: 32 WN gate rows and the same up rows), and walks K
// in its blocks of 128.  One 16x16x128 instruction makes a 16 x 16 piece of a block's sum; the piece is multiplied by
// both scales and added to its 32-bit accumulator on the vector units, while the matrix cores make the next ones.
//
// 8192 x 13824 x 5120: 497 to 526 us from card to card, 2.2 to 2.3 PFLOP/s; the library's product of the same values without
// scales takes 419 to 434, one of 8192 cubed reaches 2.86 to 3.09 PFLOP/s.  Bound by what a block's 2048 cycles of matrix instructions do not
// hide: 3700 to 3900 pass a block (256 x 256), the matrix cores are busy 55%, the vector units, which add the pieces, 48%;
// returns of LDS reads stand in the way of the matrix instructions, and the clock falls (1.7 GHz of 2.4 while counters are read).  Steps that made it
// (us): one tile shape, copies a block ahead 642; pieces added three steps behind their instruction, copies between
// the instructions 568; operands two column blocks ahead 561; outputs through LDS in whole lines 543 to 491, 3000 x 20000 x
// 1024 114 to 85 (32 bytes of a line at a time wrote 368 MB for 226).  Measured and dropped: W from memory straight into
// registers (256 x 192: 918 for 568), lines touched ahead, the order of K turned per workgroup (563 to 607 for 571).
//
// WHOLE (E4M3 and 32-bit rows): the operands become binary16 values in registers and a piece takes four 16-bit instructions, 64 cycles for
// 32.  Such an instruction leaves the vector units no room (measured: one and n vector operations behind it take 17 + 4 n
// cycles), so that a block of 256 x 128 takes its 2048 cycles of matrix instructions and, behind one another, the 1900
// of conversions and additions: 1.6 to 1.9 us (matrix cores busy 42%, vector units 55%).  2048 x 11008 x 4096 gated 360 us, 1.03
// PFLOP/s (the library's binary16 product of that size 414, one of 8192 cubed 1.54 PFLOP/s).  Measured and dropped: a block in two halves of 64 columns with the conversions spread
// evenly over its pieces, whose sums are scaled twice, 389.
#include "scaled_device.h"

namespace hts {
namespace {

// The tile of outputs of ES bytes as it lies in LDS on its way out: BM rows of BNO, their 16-byte chunks XORed with the lane
// group that writes them, so that 16 rows written at once (NBJ apart) lie in 16 different chunks.
template <int BNO, int NBJ, int ES>
__device__ __forceinline__ uint32_t image_at(int row, int byte) {
    constexpr int PITCH = BNO * ES, CHUNKS = PITCH / 16;
    return (uint32_t)(row * PITCH + (((byte >> 4) ^ (row / NBJ % 16 % CHUNKS)) << 4) + (byte & 15));
}
// From there to memory, 16 bytes a lane, a row's lanes next to one another (rows of Y are 8 bytes aligned at least).
template <int BNO, int BM, int NBJ, int ES, int THREADS>
__device__ __forceinline__ void store_image(uint8_t* Y, int64_t ldy, int64_t rows, int64_t cols) {
    typedef u32x4 u32x4_of_8 __attribute__((aligned(8)));
    constexpr int CHUNKS = BNO * ES / 16, PER = 16 / ES;
#pragma unroll
    for (int it = 0; it < BM * CHUNKS / THREADS; ++it) {
        const int id = it * THREADS + threadIdx.x, row = id / CHUNKS, c = id % CHUNKS;
        const int64_t left = cols - c * PER;
        if (row >= rows || left <= 0) continue;
        const u32x4 v = ld16(smem + image_at<BNO, NBJ, ES>(row, 16 * c));
        uint8_t* to = Y + (row * ldy + c * PER) * ES;
        if (left >= PER) {
            *reinterpret_cast<u32x4_of_8*>(to) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)                    // (E4M3 rows end with whole chunks)
                if (e < left) reinterpret_cast<uint16_t*>(to)[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
        }
    }
}

template <int WN, int WM, int BM>
struct TileShape {
    static constexpr int NW = WN * WM, BN = 64 * WN, WTM = BM / WM, NBJ = WTM / 16;
    static constexpr int WJ = BN / (8 * NW), XJ = BM / (8 * NW);      // copies of 1 KB per wave and block
    static constexpr int XOFF = BN * 128, SOFF = XOFF + BM * 128, STAGE = SOFF + BM * 4;
    static constexpr int TOTAL = 2 * STAGE;
    static constexpr int H = NBJ / 2;                     // a block's X: columns bj < H, then the others
    static constexpr int XH = XJ / 2, PC = WJ + XH, QC = 1 + XH;   // copies per wave: W, X below H; scales, X from H on
    static_assert(XJ % 2 == 0 && NBJ % 4 == 0 && BM / 64 <= NW && WTM / 16 % 2 == 0, "copies");
    static_assert(WN * BM * 4 <= STAGE, "the blocks' largest values fit");
};

// Workgroup id -> tile: each XCD (id % 8) takes a contiguous range of the order below, groups of kGroup tiles of W, W
// fastest inside a group: the 32 workgroups that an XCD runs at once share W and X in its L2.
constexpr int kGroup = 4;
__device__ __forceinline__ void block_of(int id, int NB, int MB, int& nb, int& mb) {
    const int total = NB * MB, per = total / 8;
    if (id < 8 * per) id = (id % 8) * per + id / 8;
    const int grp = id / (kGroup * MB), in = id % (kGroup * MB), first = grp * kGroup;
    const int n = NB - first < kGroup ? NB - first : kGroup;
    nb = first + in % n;
    mb = in / n;
}

template <bool GATED, bool WHOLE, int WN, int WM, int BM>
__global__ __launch_bounds__(64 * WN * WM, 2) void scaled_tile_kernel(const ScaledArgs a, int NB, int MB) {
    using T = TileShape<WN, WM, BM>;
    constexpr int NW = T::NW, NBJ = T::NBJ, BNO = GATED ? T::BN / 2 : T::BN, RW = GATED ? 32 : 64;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave % WN, wm = wave / WN;
    int nb, mb;
    block_of(blockIdx.x, NB, MB, nb, mb);
    const int64_t n0 = (int64_t)nb * BNO, m0 = (int64_t)mb * BM;
    const int KB = (int)((a.K + 127) / 128);
    const int split = blockIdx.y;
    const int kb0 = split * KB / a.nsplit, kb1 = (split + 1) * KB / a.nsplit;

    // copies: a lane takes chunk `ch` of a row; LDS chunk position = chunk ^ ((row / 2) & 7)
    const int ch = (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7);
    const int rows_n = (int)(a.N - n0 < BNO ? a.N - n0 : BNO), rows_m = (int)(a.M - m0 < BM ? a.M - m0 : BM);
    const rsrc_t xr = make_rsrc(a.X + m0 * a.ldx, (uint32_t)((rows_m - 1) * a.ldx + a.K));
    rsrc_t wr[2];
    wr[0] = make_rsrc(a.W[0] + n0 * a.ldw[0], (uint32_t)((rows_n - 1) * a.ldw[0] + a.K));
    wr[1] = GATED ? make_rsrc(a.W[1] + n0 * a.ldw[1], (uint32_t)((rows_n - 1) * a.ldw[1] + a.K)) : wr[0];
    uint32_t wvo[T::WJ], xvo[T::XJ];
    // first LDS row of X copy v: rows of the columns below H come first
    auto x_row = [&](int v) {
        const int r = 8 * (wave + NW * (v % T::XH)), half = T::WTM / 2;
        return r / half * T::WTM + r % half + (v >= T::XH ? half : 0);
    };
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
        const int t = x_row(v) + (lane >> 3);
        int m = t / T::WTM * T::WTM + NBJ * (t & 15) + t % T::WTM / 16;
        m = m < rows_m ? m : rows_m - 1;
        xvo[v] = (uint32_t)(m * a.ldx) + 16 * ch;
    }
    const int sj = wave % (BM / 64), sm = 64 * sj + lane;             // (copied by more than one wave, the same values)
    const float* xs = a.xs + m0 + (sm < rows_m ? sm : rows_m - 1);
    const int tail = (int)(a.K - (int64_t)128 * (KB - 1));            // columns of the last block

    // copy c of block kb: W, X below H (0 .. PC - 1), the scales, X from H on (PC .. PC + QC - 1).  Past the last block
    // of this part the copies stay, so that as many are in flight in every step, but read zeros from outside
    // (the scales: once more the last ones).
    auto outside = [&](int kb) { return 16 * ch >= (kb >= kb1 ? 0 : kb == KB - 1 ? tail : 128); };
    auto copy = [&](int kb, int c, bool cut) {
        const uint32_t st = (kb & 1) * T::STAGE, so = kb < kb1 ? 128u * kb : 0u;
        if (c < T::WJ) {
            const int job = wave + NW * c;
            copy16(wr[GATED ? (job >> 2) & 1 : 0], st + 1024 * job, cut ? kOutside : wvo[c], so);
        } else if (c == T::PC) {
            copy4(xs + (int64_t)(kb < kb1 ? kb : kb1 - 1) * a.ldxs, st + T::SOFF + 256 * sj);
        } else {
            const int v = c < T::PC ? c - T::WJ : c - T::PC - 1 + T::XH;
            copy16(xr, st + T::XOFF + 128 * x_row(v), cut ? kOutside : xvo[v], so);
        }
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
        // taken here: read at its first use, the wait for it would be one for every copy in flight, in every block
        asm volatile("" : "+v"(wsv[0]), "+v"(wsv[1]));
    };
    const int i = lane & 15, g = lane >> 4;
    const int c0 = 16 * (g ^ ((i >> 1) & 7)), c1 = 16 * ((4 + g) ^ ((i >> 1) & 7));
    const uint32_t abase = wn * 8192 + i * 128, bbase = T::XOFF + wm * T::WTM * 128 + i * 128;
    const uint32_t sbase = T::SOFF + 4 * (wm * T::WTM + NBJ * i);

    // One block's sums: step t = 4 bj + b makes the piece (b, bj) (WHOLE: W is converted during the first column, the next
    // column of X during each) and adds the scaled piece of step t - 3, whose matrix
    // instruction has ended by then.  B of column block bj + 2 is read during bj (one ahead, the reads came too late:
    // LDS answers after more than four matrix instructions), the next block's first two and its A during the last two.  Two
    // barriers a block say what has landed and what has been read by all: one before the first read of the columns from H
    // on, behind which the places of W and of the other columns are free, and one before the next block's first reads,
    // behind which the rest is.  So every copy is issued more than a block's time before it is needed.
    auto read_a = [&](uint32_t st, int b) { return cat8(ld16(smem + st + abase + 2048 * b + c0), ld16(smem + st + abase + 2048 * b + c1)); };
    auto read_b = [&](uint32_t st, int bj) { return cat8(ld16(smem + st + bbase + 2048 * bj + c0), ld16(smem + st + bbase + 2048 * bj + c1)); };
    auto read_s = [&](uint32_t st, int bj) { return *reinterpret_cast<const float*>(smem + st + sbase + 4 * bj); };
    u32x8 A[4], B[2];
    Halves AH[4], BH, BN;
    float sx[2];
    f32x4 p[4];
    float s0 = 0.f, s1 = 0.f;          // scales of the pieces not yet added
#pragma unroll
    for (int b = 0; b < 4; ++b) p[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto add = [&](int b, int bj, float s) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[b][bj][e] = __builtin_fmaf(p[b][e], s, acc[b][bj][e]);
    };
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int c = 0; c < T::PC + T::QC; ++c) copy(kb0 + k, c, outside(kb0 + k));
    landed_but<T::XH + T::PC + T::QC>();
    {
        const uint32_t st = (kb0 & 1) * T::STAGE;
#pragma unroll
        for (int b = 0; b < 4; ++b) A[b] = read_a(st, b);
#pragma unroll
        for (int bj = 0; bj < 2; ++bj) {
            B[bj] = read_b(st, bj);
            sx[bj] = read_s(st, bj);
        }
        if (WHOLE) BH = e4m3_halves(B[0]);
    }
    for (int kb = kb0; kb < kb1; ++kb) {
        if (((kb - kb0) & 63) == 0) load_ws(kb);
        const bool cut = outside(kb + 2);
        const uint32_t st = (kb & 1) * T::STAGE, sn = T::STAGE - st;
        const int l = (kb - kb0) & 63;
        const float w0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wsv[0]), l));
        const float w1 = GATED ? __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wsv[1]), l)) : w0;
#pragma unroll
        for (int bj = 0; bj < NBJ; ++bj) {
            if (bj == T::H - 2) landed_but<T::PC + T::QC>();      // X from H on is in; everyone has read the rest
            if (bj == NBJ - 2) landed_but<T::XH + T::PC>();       // the next block's W, first X and scales are in;
                                                                  // everyone has read this block
            const u32x8 Bn = bj + 2 < NBJ ? read_b(st, bj + 2) : read_b(sn, bj + 2 - NBJ);
            const float sn2 = bj + 2 < NBJ ? read_s(st, bj + 2) : read_s(sn, bj + 2 - NBJ);
            const float t0 = sx[0] * w0, t1 = GATED ? sx[0] * w1 : t0;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int last = bj == 0 ? NBJ - 1 : bj - 1;
                if constexpr (WHOLE) {
                    if (bj == 0) AH[b] = e4m3_halves(A[b]);
                    p[b] = mfma_block_whole(AH[b], BH);
                    if (b & 1) BN.v[b / 2] = e4m3_halves(b / 2 ? hi4(B[1]) : lo4(B[1]));
                } else {
                    p[b] = mfma_block(A[b], B[0]);
                }
                if (bj + 1 == NBJ) A[b] = read_a(sn, b);
                // the copies of block kb + 2 go between the matrix instructions, into what has been read
                constexpr int FIRST = T::H - 2, SLOTS = 4 * (NBJ - T::H);
                const int slot = 4 * (bj - FIRST) + b;
                if (slot >= 0 && slot < SLOTS)
#pragma unroll
                    for (int c = T::PC * slot / SLOTS; c < T::PC * (slot + 1) / SLOTS; ++c) copy(kb + 2, c, cut);
                if (bj + 2 == NBJ && b < T::QC) copy(kb + 2, T::PC + b, cut);
                if (b < 3) add(b + 1, last, (GATED && b + 1 >= 2) ? s1 : s0);
                else add(0, bj, t0);
                __builtin_amdgcn_sched_barrier(0);
            }
            s0 = t0;
            s1 = t1;
            B[0] = B[1];
            B[1] = Bn;
            if (WHOLE) BH = BN;
            sx[0] = sx[1];
            sx[1] = sn2;
        }
    }
#pragma unroll
    for (int b = 1; b < 4; ++b) add(b, NBJ - 1, (GATED && b >= 2) ? s1 : s0);
    __syncthreads();                   // no copy is left in flight: LDS is free

    // lane (j + 16 q) holds rows 4 q .. 4 q + 3 of block b for row NBJ j + bj of X
    const int64_t m1 = m0 + wm * T::WTM + NBJ * i;
    if (a.part) {
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
        if constexpr (WHOLE && BNO == 128) {
            if (a.y_dtype == HTS_FP8_E4M3) {
                static_assert(BM * BNO + WN * BM * 4 <= T::TOTAL, "the rows and their largest values fit");
                float* tops = reinterpret_cast<float*>(smem + BM * BNO);
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
#pragma unroll
                for (int bj = 0; bj < NBJ; ++bj) {
                    const int at = wm * T::WTM + NBJ * i + bj;
                    float top = kLeastTop;
#pragma unroll
                    for (int w = 0; w < WN; ++w) top = fmaxf(top, tops[w * BM + at]);
                    const float r = kE4m3Max / top;
                    if (wn == 0 && g == 0 && m1 + bj < a.M) a.ys[nb * a.ldys + m1 + bj] = top / kE4m3Max;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float f[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[e] = acc[b][bj][e] * r;
                        *reinterpret_cast<uint32_t*>(smem + image_at<BNO, NBJ, 1>(at, (int)(nr - n0) + 16 * b + 4 * g)) =
                            narrow4_e4m3(f);
                    }
                }
                __syncthreads();
                store_image<BNO, BM, NBJ, 1, 64 * T::NW>(static_cast<uint8_t*>(a.Y) + m0 * a.ldy + n0, a.ldy, a.M - m0, a.N - n0);
                return;
            }
        }
    }
    if (a.y_dtype != HTS_F32) {
        static_assert(BM * BNO * 2 <= T::TOTAL, "the outputs fit");
#pragma unroll
        for (int b = 0; b < (GATED ? 2 : 4); ++b)
#pragma unroll
            for (int bj = 0; bj < NBJ; ++bj)
                store_y4(smem + image_at<BNO, NBJ, 2>(wm * T::WTM + NBJ * i + bj, 2 * ((int)(nr - n0) + 16 * b + 4 * g)), 0,
                         a.y_dtype, acc[b][bj]);
        __syncthreads();
        store_image<BNO, BM, NBJ, 2, 64 * T::NW>(static_cast<uint8_t*>(a.Y) + 2 * (m0 * a.ldy + n0), a.ldy, a.M - m0, a.N - n0);
        return;
    }
#pragma unroll
    for (int b = 0; b < (GATED ? 2 : 4); ++b) {
        const int64_t n = nr + 16 * b + 4 * g;
#pragma unroll
        for (int bj = 0; bj < NBJ; ++bj)
            if (m1 + bj < a.M && n < a.N) store_upto4(a.Y, (m1 + bj) * a.ldy + n, a.N - n, a.y_dtype, acc[b][bj]);
    }
}

template <bool GATED, bool WHOLE, int WN, int WM, int BM>
hipError_t launch_shape(const ScaledArgs& a, hipStream_t s) {
    using T = TileShape<WN, WM, BM>;
    auto kern = scaled_tile_kernel<GATED, WHOLE, WN, WM, BM>;
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

template <bool WHOLE, int WN, int WM, int BM>
hipError_t launch_sums(const ScaledArgs& a, hipStream_t s) {
    return a.gated ? launch_shape<true, WHOLE, WN, WM, BM>(a, s) : launch_shape<false, WHOLE, WN, WM, BM>(a, s);
}

}  // namespace

hipError_t launch_scaled_tile(const ScaledArgs& a, ScaledKernel k, hipStream_t s) {
    if (a.y_dtype == HTS_FP8_E4M3 && !a.part && !writes_e4m3(k)) return hipErrorInvalidValue;
    const bool whole = whole_sums(a.y_dtype);
    if (k == TILE_256x256) return whole ? hipErrorInvalidValue : launch_sums<false, 4, 2, 256>(a, s);
    if (k == TILE_256x128) return whole ? launch_sums<true, 4, 2, 128>(a, s) : launch_sums<false, 4, 2, 128>(a, s);
    if (k == TILE_128x128) return whole ? launch_sums<true, 2, 2, 128>(a, s) : launch_sums<false, 2, 2, 128>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace hts
