// Block-scaled 8-bit product for middling M: a ring of blocks in LDS keeps the weights streaming.
//
// Between a handful of rows and the matrix cores' range the weights' bytes set the pace, and what hides their latency
// is bytes in flight.  A workgroup of WN x WM waves owns 16 AB WN rows of W and 16 NB WM rows of X (the gated form: half
// of its W rows from the gate, half from up) and copies blocks of 128 columns into a ring of NST stages, NST - 1 ahead;
// one barrier a block says that the next one has landed and the last one has been read.  Each wave makes AB x NB pieces
// of 16 x 16 with one 16x16x128 instruction each, multiplies them by both scales and adds them in 32 bits.
//
// Bound by the weights' bytes as long as one row of workgroups covers X: 24 x 32001 x 4096, 131 MB, 24.4 us, 5.4 TB/s; 48 rows of
// two 13824 x 5120, 142 MB, 32.5 us, 4.4 TB/s, each byte fetched once (measured).  With more rows it is the step itself, 0.9
// us for 48 KB of copies, LDS reads and products that only partly overlap: 200 x 5000 x 5136, 26 MB, 20.4 us, the matrix cores
// busy 10%.  Rows that are no whole number of cache lines apart cost about a sixth (gated 333 x 5504: K = 4096 36.6 us, 4144 43.0).
// Measured against this form (us): two kernels back to back in place of the ring, 24 x 32001 x 4096 54.9 and 48 rows of two
// 13824 x 5120 82; operands read a step ahead, no difference.  Whole sums (WHOLE: E4M3 and 32-bit rows) make a step longer, 0.92 to 1.22
// us for 128 x 64: 64 x 11008 x 4096 gated 24.2 (16-bit rows) and 31.2, 48 x 13824 x 5120 32.8 and 40.5.
#include "scaled_device.h"

namespace hts {
namespace {

// Rows of W and X a workgroup, WK blocks of K a step (one for each group of WN x WM waves), NST steps in the ring.
template <int AB, int NB, int WN, int WM, int WK, int NST>
struct RingShape {
    static constexpr int NG = WN * WM, NW = NG * WK, BN = 16 * AB * WN, BM = 16 * NB * WM;
    static constexpr int WJ = BN / (8 * NG), XJ = BM > 8 * NG ? BM / (8 * NG) : 1;      // copies of 1 KB per wave and step
    static constexpr int C = WJ + XJ + 1;
    static constexpr int XOFF = BN * 128, SOFF = XOFF + BM * 128, BLOCK = SOFF + (BM < 64 ? 256 : BM * 4), STAGE = WK * BLOCK;
    static constexpr int SUMS = (WK - 1) * NG * AB * NB * 1024;       // the groups' sums meet here
    static constexpr int TOTAL = NST * STAGE > SUMS ? NST * STAGE : SUMS;
    static_assert(BN % (8 * NG) == 0 && (BM % (8 * NG) == 0 || 8 * NG % BM == 0) && BM <= 64 * NG, "copies");
    static_assert(NST >= 2 && (NST - 1) * C < 64 && TOTAL <= 160 * 1024 && NW <= 16, "ring");
};

template <bool GATED, bool ONCE, bool WHOLE, int AB, int NB, int WN, int WM, int WK, int NST>
__global__ __launch_bounds__(64 * WN * WM * WK) void scaled_ring_kernel(const ScaledArgs a, int NBK, int MBK) {
    using T = RingShape<AB, NB, WN, WM, WK, NST>;
    static_assert(!GATED || AB % 2 == 0, "gate and up");
    constexpr int NG = T::NG, BNO = GATED ? T::BN / 2 : T::BN, RW = GATED ? 8 * AB : 16 * AB, HB = GATED ? AB / 2 : AB;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wk = wave / NG, wg = wave % NG, wn = wg % WN, wm = wg / WN;
    // each XCD (id % 8) takes a contiguous range, the workgroups of the same rows of W next to one another: its L2 serves them
    // (us, against W's rows one after another: 128 x 13824 x 5120 26.7 to 21.9, gated 1000 x 704 x 4096 19.8 to 17.5; 512 x
    // 2048 x 2048, where all lies in the caches, 9.6 to 10.1)
    int id = blockIdx.x;
    if (MBK > 1 && id < NBK * MBK / 8 * 8) id = id % 8 * (NBK * MBK / 8) + id / 8;
    const int nb = id / MBK, mb = id % MBK;
    const int64_t n0 = (int64_t)nb * BNO, m0 = (int64_t)mb * T::BM;
    const int KB = (int)((a.K + 127) / 128);
    const int split = blockIdx.y;
    const int kb0 = split * KB / a.nsplit, kb1 = (split + 1) * KB / a.nsplit;
    // step t takes blocks kb0 + WK turned(t) .., group wk the wk-th of them: workgroups of different rows start at
    // different columns, so that rows a power of two apart are not read from the same few channels at once
    const int steps = (kb1 - kb0 + WK - 1) / WK, rot = nb * 5 % steps;
    auto block_at = [&](int t) { return kb0 + WK * (t + rot < steps ? t + rot : t + rot - steps) + wk; };

    const int rows_n = (int)(a.N - n0 < BNO ? a.N - n0 : BNO), rows_m = (int)(a.M - m0 < T::BM ? a.M - m0 : T::BM);
    const rsrc_t xr = make_rsrc(a.X + m0 * a.ldx, (uint32_t)((rows_m - 1) * a.ldx + a.K));
    rsrc_t wr[2];
    wr[0] = make_rsrc(a.W[0] + n0 * a.ldw[0], (uint32_t)((rows_n - 1) * a.ldw[0] + a.K));
    wr[1] = GATED ? make_rsrc(a.W[1] + n0 * a.ldw[1], (uint32_t)((rows_n - 1) * a.ldw[1] + a.K)) : wr[0];
    // a copy takes 8 rows of 128 bytes, a lane one chunk; chunk c of row r lies at place c ^ ((r / 2) & 7)
    uint32_t wvo[T::WJ], xvo[T::XJ];
    int wup[T::WJ], wch[T::WJ], xch[T::XJ], xjob[T::XJ];
#pragma unroll
    for (int v = 0; v < T::WJ; ++v) {
        const int job = wg + NG * v, r = 8 * job + (lane >> 3);
        const int w = r / (16 * AB), t = r % (16 * AB);               // wave w's row t: its gate rows, then its up rows
        wup[v] = GATED ? __builtin_amdgcn_readfirstlane((8 * job) % (16 * AB) / RW) : 0;
        int n = RW * w + (GATED ? t % RW : t);
        n = n < rows_n ? n : rows_n - 1;                              // rows past N feed outputs that are not stored
        wch[v] = 16 * ((lane & 7) ^ ((4 * job + (lane >> 4)) & 7));
        wvo[v] = (uint32_t)(n * a.ldw[wup[v]]) + wch[v];
    }
#pragma unroll
    for (int v = 0; v < T::XJ; ++v) {
        xjob[v] = (wg + NG * v) % (T::BM / 8);                        // (few rows: copied by more than one wave)
        int m = 8 * xjob[v] + (lane >> 3);
        m = m < rows_m ? m : rows_m - 1;
        xch[v] = 16 * ((lane & 7) ^ ((4 * xjob[v] + (lane >> 4)) & 7));
        xvo[v] = (uint32_t)(m * a.ldx) + xch[v];
    }
    const int sj = wg % ((T::BM + 63) / 64), sm = 64 * sj + lane;
    const float* xs = a.xs + m0 + (sm < rows_m ? sm : rows_m - 1);
    const int tail = (int)(a.K - (int64_t)128 * (KB - 1));            // columns of the last block

    // Past the last step, and past this part's last block, the copies stay, so that as many are in flight in every step,
    // but read zeros from outside (the scales: the last ones).
    auto copy = [&](int t, uint32_t st) __attribute__((always_inline)) {
        const int at = t < steps ? block_at(t) : kb1;
        const int cols = at >= kb1 ? 0 : at == KB - 1 ? tail : 128;
        const uint32_t so = (uint32_t)__builtin_amdgcn_readfirstlane(at < kb1 ? 128 * at : 0);
        st += wk * T::BLOCK;
#pragma unroll
        for (int v = 0; v < T::WJ; ++v)
            copy16<ONCE>(GATED ? wr[wup[v]] : wr[0], st + 1024 * (wg + NG * v), wch[v] >= cols ? kOutside : wvo[v], so);
#pragma unroll
        for (int v = 0; v < T::XJ; ++v) copy16(xr, st + T::XOFF + 1024 * xjob[v], xch[v] >= cols ? kOutside : xvo[v], so);
        copy4(xs + (int64_t)(at < kb1 ? at : kb1 - 1) * a.ldxs, st + T::SOFF + 256 * sj);
    };

    f32x4 acc[AB][NB];
#pragma unroll
    for (int b = 0; b < AB; ++b)
#pragma unroll
        for (int c = 0; c < NB; ++c) acc[b][c] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int64_t nr = n0 + RW * wn;
    const int64_t srow = (nr < a.N ? nr : a.N - 1) / 128;
    float wsv[2] = {0.f, 0.f};
    auto load_ws = [&](int t) __attribute__((always_inline)) {        // the weights' scales of 64 steps, one per lane
        int k = t + lane < steps ? block_at(t + lane) : kb1 - 1;
        k = k < kb1 ? k : kb1 - 1;
        wsv[0] = a.ws[0][srow * a.ldws[0] + k];
        if (GATED) wsv[1] = a.ws[1][srow * a.ldws[1] + k];
        // taken here: read at its first use, the wait for it would be one for every copy in flight, in every step
        asm volatile("" : "+v"(wsv[0]), "+v"(wsv[1]));
    };
    const int i = lane & 15, g = lane >> 4;
    const int c0 = 16 * (g ^ ((i >> 1) & 7)), c1 = 16 * ((4 + g) ^ ((i >> 1) & 7));
    const uint32_t abase = wk * T::BLOCK + wn * AB * 2048 + i * 128, bbase = wk * T::BLOCK + T::XOFF + wm * NB * 2048 + i * 128;
    const uint32_t sbase = wk * T::BLOCK + T::SOFF + 4 * (16 * NB * wm + i);

#pragma unroll
    for (int k = 0; k < NST - 1; ++k) copy(k, k * T::STAGE);
    load_ws(0);
    uint32_t st = 0, free = (NST - 1) * T::STAGE;
    for (int t = 0; t < steps; ++t) {
        if (t && (t & 63) == 0) load_ws(t);
        landed_but<(NST - 2) * T::C>();                               // this step is in, and the last one's place is free
        u32x8 A[AB], B[NB];
        float sx[NB];
#pragma unroll
        for (int c = 0; c < NB; ++c) sx[c] = *reinterpret_cast<const float*>(smem + st + sbase + 64 * c);
#pragma unroll
        for (int b = 0; b < AB; ++b) A[b] = cat8(ld16(smem + st + abase + 2048 * b + c0), ld16(smem + st + abase + 2048 * b + c1));
#pragma unroll
        for (int c = 0; c < NB; ++c) B[c] = cat8(ld16(smem + st + bbase + 2048 * c + c0), ld16(smem + st + bbase + 2048 * c + c1));
        __builtin_amdgcn_sched_barrier(0);                            // the reads are asked for before the copies
        copy(t + NST - 1, free);
        const float w0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wsv[0]), t & 63));
        const float w1 = GATED ? __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wsv[1]), t & 63)) : w0;
        Halves AH[AB];
        if (WHOLE)
#pragma unroll
            for (int b = 0; b < AB; ++b) AH[b] = e4m3_halves(A[b]);
#pragma unroll
        for (int c = 0; c < NB; ++c) {
            Halves BH;
            if (WHOLE) BH = e4m3_halves(B[c]);
#pragma unroll
            for (int b = 0; b < AB; ++b) {
                const f32x4 p = WHOLE ? mfma_block_whole(AH[b], BH) : mfma_block(A[b], B[c]);
                const float s = sx[c] * (GATED && b >= HB ? w1 : w0);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[b][c][e] = __builtin_fmaf(p[e], s, acc[b][c][e]);
            }
        }
        free = st;
        st = st + T::STAGE == NST * T::STAGE ? 0 : st + T::STAGE;
    }
    __syncthreads();                                                  // no copy is left in flight: LDS is free
    if constexpr (WK > 1) {                                           // the groups' sums, in order
        f32x4* sums = reinterpret_cast<f32x4*>(smem);
        if (wk > 0)
#pragma unroll
            for (int b = 0; b < AB; ++b)
#pragma unroll
                for (int c = 0; c < NB; ++c) sums[(((wk - 1) * NG + wg) * AB * NB + b * NB + c) * 64 + lane] = acc[b][c];
        __syncthreads();
        if (wk > 0) return;
#pragma unroll
        for (int k = 0; k < WK - 1; ++k)
#pragma unroll
            for (int b = 0; b < AB; ++b)
#pragma unroll
                for (int c = 0; c < NB; ++c) {
                    const f32x4 v = sums[((k * NG + wg) * AB * NB + b * NB + c) * 64 + lane];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[b][c][e] += v[e];
                }
    }

    // lane (j + 16 q) holds rows 4 q .. 4 q + 3 of block b for row j of block c of X
#pragma unroll
    for (int c = 0; c < NB; ++c) {
        const int64_t m = m0 + 16 * (NB * wm + c) + i;
        if (m >= a.M) continue;
        if (a.part) {
            const int64_t plane = a.M * a.ldp;
            float* part = a.part + (int64_t)split * (GATED ? 2 : 1) * plane + m * a.ldp;
#pragma unroll
            for (int b = 0; b < AB; ++b) {
                const int64_t n = nr + 16 * (b % HB) + 4 * g;
                if (n < a.ldp) *reinterpret_cast<f32x4*>(part + (b >= HB ? plane : 0) + n) = acc[b][c];
            }
            continue;
        }
#pragma unroll
        for (int b = 0; b < HB; ++b) {
            const int64_t n = nr + 16 * b + 4 * g;
            f32x4 y = acc[b][c];
            if constexpr (GATED)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = act_value(a.act, y[e]) * acc[b + HB][c][e];
            if (n < a.N) store_upto4(a.Y, m * a.ldy + n, a.N - n, a.y_dtype, y);
        }
    }
}

template <bool GATED, bool ONCE, bool WHOLE, int AB, int NB, int WN, int WM, int WK, int NST>
hipError_t launch_shape(const ScaledArgs& a, hipStream_t s) {
    using T = RingShape<AB, NB, WN, WM, WK, NST>;
    auto kern = scaled_ring_kernel<GATED, ONCE, WHOLE, AB, NB, WN, WM, WK, NST>;
    static DeviceOnce lds_limit;
    hipError_t e = lds_limit.run([&] {
        return hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, T::TOTAL);
    });
    if (e != hipSuccess) return e;
    constexpr int BNO = GATED ? T::BN / 2 : T::BN;
    const int NBK = (int)((a.N + BNO - 1) / BNO), MBK = (int)((a.M + T::BM - 1) / T::BM);
    kern<<<dim3((unsigned)NBK * MBK, (unsigned)a.nsplit), dim3(64 * T::NW), T::TOTAL, s>>>(a, NBK, MBK);
    return hipGetLastError();
}

// Weights of 64 MB and more, rows of whole cache lines, and one row of workgroups for all rows of X: each line is read once, and
// no other call finds it in the caches (24 x 32001 x 4096: 27.6 us, 31.0 without; 48 rows of two 13824 x 5120: 32.8 and 36.1.
// On rows of 5136, whose lines two steps share, 45.2 and 43.4; 16 x 11008 x 4096 called again and again 12.8 and 11.5).
template <bool GATED, bool WHOLE, int AB, int NB, int WN, int WM, int WK, int NST>
hipError_t launch_sums(const ScaledArgs& a, hipStream_t s) {
    // (with whole sums, weights of that size and up to 128 rows run on smaller rings or on tiles)
    if constexpr (WHOLE && NB * WM == 8) return launch_shape<GATED, false, WHOLE, AB, NB, WN, WM, WK, NST>(a, s);
    bool once = a.M <= 16 * NB * WM && a.N * a.K * (GATED ? 2 : 1) >= int64_t(64) << 20;
    for (int w = 0; w < (GATED ? 2 : 1); ++w) once = once && a.ldw[w] % 128 == 0 && reinterpret_cast<uintptr_t>(a.W[w]) % 128 == 0;
    return once ? launch_shape<GATED, true, WHOLE, AB, NB, WN, WM, WK, NST>(a, s) : launch_shape<GATED, false, WHOLE, AB, NB, WN, WM, WK, NST>(a, s);
}
template <int AB, int NB, int WN, int WM, int WK, int NST>
hipError_t launch_any(const ScaledArgs& a, hipStream_t s) {
    const bool whole = whole_sums(a.y_dtype);
    if (a.gated) return whole ? launch_sums<true, true, AB, NB, WN, WM, WK, NST>(a, s) : launch_sums<true, false, AB, NB, WN, WM, WK, NST>(a, s);
    return whole ? launch_sums<false, true, AB, NB, WN, WM, WK, NST>(a, s) : launch_sums<false, false, AB, NB, WN, WM, WK, NST>(a, s);
}

}  // namespace

hipError_t launch_scaled_ring(const ScaledArgs& a, ScaledKernel k, hipStream_t s) {
    if (a.y_dtype == HTS_FP8_E4M3 && !a.part) return hipErrorInvalidValue;
#define HTS_RING(name, AB, NB, WN, WM, WK, NST) \
    if (k == name) return launch_any<AB, NB, WN, WM, WK, NST>(a, s)
    HTS_RING(RING_32x16, 2, 1, 1, 1, 8, 3);
    HTS_RING(RING_64x16, 2, 1, 2, 1, 2, 4);
    HTS_RING(RING_32x32, 2, 2, 1, 1, 4, 4);
    HTS_RING(RING_64x32, 2, 2, 2, 1, 2, 4);
    HTS_RING(RING_64x64, 2, 4, 2, 1, 2, 4);
    HTS_RING(RING_128x64, 2, 4, 4, 1, 2, 3);
    HTS_RING(RING_128x128, 2, 4, 4, 2, 1, 4);
#undef HTS_RING
    return hipErrorInvalidValue;
}

}  // namespace hts
