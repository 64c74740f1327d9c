// Device pieces of the block-scaled 8-bit kernels.
#pragma once

#include <type_traits>

#include "gemm_common.h"
#include "scaled_internal.h"
#include "serve_device.h"

namespace hts {

// A block's largest magnitude a (a zero block: 2^-100, so that its scale stays a normal number) gives its scale a / 448
// and the factor 448 / a that its values are multiplied by; each is rounded once to 32 bits.
constexpr float kLeastTop = 0x1p-100f, kE4m3Max = 448.0f;

__device__ __forceinline__ float act_value(int act, float g) {
    if (act == HTS_ACT_SILU) return g / (1.0f + expf(-g));
    if (act == HTS_ACT_GELU) return 0.5f * g * (1.0f + erff(g * 0.70710678f));
    // tanh form: g * sigmoid(2 z), z = sqrt(2 / pi) (g + 0.044715 g^3)
    const float z = 1.5957691f * (g + 0.044715f * g * g * g);
    return g / (1.0f + expf(-z));
}

// 16x16x128 product of E4M3 values from zero: the block's own sum, before its scales.  Unit block scales (the form
// without scale operands).  Within each group of eight products along K the instruction keeps 13 bits below the largest
// one's power of two and drops the rest (measured); groups are added in 32 bits.
__device__ __forceinline__ f32x4 mfma_block(u32x8 a, u32x8 b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8, a), __builtin_bit_cast(i32x8, b),
                                                            f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// The same sum with every product whole: E4M3 values are binary16 values, and the 16-bit instructions drop nothing.
// 7e-8 of the result's norm in place of 1.5e-5 (K = 4096), for twice the matrix cores' time and the conversions.
__device__ __forceinline__ u32x8 e4m3_halves(u32x4 q) {
    u32x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q[i], 1.0f, false));
        r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q[i], 1.0f, true));
    }
    return r;
}
struct Halves {
    u32x8 v[2];
};
__device__ __forceinline__ Halves e4m3_halves(u32x8 q) { return {{e4m3_halves(lo4(q)), e4m3_halves(hi4(q))}}; }
__device__ __forceinline__ f32x4 mfma_block_whole(const Halves& a, const Halves& b) {
    f32x4 c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const u32x8 x = a.v[u / 2], y = b.v[u / 2];
        c[u] = mfma_dense<F16T>(u & 1 ? hi4(x) : lo4(x), u & 1 ? hi4(y) : lo4(y), u ? c[u - 1] : f32x4{0.f, 0.f, 0.f, 0.f});
        // (alive till here: its registers and the result's are the same or apart, never some of them shared, which waits)
        if (u) asm volatile("" ::"v"(c[u - 1]));
    }
    return c[3];
}

// ---- from global memory to registers and LDS ----

typedef __attribute__((address_space(3))) void lds_t;
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __amdgpu_buffer_rsrc_t rsrc_t;

extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
// Past every buffer's end (their bytes stay below 2^31): such a lane reads zeros.
constexpr uint32_t kOutside = 0x80000000u;

// 16 bytes a lane into LDS.  ONCE: what no other workgroup reads claims no place in the caches.
template <bool ONCE = false>
__device__ __forceinline__ void copy16(rsrc_t r, uint32_t lds_off, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_t*)((lds_u8*)smem + lds_off), 16, voff, soff, 0, ONCE ? 2 : 0);
}
__device__ __forceinline__ void copy4(const void* g, uint32_t lds_off) {
    __builtin_amdgcn_global_load_lds(g, (lds_t*)((lds_u8*)smem + lds_off), 4, 0, 0);
}

// All but this wave's N youngest copies have landed and its LDS reads are back; then the same of the whole workgroup.
template <int N>
__device__ __forceinline__ void landed_but() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));      // lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// ---- rows to E4M3 ----

// 16 consecutive values at column c of a row (c and K multiples of 16), as floats.
template <int DT>
__device__ __forceinline__ void load_values16(const void* row, int64_t c, float (&f)[16]) {
    if constexpr (DT == HTS_F32) {
        const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(row) + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 v = p[i];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[4 * i + e] = v[e];
        }
    } else {
        using T = typename std::conditional<DT == HTS_BF16, BF16T, F16T>::type;
        const uint16_t* p = static_cast<const uint16_t*>(row) + c;
        widen8<T>(ld16(p), f);
        widen8<T>(ld16(p + 8), f + 8);
    }
}

__device__ __forceinline__ float top16(const float (&f)[16]) {
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) t = fmaxf(t, fabsf(f[e]));
    return t;
}

__device__ __forceinline__ u32x4 scaled16(float (&f)[16], float r) {
    u32x4 q;
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] *= r;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = narrow4_e4m3(f + 4 * i);
    return q;
}

// A block's largest magnitude from its eight lanes' values, and at least kLeastTop.
__device__ __forceinline__ float block_top(const float (&f)[16]) {
    float t = top16(f);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) t = fmaxf(t, __shfl_xor(t, o));
    return fmaxf(t, kLeastTop);
}

// Up to four consecutive outputs of a row from column n on, those below N.
__device__ __forceinline__ void store_upto4(void* Y, int64_t off, int64_t left, int32_t dt, f32x4 v) {
    if (left >= 4) {
        store_y4(Y, off, dt, v);
    } else {
        for (int e = 0; e < 3; ++e)
            if (e < left) store_y1(Y, off + e, dt, v[e]);
    }
}

}  // namespace hts
