// Device helpers of the serving kernels: 8 consecutive 16-bit values to and from floats.
#pragma once

#include "device_common.h"

namespace hts {

template <typename T> __device__ __forceinline__ void widen8(u32x4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = widen<T>(v[i] & 0xFFFFu);
        f[2 * i + 1] = widen<T>(v[i] >> 16);
    }
}

// Two floats to two 16-bit values in a word, round to nearest even (one packed conversion for bfloat16).
template <typename T> __device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    if constexpr (T::id == BF16T::id) return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
    else return __builtin_bit_cast(uint32_t, f16x2{(_Float16)lo, (_Float16)hi});
}

template <typename T> __device__ __forceinline__ u32x4 narrow8(const float* f) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = narrow2<T>(f[2 * i], f[2 * i + 1]);
    return v;
}

// A 16-byte store that does not claim a place in the caches.
__device__ __forceinline__ void stream16(void* p, u32x4 v) { __builtin_nontemporal_store(v, (u32x4*)p); }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Four floats to four E4M3 bytes, round to nearest even, magnitudes past 448 saturated, NaN kept.
__device__ __forceinline__ float e4m3_range(float x) {
    return x != x ? x : fminf(fmaxf(x, -448.0f), 448.0f);
}
__device__ __forceinline__ uint32_t narrow4_e4m3(const float* f) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_range(f[0]), e4m3_range(f[1]), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(e4m3_range(f[2]), e4m3_range(f[3]), v, true);
}

}  // namespace hts
