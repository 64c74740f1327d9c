// Host-side argument checks and error text shared by the files of the C API (defined in hts_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hts.h"

namespace hts {
namespace api {

// Record the detail of a failing call (hts_last_error) and return its status.
__attribute__((format(printf, 2, 3))) hts_status fail(hts_status s, const char* fmt, ...);
// Clear the detail; HTS_OK.
hts_status ok();
const char* last_error();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool is16bit(int32_t dt) { return dt == HTS_F16 || dt == HTS_BF16; }

// ld >= minv and a multiple of mult
hts_status check_ld(int64_t ld, int64_t minv, int mult, const char* name);
// not NULL and 16-byte aligned
hts_status check_ptr(const void* p, const char* name);
hts_status hip_status(hipError_t e, const char* what);

// HTS_DEBUG=1: range checks of device buffers before anything is enqueued.
bool debug_mode();
// Bytes of a row-major block of `rows` rows of `cols` elements of `es` bytes, leading dimension ld.
uint64_t block_bytes(int64_t rows, int64_t cols, int64_t ld, int es);
// [p, p + bytes) lies inside one device allocation (NULL and empty ranges pass).
hts_status debug_range(const void* p, uint64_t bytes, const char* name);

}  // namespace api
}  // namespace hts
