// Block tables, slots and positions of one step from request lengths (hts_kv_step).
//
// With c, a the cached and added tokens of a request and P the page size, the step's tokens start
// at the prefix sum of a, and its pages are free[head + prefix sum of (ceil((c+a)/P) - ceil(c/P))
// + ...].  Both sums run over the requests, so every workgroup makes them for itself in LDS (at
// most 4096 requests: two loads and a scan, no second launch and no wait between workgroups) and
// then finds the request of each of its tokens and of each new page by binary search.  A token's
// page is read from the table if it was there before the step and from the free list if the step
// opens it, so no workgroup reads an entry that another one writes.  Bound by latency: a chain of
// one load, the scan, the search and one dependent load.
#include "serve_device.h"
#include "serve_internal.h"

namespace hts {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxInt = 0x7FFFFFFF;

// pages that hold n tokens (n cut to the table's width)
__device__ __forceinline__ int64_t pages_of(const KvStepArgs& g, int64_t n) {
    return (min(n, g.width << g.page_shift) + (1 << g.page_shift) - 1) >> g.page_shift;
}

// Last request b with first[b] <= x (first is non-decreasing, first[0] <= x).
__device__ __forceinline__ int find(const uint32_t* first, int n, uint32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// EACH: requests of a thread
template <int EACH>
__global__ __launch_bounds__(kThreads) void kv_step_kernel(KvStepArgs g) {
    extern __shared__ uint32_t sums[];
    uint32_t* first = sums;              // first token of each request (saturated at 2^31 - 1)
    uint32_t* opened = sums + g.B;       // pages opened before each request (below 2^31)
    uint32_t* held = sums + 2 * g.B;     // tokens in the cache
    __shared__ int64_t wave_a[kThreads / 64], wave_n[kThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t head = g.free_head ? max(g.free_head[0], 0) : 0;
    int c[EACH], a[EACH];                // all loads go out before the first is used
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int b = tid * EACH + i;
        c[i] = b < g.B ? max(g.cached[b], 0) : 0;
        a[i] = b < g.B ? max(g.added[b], 0) : 0;
    }
    int64_t sa = 0, sn = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        sa += a[i];
        sn += pages_of(g, (int64_t)c[i] + a[i]) - pages_of(g, c[i]);
    }
    int64_t ia = sa, in = sn;            // inclusive sums over the wave
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t ua = __shfl_up(ia, o), un = __shfl_up(in, o);
        if (lane >= o) {
            ia += ua;
            in += un;
        }
    }
    if (lane == 63) {
        wave_a[wave] = ia;
        wave_n[wave] = in;
    }
    __syncthreads();
    int64_t ea = ia - sa, en = in - sn, all_a = 0, all_n = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        if (w < wave) {
            ea += wave_a[w];
            en += wave_n[w];
        }
        all_a += wave_a[w];
        all_n += wave_n[w];
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int b = tid * EACH + i;
        if (b >= g.B) break;
        first[b] = (uint32_t)min(ea, kMaxInt);
        opened[b] = (uint32_t)en;
        held[b] = (uint32_t)c[i];
        const int64_t len = (int64_t)c[i] + a[i];
        if (blockIdx.x == 0) {
            g.lengths[b] = (int32_t)min(min(len, g.width << g.page_shift), kMaxInt);
            g.starts[b] = (int32_t)min(ea, kMaxInt);
        }
        ea += a[i];
        en += pages_of(g, len) - pages_of(g, c[i]);
    }
    if (blockIdx.x == 0 && tid == 0) {
        g.starts[g.B] = (int32_t)min(all_a, kMaxInt);
        g.head_out[0] = (int32_t)min(head + all_n, kMaxInt);
    }
    __syncthreads();

    const int64_t step = (int64_t)gridDim.x * kThreads, me = (int64_t)blockIdx.x * kThreads + tid;
    for (int64_t t = me; t < g.tokens; t += step) {
        int64_t slot = -1, pos = -1;
        if (t < all_a) {
            const int b = find(first, g.B, (uint32_t)t);
            pos = (int64_t)held[b] + (t - first[b]);
            const int64_t j = pos >> g.page_shift, have = pages_of(g, held[b]);
            if (j < g.width) {
                int64_t id = -1;
                if (j < have) {
                    id = g.table[b * g.ldt + j];
                } else {
                    const int64_t at = head + opened[b] + (j - have);
                    if (at < g.n_free) id = g.free_pages[at];
                }
                if (id >= 0) slot = (id << g.page_shift) + (pos & ((1 << g.page_shift) - 1));
            }
            pos = min(pos, kMaxInt);
        }
        g.slots[t] = slot;
        g.positions[t] = (int32_t)pos;
    }
    for (int64_t p = me; p < all_n; p += step) {
        const int b = find(opened, g.B, (uint32_t)p);
        const int64_t at = head + p;
        g.table[b * g.ldt + pages_of(g, held[b]) + (p - opened[b])] = at < g.n_free ? g.free_pages[at] : -1;
    }
}

}  // namespace

hipError_t launch_kv_step(const KvStepArgs& a, hipStream_t s) {
    const int64_t work = a.tokens > a.B ? a.tokens : a.B;
    const int64_t want = (work + 2 * kThreads - 1) / (2 * kThreads);
    const unsigned blocks = (unsigned)(want < 1 ? 1 : want > 512 ? 512 : want);
    const size_t lds = 3 * (size_t)a.B * sizeof(uint32_t);
    if (a.B <= kThreads) kv_step_kernel<1><<<dim3(blocks), dim3(kThreads), lds, s>>>(a);
    else if (a.B <= 4 * kThreads) kv_step_kernel<4><<<dim3(blocks), dim3(kThreads), lds, s>>>(a);
    else kv_step_kernel<kMaxStepRequests / kThreads><<<dim3(blocks), dim3(kThreads), lds, s>>>(a);
    return hipGetLastError();
}

}  // namespace hts
