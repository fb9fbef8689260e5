// paged_common.cuh -- what the paged-cache kernels share on the device: a
// request's place in the batch, which keys a tile of its queries sees, and
// prefix sums over the requests.
#pragma once

#include "cider_device.cuh"
#include "paged.h"

namespace cider {

// Request b's rows [start, start + n) of q and its L keys, cut to what the
// call's buffers hold; query i is at position L - n + i.
struct PagedRequest {
    int start, n, L;
};

__device__ __forceinline__ PagedRequest paged_request(const PagedAttnArgs& a, int b, bool* bad) {
    const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), len = __ldg(a.kv_len + b);
    const int64_t cap = static_cast<int64_t>(a.width) << a.c.ps_log2;  // <= 2^30
    PagedRequest r;
    r.start = min(max(c0, 0), a.T);
    r.n = max(min(c1, a.T) - r.start, 0);
    r.L = static_cast<int>(min(static_cast<int64_t>(max(len, 0)), cap));
    *bad = c0 < 0 || c1 < c0 || c1 > a.T || len != r.L;
    return r;
}

// A tile of queries at positions pmin .. pmax of one request and the blocks of
// KB keys that it reads: first those that hold sinks in front of the window,
// then those from the window's lowest key to pmax.  `vb` numbers them in that
// order.
template <int KB>
struct PagedSpan {
    int pmin, pmax;
    int sink_blocks, first_block, blocks;

    __device__ __forceinline__ void set(int pmin_, int pmax_, int window, int sinks) {
        pmin = pmin_;
        pmax = pmax_;
        const int lo = window > 0 ? max(0, pmin - window + 1) : 0;  // lowest key in some query's window
        sink_blocks = window > 0 ? (min(sinks, lo) + KB - 1) / KB : 0;
        first_block = max(lo / KB, sink_blocks);
        const int end = pmax < 0 ? 0 : pmax / KB + 1;
        sink_blocks = min(sink_blocks, end);
        blocks = sink_blocks + max(0, end - first_block);
    }
    __device__ __forceinline__ int block(int vb) const { return vb < sink_blocks ? vb : vb - sink_blocks + first_block; }
};

__device__ __forceinline__ bool paged_sees(int key, int pos, int window, int sinks) {
    return key <= pos && (window <= 0 || key > pos - window || key < sinks);
}

// Exclusive prefix sum of a value per thread; `total` gets the sum.  s_warp:
// one value per warp.  Every thread calls it.
template <int NT>
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t* s_warp, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int64_t base = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) base += s_warp[w];
        sum += s_warp[w];
    }
    *total = sum;
    return base + x - v;
}

// The last b in [0, B) with pre[b] <= x, for x in [0, pre[B]) and pre
// non-decreasing from pre[0] = 0: the request that x falls in.
template <typename T>
__device__ __forceinline__ int find_request(const T* pre, int B, T x) {
    int lo = 0, hi = B;  // pre[lo] <= x < pre[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

}  // namespace cider
