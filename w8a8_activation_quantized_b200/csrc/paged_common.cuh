// paged_common.cuh -- what the paged-cache kernels share on the device: a
// request's place in the batch, which keys a tile of its queries sees, and
// prefix sums over the requests.
#pragma once

#include <algorithm>

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

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// Tensor maps of K and V for boxes of 64 dims x box_keys keys of one head and
// page (128-byte swizzle).  Dimension 0 is D; the token, the head and the page
// follow by ascending stride, the first two at *d_tok and *d_head.
inline bool paged_cache_maps(const PagedCache& c, int box_keys, CUtensorMap* tmK, CUtensorMap* tmV, int* d_tok, int* d_head) {
    struct Dim {
        int64_t n, stride;
        int id;
    } dim[3] = {{c.page_size, c.st, 0}, {c.H_kv, c.sh, 1}, {c.num_pages, c.sp, 2}};
    std::stable_sort(dim, dim + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D)}, strides[3];
    cuuint32_t box[4] = {64, 1, 1, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        dims[i + 1] = dim[i].n;
        strides[i] = std::max<int64_t>(dim[i].stride, c.D) * 2;  // a dimension of one element (stride 0): any will do
        if (dim[i].id == 0) {
            *d_tok = i + 1;
            box[i + 1] = box_keys;
        }
        if (dim[i].id == 1) *d_head = i + 1;
    }
    const auto type = c.dt == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return encode_tensor_map(tmK, type, 4, c.k, dims, strides, box, ones, CU_TENSOR_MAP_SWIZZLE_128B) &&
           encode_tensor_map(tmV, type, 4, c.v, dims, strides, box, ones, CU_TENSOR_MAP_SWIZZLE_128B);
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

// a / b for a >= 0, b > 0: in 32 bits, which takes a fraction of the time, where
// both fit (nearly always: blocks of a batch).
__device__ __forceinline__ int64_t div_nonneg(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
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
