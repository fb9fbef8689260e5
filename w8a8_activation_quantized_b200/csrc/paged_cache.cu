// paged_cache.cu -- block tables and slots from the requests' lengths, and the
// write of new keys and values into their pages.
//
// Tables.  need_b = ceil((c_b + n_b) / ps) - ceil(c_b / ps); the new entries
// of all requests, in order, are free_pages[0], free_pages[1], ...; token t of
// the packed batch belongs to the request b with cu_b <= t < cu_(b+1) and sits
// at position p = c_b + t - cu_b.  The bytes are few (a decode step of 64
// requests moves 1 KB): launches and round trips are what costs.  So one
// launch does it all: every CTA computes the two prefix sums over all requests
// itself (at most 4096, 16 per thread) instead of waiting for another CTA's,
// and takes its share of the tokens and of the new entries, finding each one's
// request by binary search in shared memory.  A token in a new page takes the
// page number from free_pages, not from the table, so no CTA reads an entry
// that another one writes.  In a captured graph 3.4 us for 64 decoding requests, 4.1
// for 512 with chunks.
//
// Write.  A copy of T rows of K and of V at 16 bytes per thread; bound by its
// bytes (HBM), or by the launch for a decode step: 16000 rows of 8 heads of 128, of
// which 500 are padding (slot -1: neither read nor written), take 21.2 us (127 MB,
// 6.0 TB/s), 61 rows 2.8.
#include <algorithm>

#include "paged_common.cuh"

namespace cider {
namespace {

constexpr int kTabThreads = 256;

__device__ __forceinline__ int sat_int(int64_t v) { return static_cast<int>(min(v, static_cast<int64_t>(INT32_MAX))); }

// Lengths of request b as the call uses them, and whether they had to be cut.
struct TabLen {
    int c, n, first, need;
};
__device__ __forceinline__ TabLen tab_len(const PagedTablesArgs& a, int b, bool* bad) {
    const int c0 = __ldg(a.cached + b), n0 = __ldg(a.fresh + b);
    const int cap = a.width << a.ps_log2;  // <= 2^30
    TabLen r;
    r.c = max(c0, 0);
    r.n = max(n0, 0);
    const int64_t len = static_cast<int64_t>(r.c) + r.n;
    *bad = c0 < 0 || n0 < 0 || len > cap;
    r.first = (min(r.c, cap) + a.page_size - 1) >> a.ps_log2;
    r.need = ((static_cast<int>(min(len, static_cast<int64_t>(cap))) + a.page_size - 1) >> a.ps_log2) - r.first;
    return r;
}

__global__ void __launch_bounds__(kTabThreads) k_paged_tables(PagedTablesArgs a) {
    extern __shared__ int32_t s_tab[];
    int32_t* s_cu = s_tab;               // [B + 1] new tokens before each request
    int32_t* s_page = s_tab + a.B + 1;   // [B + 1] new pages before each request
    __shared__ int64_t s_warp[kTabThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int per = (a.B + kTabThreads - 1) / kTabThreads;
    const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    int64_t tok = 0, pages = 0;
    bool any_bad = false;
    for (int b = b0; b < b1; ++b) {
        bool bad;
        const TabLen r = tab_len(a, b, &bad);
        any_bad |= bad;
        tok += r.n;
        pages += r.need;
    }
    int64_t all_tok, all_pages;
    int64_t t0 = block_prefix<kTabThreads>(tok, s_warp, &all_tok);
    int64_t p0 = block_prefix<kTabThreads>(pages, s_warp, &all_pages);
    for (int b = b0; b < b1; ++b) {
        bool bad;
        const TabLen r = tab_len(a, b, &bad);
        s_cu[b] = sat_int(t0);
        s_page[b] = sat_int(p0);
        t0 += r.n;
        p0 += r.need;
        if (blockIdx.x == 0) {
            a.cu[b] = s_cu[b];
            a.kv_len[b] = static_cast<int>(min(static_cast<int64_t>(r.c) + r.n, static_cast<int64_t>(a.width) << a.ps_log2));
        }
    }
    if (threadIdx.x == 0) {
        s_cu[a.B] = sat_int(all_tok);
        s_page[a.B] = sat_int(all_pages);
        if (blockIdx.x == 0) {
            a.cu[a.B] = s_cu[a.B];
            a.taken[0] = s_page[a.B];
            any_bad |= all_tok > a.rows || all_pages > a.num_free;
        }
    }
    __syncthreads();
    const int stride = gridDim.x * kTabThreads, id = blockIdx.x * kTabThreads + threadIdx.x;
    // the new entries (all_pages <= B * width)
    for (int64_t x = id; x < s_page[a.B]; x += stride) {
        const int b = find_request(s_page, a.B, static_cast<int32_t>(x));
        bool bad;
        const TabLen r = tab_len(a, b, &bad);
        const int page = x < a.num_free ? __ldg(a.free_pages + x) : -1;
        const bool ok = page >= 0 && page < a.num_pages;
        any_bad |= !ok;
        a.table[b * a.ld_table + r.first + (static_cast<int>(x) - s_page[b])] = ok ? page : -1;
    }
    // the tokens' slots
    for (int64_t t = id; t < a.rows; t += stride) {
        int slot = -1;
        if (t < s_cu[a.B]) {
            const int b = find_request(s_cu, a.B, static_cast<int32_t>(t));
            bool bad;
            const TabLen r = tab_len(a, b, &bad);
            const int64_t pos = static_cast<int64_t>(r.c) + (t - s_cu[b]);
            const int64_t j = pos >> a.ps_log2;
            if (j < a.width) {
                int page;
                if (j >= r.first) {
                    const int64_t x = static_cast<int64_t>(s_page[b]) + (j - r.first);
                    page = x < a.num_free ? __ldg(a.free_pages + x) : -1;
                } else {
                    page = a.table[b * a.ld_table + j];
                }
                const bool ok = page >= 0 && page < a.num_pages;
                any_bad |= !ok;
                if (ok) slot = (page << a.ps_log2) | static_cast<int>(pos & (a.page_size - 1));
            }
        }
        a.slots[t] = slot;
    }
    if (any_bad) atomicOr(a.status, kStatusIndex);
}

constexpr int kAppThreads = 256;
constexpr int kAppUnroll = 4;  // 16-byte pieces of K, and of V, in flight per thread

__global__ void __launch_bounds__(kAppThreads) k_paged_append(PagedCache c, const uint4* __restrict__ k_new,
                                                              int64_t ld_k, const uint4* __restrict__ v_new,
                                                              int64_t ld_v, const int32_t* __restrict__ slots, int T,
                                                              unsigned* status) {
    pdl_wait();
    pdl_trigger();
    // strides in 16-byte pieces; a token's row is H_kv heads of 2^dlog pieces
    const int dlog = c.D == 128 ? 4 : 3;
    const unsigned row = static_cast<unsigned>(c.H_kv) << dlog;
    const int64_t total = static_cast<int64_t>(T) * row;
    const int64_t sp = c.sp >> 3, sh = c.sh >> 3, st = c.st >> 3;
    const int nslots = c.num_pages << c.ps_log2;
    uint4* kc = reinterpret_cast<uint4*>(c.k);
    uint4* vc = reinterpret_cast<uint4*>(c.v);
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * (kAppThreads * kAppUnroll) + threadIdx.x; base < total;
         base += static_cast<int64_t>(gridDim.x) * (kAppThreads * kAppUnroll)) {
        uint4 kv[kAppUnroll], vv[kAppUnroll];
        int64_t dst[kAppUnroll];
#pragma unroll
        for (int u = 0; u < kAppUnroll; ++u) {
            const int64_t x = base + u * kAppThreads;
            dst[u] = -1;
            if (x >= total) continue;
            const int t = static_cast<int>(x / row);
            const unsigned e = static_cast<unsigned>(x - static_cast<int64_t>(t) * row);
            const int slot = __ldg(slots + t);
            if (slot < 0 || slot >= nslots) {
                if (slot != -1 && e == 0) atomicOr(status, kStatusIndex);
                continue;
            }
            dst[u] = (slot >> c.ps_log2) * sp + (e >> dlog) * sh + (slot & (c.page_size - 1)) * st + (e & ((1u << dlog) - 1));
            kv[u] = __ldg(k_new + t * (ld_k >> 3) + e);
            vv[u] = __ldg(v_new + t * (ld_v >> 3) + e);
        }
#pragma unroll
        for (int u = 0; u < kAppUnroll; ++u) {
            if (dst[u] >= 0) {
                kc[dst[u]] = kv[u];
                vc[dst[u]] = vv[u];
            }
        }
    }
}

}  // namespace

cudaError_t launch_paged_tables(const PagedTablesArgs& a, int num_sms, cudaStream_t st) {
    // one thread per token or per possible new entry, whichever are more, up
    // to one CTA per SM
    const int64_t work = std::max<int64_t>(a.rows, std::min<int64_t>(a.num_free, static_cast<int64_t>(a.B) * a.width));
    const int grid = static_cast<int>(std::min<int64_t>(num_sms, std::max<int64_t>(1, (work + kTabThreads - 1) / kTabThreads)));
    return launch_pdl(k_paged_tables, dim3(grid), dim3(kTabThreads), (a.B + 1) * 2 * sizeof(int32_t), st, a);
}

cudaError_t launch_paged_append(const PagedCache& c, const void* k_new, int64_t ld_k, const void* v_new, int64_t ld_v,
                                const int32_t* slots, int T, int num_sms, unsigned* status, cudaStream_t st) {
    const int64_t total = static_cast<int64_t>(T) * c.H_kv * (c.D / 8);
    const int64_t ctas = (total + kAppThreads * kAppUnroll - 1) / (kAppThreads * kAppUnroll);
    const int grid = static_cast<int>(std::min<int64_t>(ctas, static_cast<int64_t>(num_sms) * 8));
    return launch_pdl(k_paged_append, dim3(grid), dim3(kAppThreads), 0, st, c, static_cast<const uint4*>(k_new), ld_k,
                      static_cast<const uint4*>(v_new), ld_v, slots, T, status);
}

}  // namespace cider
