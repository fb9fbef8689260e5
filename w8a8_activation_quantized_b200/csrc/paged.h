// paged.h -- arguments and launchers of the paged-cache kernels: tables and
// writes (paged_cache.cu), attention in 16-row tiles (paged_attn.cu) and in
// tensor-core tiles (paged_attn_tc.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace cider {

constexpr int kPagedMaxRequests = 4096;  // prefix sums over the requests stay in shared memory

struct PagedCache {
    char* k;
    char* v;
    int dt;  // 0 fp16, 1 bf16
    int num_pages, page_size, ps_log2, H_kv, D;
    int64_t sp, sh, st;  // strides in elements
};

struct PagedTablesArgs {
    const int32_t* cached;
    const int32_t* fresh;
    int B;
    const int32_t* free_pages;
    int num_free, num_pages, page_size, ps_log2;
    int32_t* table;
    int64_t ld_table;
    int width;
    int32_t* cu;
    int32_t* kv_len;
    int32_t* slots;
    int rows;
    int32_t* taken;
    unsigned* status;
};

struct PagedAttnArgs {
    PagedCache c;
    const void* q;
    int64_t ld_q;
    int T, H_q, G;
    const int32_t* cu;
    const int32_t* kv_len;
    int B;
    const int32_t* table;
    int64_t ld_table;
    int width;
    int window, sinks;
    float qscale;  // scale * log2(e)
    void* out;
    int64_t ld_out;
    float* part;  // workspace
    unsigned* status;
    int grid;  // CTAs of the split kernel, which is also how the merge finds its work
    int d_tok, d_head;  // which dimension of the cache's tensor maps (1 .. 3) is the token, the head; the page is the third
};

cudaError_t launch_paged_tables(const PagedTablesArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_paged_append(const PagedCache& c, const void* k_new, int64_t ld_k, const void* v_new, int64_t ld_v,
                                const int32_t* slots, int T, int num_sms, unsigned* status, cudaStream_t st);

// 16-row tiles: workspace, and the two launches (split kernel, merge).
size_t paged_rows16_bytes(int D, int num_sms);
cudaError_t launch_paged_rows16(PagedAttnArgs a, int num_sms, cudaStream_t st);

// Tensor-core tiles: whether they take a group of G heads per KV head, their
// workspace, and the launches (work list, tiles, join).
bool paged_tc_applies(int G);
size_t paged_tc_bytes(int64_t T, int64_t B, int G, int D, int num_sms);
cudaError_t launch_paged_tc(const PagedAttnArgs& a, int num_sms, cudaStream_t st);

}  // namespace cider
