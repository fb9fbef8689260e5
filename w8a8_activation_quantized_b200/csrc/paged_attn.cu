// paged_attn.cu -- attention of new tokens over a paged key/value cache, in
// tiles of 16 rows: the kernel for decode steps, where a request brings one
// token (or a few) and the K and V bytes of the cache set the time.
//
//   out = sum_j p_j V[j] / sum_j p_j,   p_j = 2^((s_j - m) scale log2 e),
//   s_j = q . K[j] over the keys j that the query sees, m a running maximum.
//
// A tile's rows are (token, head of the KV group) pairs of one request and one
// KV head in that order, so every K and V element is read once for all the
// heads that share it.  A step of one warp is 16 keys: S = Q K^T and O += P V
// are mma.sync m16n8k16 products (fp32 accumulation) whose operands come from
// shared memory by ldmatrix, P going from one to the other in registers.  With
// 16 rows at most, 8 KB of K and V feed 32 such products, which leaves the
// tensor pipe far from its rate: HBM is the bound, and the 128-row tiles of
// tcgen05 would only add latency.
//
// Loads: each warp has its own ring of kStages steps (16 keys of K and of V) in
// shared memory, filled by TMA in boxes of 16 keys x 64 dims (128-byte swizzle,
// one mbarrier per stage), so warps never wait for one another within a tile;
// two CTAs of four warps per SM keep up to 2 x 4 x 3 x 8 KB = 192 KB in flight.
// (With 16-byte cp.async in their place the loads took half of the kernel's
// instructions: four requests of up to 32K keys 38.7 us, with TMA see below.)
// Pages that no query of the tile sees are not read.  Where only some keys of a
// step are seen by any query, the other rows of V are zeroed in shared memory:
// what the cache's unwritten slots hold may be NaN, and 0 x NaN is not 0.
//
// Split: the work of the whole batch is one line of blocks of 64 keys -- per
// request, per 16-row tile, per KV head, its blocks -- cut into equal pieces,
// one per CTA (two CTAs per SM).  No CTA has more than its share, whatever the
// requests' lengths are, and a CTA is the only one to touch a tile unless the
// cut falls inside it.  A piece of a tile that was cut goes, unnormalised in
// fp32 with its maximum and sum, to one of the CTA's two places in the
// workspace (the first piece of its share, or the last), and a second kernel
// joins the pieces.  The lengths are in device memory, so every CTA computes
// the line's prefix sums over the requests by itself.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "paged_common.cuh"

namespace cider {
namespace {

constexpr int kRows = 16;      // rows of a tile (mma M)
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 16;      // keys per warp and step
constexpr int kBlock = kWarps * kStep;  // keys per block of the line
constexpr int kStages = 3;
constexpr int kCtasPerSm = 2;
// Shortest share of a CTA, in blocks: below it the pieces' join costs more
// than the parallelism gains.
constexpr int kMinShare = 1;

__device__ __forceinline__ float ex2(float x) {  // 2^x, PTX ex2.approx (relative error near 2^-22)
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Weights are made as 2^(x + kPOff): for fp16 up to 2^15, so that weights down
// to 2^-29 of the largest keep all 11 bits (fp16 is subnormal below 2^-14);
// bf16 has the range of fp32.  The factor cancels in O / l.
template <typename T>
constexpr float kPOff = std::is_same<T, __half>::value ? 15.0f : 0.0f;

template <typename T>
__device__ __forceinline__ bool any_nonfinite(const uint4& v) {
    constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= (w[i] & e) == e || (w[i] & (e << 16)) == (e << 16);
    return bad;
}

// The line of blocks: request b's tiles and blocks per tile.
struct Line {
    int64_t total, share;
};
__device__ __forceinline__ int64_t request_blocks(const PagedAttnArgs& a, const PagedRequest& r, int* tiles, int* blocks) {
    const int rows = r.n * a.G;
    *tiles = (rows + kRows - 1) / kRows;
    *blocks = 0;
    if (r.n == 0) return 0;
    // the most that any of its tiles reads; a tile that sees nothing still has
    // one block, so that its zeros get written
    PagedSpan<kBlock> last;
    const int span = min(r.n, (kRows - 1) / a.G + 2);  // most tokens in a tile
    last.set(max(r.L - span, r.L - r.n), r.L - 1, a.window, a.sinks);
    // earlier tiles: no more blocks without a window; with one, the window's
    // start may fall one block earlier
    *blocks = max(1, last.blocks + (a.window > 0 && *tiles > 1 ? 1 : 0));
    return static_cast<int64_t>(*tiles) * a.c.H_kv * *blocks;
}

// pre[b] = blocks of the requests before b.  Returns the line and reports bad
// lengths (block 0).
__device__ __forceinline__ Line make_line(const PagedAttnArgs& a, int64_t* pre, int64_t* s_warp, bool report) {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    int64_t sum = 0;
    bool any_bad = false;
    for (int b = b0; b < b1; ++b) {
        bool bad;
        int tiles, blocks;
        const PagedRequest r = paged_request(a, b, &bad);
        any_bad |= bad;
        pre[b] = sum;
        sum += request_blocks(a, r, &tiles, &blocks);
    }
    if (any_bad && report) atomicOr(a.status, kStatusIndex);
    Line line;
    const int64_t base = block_prefix<kThreads>(sum, s_warp, &line.total);
    for (int b = b0; b < b1; ++b) pre[b] += base;
    if (threadIdx.x == 0) pre[a.B] = line.total;
    __syncthreads();
    line.share = max(static_cast<int64_t>(kMinShare), (line.total + a.grid - 1) / a.grid);
    return line;
}

// One tile: a request, a KV head, 16 rows.
struct Tile {
    PagedRequest r;
    int b, head, row0, rows;  // rows [row0, row0 + rows) of the request's (token, head) rows
    int blocks;               // its length on the line
    int64_t begin;            // its first block on the line
};
__device__ __forceinline__ Tile find_tile(const PagedAttnArgs& a, const int64_t* pre, int64_t x) {
    Tile t;
    t.b = find_request(pre, a.B, x);
    bool bad;
    int tiles;
    t.r = paged_request(a, t.b, &bad);
    request_blocks(a, t.r, &tiles, &t.blocks);
    const int64_t u = (x - pre[t.b]) / t.blocks;  // tile * H_kv + head
    t.begin = pre[t.b] + u * t.blocks;
    t.head = static_cast<int>(u % a.c.H_kv);
    t.row0 = static_cast<int>(u / a.c.H_kv) * kRows;
    t.rows = min(kRows, t.r.n * a.G - t.row0);
    return t;
}

// Element offset of a request's (token, head) row f in q (at ld) or out.
__device__ __forceinline__ int64_t row_offset(const PagedAttnArgs& a, int start, int head, int f, int64_t ld) {
    const int i = f / a.G;
    return (start + i) * ld + static_cast<int64_t>(head * a.G + (f - i * a.G)) * a.c.D;
}

// A tile in several pieces, in the record of the CTA that has the first: their
// number, the first one's slot (the others are in slot 0 of the CTAs behind),
// and the tile's place in out.  0 pieces: none.
struct Join {
    int pieces, slot, start, head, row0, rows;
};

// Workspace: two places per CTA for partial results (slot 0: the first piece of
// its share, 1: the last one), their maxima and sums, and a record per CTA.
template <int D>
__device__ __forceinline__ float* part_o(const PagedAttnArgs& a, int64_t c, int slot) {
    return a.part + (c * 2 + slot) * (kRows * D);
}
template <int D>
__device__ __forceinline__ float2* part_ml(const PagedAttnArgs& a, int64_t c, int slot) {
    return reinterpret_cast<float2*>(a.part + static_cast<int64_t>(a.grid) * 2 * kRows * D) + (c * 2 + slot) * kRows;
}

template <int D>
__device__ __forceinline__ Join* part_join(const PagedAttnArgs& a) {
    return reinterpret_cast<Join*>(a.part + static_cast<int64_t>(a.grid) * 2 * kRows * (D + 2));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) k_paged_attn(const __grid_constant__ CUtensorMap tmK,
                                                                     const __grid_constant__ CUtensorMap tmV,
                                                                     const __grid_constant__ PagedAttnArgs a) {
    constexpr int kHalf = kStep * D * 2;                 // bytes of K (or V) of one step
    constexpr int kAtom = kStep * 128;                   // bytes of 64 dims of it
    constexpr int kPieces = kStep * (D / 8) / 32;        // 16-byte pieces of V per lane and step
    constexpr int kNd = D / 16;                          // d-steps of 16
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t s_full[kWarps][kStages];
    __shared__ int s_abort;
    __shared__ int64_t s_warp[kWarps];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int64_t* pre = reinterpret_cast<int64_t*>(ring + kWarps * kStages * 2 * kHalf);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, qd = lane & 3;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int i = 0; i < kWarps * kStages; ++i) mbar_init(&s_full[0][0] + i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    uint64_t* full = s_full[warp];
    pdl_wait();
    pdl_trigger();
    const Line line = make_line(a, pre, s_warp, blockIdx.x == 0);  // its barriers also publish the mbarriers
    const int64_t x1 = min(line.total, (blockIdx.x + 1) * line.share);
    uint8_t* my_ring = ring + warp * (kStages * 2 * kHalf);
    const uint32_t my_ring_u = smem_u32(my_ring);
    bool ok = true;          // no wait has run out
    uint32_t loads = 0;      // steps of this warp before the tile's: the ring goes on across tiles
    // where a lane's rows of a ldmatrix begin within an atom, for its 16 dims 0 .. 3
    const int mm = lane >> 3, mr = lane & 7;
    uint32_t k_off[4], v_off[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        k_off[i] = ((mm >> 1) * 8 + mr) * 128 + (((2 * i + (mm & 1)) ^ mr) << 4);
        v_off[i] = ((mm & 1) * 8 + mr) * 128 + (((2 * i + (mm >> 1)) ^ mr) << 4);
    }

    if (threadIdx.x == 0) part_join<D>(a)[blockIdx.x].pieces = 0;
    for (int64_t x = blockIdx.x * line.share; x < x1;) {
        const Tile t = find_tile(a, pre, x);
        const int64_t xe = min(x1, t.begin + t.blocks);
        PagedSpan<kBlock> span;
        const int i0 = t.row0 / a.G, i1 = (t.row0 + t.rows - 1) / a.G;
        span.set(t.r.L - t.r.n + i0, t.r.L - t.r.n + i1, a.window, a.sinks);
        const int vb0 = static_cast<int>(x - t.begin);
        const int nsteps = max(0, min(static_cast<int>(xe - t.begin), span.blocks) - vb0);  // the same for all warps
        const int32_t* table = a.table + t.b * a.ld_table;

        // Queries: fragments of the 16 x D tile, zero rows beyond it.  Lane
        // (g, qd) holds rows g and g + 8, dims 16 kk + 2 qd + {0, 1} and + 8.
        uint32_t qf[kNd][4];
        int pos[2];
        {
            const T* q0 = static_cast<const T*>(a.q);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int row = g + 8 * hh;
                pos[hh] = t.r.L - t.r.n + (t.row0 + row) / a.G;
                const bool live = row < t.rows;
                const T* p = q0 + (live ? row_offset(a, t.r.start, t.head, t.row0 + row, a.ld_q) : 0) + 2 * qd;
#pragma unroll
                for (int kk = 0; kk < kNd; ++kk) {
                    qf[kk][hh] = live ? __ldg(reinterpret_cast<const uint32_t*>(p + kk * 16)) : 0u;
                    qf[kk][2 + hh] = live ? __ldg(reinterpret_cast<const uint32_t*>(p + kk * 16 + 8)) : 0u;
                }
            }
        }

        float o[2 * kNd][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 2 * kNd; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;

        // Page numbers of 32 steps of this warp, one per lane; -1: none, or one
        // that the cache does not have.  `lost`: a bit per stage of the ring
        // whose step has no page.
        int pages = -1;
        uint32_t lost = 0;
        auto fetch_pages = [&](int s) {
            pages = -1;
            if (s + lane < nsteps) {
                const int key0 = span.block(vb0 + s + lane) * kBlock + warp * kStep;
                if (key0 < t.r.L) {
                    const int e = key0 >> a.c.ps_log2;  // < width, because L <= width * page_size
                    const bool used = key0 <= span.pmax && (a.window <= 0 || key0 + kStep - 1 > span.pmin - a.window || key0 < a.sinks);
                    if (used) {
                        const int p = __ldg(table + e);
                        if (p >= 0 && p < a.c.num_pages)
                            pages = p;
                        else
                            atomicOr(a.status, kStatusIndex);
                    }
                }
            }
        };
        // Starts the copies of step s into its stage.  The pages of steps s ..
        // are in `pages` (refilled every 32 steps).
        auto load_step = [&](int s) {
            if (s >= nsteps) return;
            if ((s & 31) == 0) fetch_pages(s);
            const int page = __shfl_sync(0xffffffffu, pages, s & 31);
            const int st = (loads + s) % kStages;
            lost = page >= 0 ? lost & ~(1u << st) : lost | (1u << st);
            if (lane == 0) {
                uint8_t* dst = my_ring + st * (2 * kHalf);
                if (page < 0) {
                    mbar_arrive(&full[st]);
                    return;
                }
                mbar_arrive_expect_tx(&full[st], 2 * kHalf);
                const int key0 = span.block(vb0 + s) * kBlock + warp * kStep;
                int c[4] = {0, page, page, page};
#pragma unroll
                for (int d = 1; d < 4; ++d) {
                    if (d == a.d_tok) c[d] = key0 & (a.c.page_size - 1);
                    if (d == a.d_head) c[d] = t.head;
                }
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    tma_load_4d(dst + h * kAtom, &tmK, &full[st], h * 64, c[1], c[2], c[3]);
                    tma_load_4d(dst + kHalf + h * kAtom, &tmV, &full[st], h * 64, c[1], c[2], c[3]);
                }
            }
        };

#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) load_step(s);
        for (int s = 0; s < nsteps; ++s) {
            __syncwarp();  // every lane has read the stage that the next copies overwrite
            load_step(s + kStages - 1);
            const uint32_t n = loads + s, stage = n % kStages;
            if (ok) ok = mbar_wait(&full[stage], (n / kStages) & 1, a.status, &s_abort);
            __syncwarp();
            if ((lost >> stage) & 1u) continue;  // no page: nothing of the step is seen
            uint8_t* sv = my_ring + stage * (2 * kHalf) + kHalf;
            const uint32_t kst = my_ring_u + stage * (2 * kHalf);
            const uint32_t vst = kst + kHalf;
            const int key0 = span.block(vb0 + s) * kBlock + warp * kStep;

            float sc[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[j][e] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < kNd; ++kk) {
                uint32_t b[4];
                ldsm4(kst + (kk >> 2) * kAtom + k_off[kk & 3], b);
                mma16816<T>(sc[0], qf[kk], b[0], b[1]);
                mma16816<T>(sc[1], qf[kk], b[2], b[3]);
            }
            // masks, unless every row sees every key of the step
            const bool whole = key0 + kStep - 1 <= span.pmin &&
                               (a.window <= 0 || key0 > span.pmax - a.window || key0 + kStep <= a.sinks);
            // A row that has seen a key has a finite maximum, even if the score
            // was -inf (its result is then 0 / 0, as the formula's), and only
            // one that has seen none keeps -inf (its result is 0).
            float low[2] = {-FLT_MAX, -FLT_MAX};
            if (!whole) {
                low[0] = low[1] = -INFINITY;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + j * 8 + 2 * qd + (e & 1);
                        if (paged_sees(key, pos[e >> 1], a.window, a.sinks))
                            low[e >> 1] = -FLT_MAX;
                        else
                            sc[j][e] = -INFINITY;
                    }
            }
            // running maximum, weights
            float mn[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                float x0 = fmaxf(fmaxf(sc[0][2 * hh], sc[0][2 * hh + 1]), fmaxf(sc[1][2 * hh], sc[1][2 * hh + 1]));
                x0 = fmaxf(x0, low[hh]);
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
                mn[hh] = fmaxf(m[hh], x0);
            }
            if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const float f = mn[hh] == m[hh] ? 1.0f : ex2((m[hh] - mn[hh]) * a.qscale);  // first keys: 2^-inf = 0
                    l[hh] *= f;
                    m[hh] = mn[hh];
#pragma unroll
                    for (int j = 0; j < 2 * kNd; ++j) {
                        o[j][2 * hh] *= f;
                        o[j][2 * hh + 1] *= f;
                    }
                }
            }
            float p[2][4];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const float ms = (m[hh] == -INFINITY ? 0.0f : m[hh]) * a.qscale - kPOff<T>;  // nothing seen yet: all p = 0
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        p[j][2 * hh + e] = ex2(fmaf(sc[j][2 * hh + e], a.qscale, -ms));
                        l[hh] += p[j][2 * hh + e];
                    }
            }
            // O += P V
            bool slow = false;
            if (!whole) {
                // Rows of V that no query of the tile sees become zeros.  If another
                // one, which some of the queries see and some do not, holds NaN or an
                // infinity, 0 x V would reach the queries that must not see it.
                bool nf = false;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    uint4* piece = reinterpret_cast<uint4*>(sv) + i * 32 + lane;
                    const int j = key0 + (((i * 32 + lane) >> 3) & (kStep - 1));
                    if (j <= span.pmax && (a.window <= 0 || j > span.pmin - a.window || j < a.sinks))
                        nf |= any_nonfinite<T>(*piece);
                    else
                        *piece = make_uint4(0, 0, 0, 0);
                }
                fence_async_shared();  // before the copies that will overwrite it
                slow = __any_sync(0xffffffffu, nf) && i0 != i1;
                __syncwarp();
            }
            if (!slow) {
                uint32_t pa[4];
                pa[0] = pack2_out<T>(p[0][0], p[0][1]);
                pa[1] = pack2_out<T>(p[0][2], p[0][3]);
                pa[2] = pack2_out<T>(p[1][0], p[1][1]);
                pa[3] = pack2_out<T>(p[1][2], p[1][3]);
#pragma unroll
                for (int jj = 0; jj < kNd; ++jj) {
                    uint32_t b[4];
                    ldsm4_t(vst + (jj >> 2) * kAtom + v_off[jj & 3], b);
                    mma16816<T>(o[2 * jj], pa, b[0], b[1]);
                    mma16816<T>(o[2 * jj + 1], pa, b[2], b[3]);
                }
            } else {
                for (int key = 0; key < kStep; ++key) {
                    const int src = (lane & ~3) | ((key & 7) >> 1);
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        // p of (row, key): tile key / 8, element key % 2, of lane src
                        float w = 0.0f;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float y = __shfl_sync(0xffffffffu, p[j][2 * hh + e], src);
                                if (j == (key >> 3) && e == (key & 1)) w = y;
                            }
                        if (paged_sees(key0 + key, pos[hh], a.window, a.sinks)) {
#pragma unroll
                            for (int j = 0; j < 2 * kNd; ++j)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    o[j][2 * hh + e] += w * to_f32<T>(*reinterpret_cast<const T*>(
                                                                sv + (j >> 3) * kAtom + key * 128 + (((j & 7) ^ (key & 7)) << 4) + (2 * qd + e) * 2));
                        }
                    }
                }
            }
        }
        loads += nsteps;
        // Join the four warps' keys: rescale to the common maximum, then add.
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
            l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
            if (qd == 0) {
                s_m[warp][g + 8 * hh] = m[hh];
                s_l[warp][g + 8 * hh] = l[hh];
            }
        }
        __syncthreads();  // also: every warp is done with its ring
        constexpr int kLdO = D + 8;  // padded rows of the exchange
        float* so = reinterpret_cast<float*>(ring) + warp * (kRows * kLdO);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int row = g + 8 * hh;
            float mx = s_m[0][row];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][row]);
            const float f = m[hh] == mx ? 1.0f : ex2((m[hh] - mx) * a.qscale);  // no keys in this warp: 2^-inf = 0
#pragma unroll
            for (int j = 0; j < 2 * kNd; ++j)
                *reinterpret_cast<float2*>(so + row * kLdO + j * 8 + 2 * qd) = make_float2(o[j][2 * hh] * f, o[j][2 * hh + 1] * f);
        }
        __syncthreads();
        const bool whole_tile = x == t.begin && xe == t.begin + t.blocks;
        const int slot = x == blockIdx.x * line.share ? 0 : 1;
        if (threadIdx.x == 0 && x == t.begin && !whole_tile)  // this CTA's last piece: the tile goes on in the next ones
            part_join<D>(a)[blockIdx.x] = Join{static_cast<int>((t.begin + t.blocks - 1) / line.share) - static_cast<int>(blockIdx.x) + 1,
                                               slot, t.r.start, t.head, t.row0, t.rows};
        for (int e = threadIdx.x; e < t.rows * (D / 4); e += kThreads) {
            const int row = e / (D / 4), d4 = (e % (D / 4)) * 4;
            float mx = s_m[0][row], ls = 0.0f;
#pragma unroll
            for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][row]);
            float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                ls += s_m[w][row] == mx ? s_l[w][row] : s_l[w][row] * ex2((s_m[w][row] - mx) * a.qscale);
                const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(ring) + (w * kRows + row) * kLdO + d4);
                v.x += y.x;
                v.y += y.y;
                v.z += y.z;
                v.w += y.w;
            }
            if (whole_tile) {
                const float inv = mx == -INFINITY ? 0.0f : 1.0f / ls;  // nothing seen: zeros
                uint2 w2;
                w2.x = pack2_out<T>(v.x * inv, v.y * inv);
                w2.y = pack2_out<T>(v.z * inv, v.w * inv);
                *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row_offset(a, t.r.start, t.head, t.row0 + row, a.ld_out) + d4) = w2;
            } else {
                *reinterpret_cast<float4*>(part_o<D>(a, blockIdx.x, slot) + row * D + d4) = v;
                if (d4 == 0) part_ml<D>(a, blockIdx.x, slot)[row] = make_float2(mx, ls);
            }
        }
        fence_async_shared();  // the exchange, before the copies that overwrite it
        __syncthreads();       // the ring is free for the next tile
        x = xe;
    }
    if (s_abort) {  // a wait ran out: give this CTA's copies in flight time to land
        const unsigned long long t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
}

// Joins the pieces of the tile in CTA c's record, c = blockIdx.x:
// out = sum_c O_c 2^(m_c - M) / sum_c l_c 2^(m_c - M).  A tile may have as many
// pieces as there are CTAs, so the threads that a tile's rows leave over share
// the pieces.
constexpr int kJoinThreads = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) k_paged_join(const __grid_constant__ PagedAttnArgs a) {
    extern __shared__ float wgt[];  // [pieces][kRows]
    __shared__ float s_inv[kRows];
    __shared__ float4 s_sum[kJoinThreads];
    pdl_wait();
    pdl_trigger();
    const Join t = part_join<D>(a)[blockIdx.x];
    if (t.pieces == 0) return;
    const int64_t c0 = blockIdx.x;
    const int np = t.pieces;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto slot_of = [&](int i) { return i == 0 ? t.slot : 0; };
    for (int row = warp; row < t.rows; row += kJoinThreads / 32) {
        float mx = -INFINITY, ls = 0.0f;
        for (int i = lane; i < np; i += 32) mx = fmaxf(mx, part_ml<D>(a, c0 + i, slot_of(i))[row].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        for (int i = lane; i < np; i += 32) {
            const float2 ml = part_ml<D>(a, c0 + i, slot_of(i))[row];
            const float f = ml.x == mx ? 1.0f : ex2((ml.x - mx) * a.qscale);
            wgt[i * kRows + row] = f;
            ls += ml.y * f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
        if (lane == 0) s_inv[row] = mx == -INFINITY ? 0.0f : 1.0f / ls;
    }
    __syncthreads();
    // four dims of a row per thread; `groups` threads share its pieces
    const int items = t.rows * (D / 4);
    const int groups = max(1, kJoinThreads / items);
    for (int e0 = 0; e0 < items; e0 += kJoinThreads) {
        const int e = groups > 1 ? static_cast<int>(threadIdx.x) % items : e0 + static_cast<int>(threadIdx.x);
        const int g = groups > 1 ? static_cast<int>(threadIdx.x) / items : 0;
        const int row = e / (D / 4), d4 = (e % (D / 4)) * 4;
        float4 v = make_float4(0, 0, 0, 0);
        if (g < groups && e < items) {
#pragma unroll 8
            for (int i = g; i < np; i += groups) {
                const float f = wgt[i * kRows + row];
                const float4 y = *reinterpret_cast<const float4*>(part_o<D>(a, c0 + i, slot_of(i)) + row * D + d4);
                v.x = fmaf(y.x, f, v.x);
                v.y = fmaf(y.y, f, v.y);
                v.z = fmaf(y.z, f, v.z);
                v.w = fmaf(y.w, f, v.w);
            }
        }
        if (groups > 1) {
            s_sum[threadIdx.x] = v;
            __syncthreads();
            if (g == 0)
                for (int i = 1; i < groups; ++i) {
                    const float4 y = s_sum[i * items + e];
                    v.x += y.x;
                    v.y += y.y;
                    v.z += y.z;
                    v.w += y.w;
                }
        }
        if (g == 0 && e < items) {
            const float inv = s_inv[row];
            uint2 w2;
            w2.x = pack2_out<T>(v.x * inv, v.y * inv);
            w2.y = pack2_out<T>(v.z * inv, v.w * inv);
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row_offset(a, t.start, t.head, t.row0 + row, a.ld_out) + d4) = w2;
        }
    }
}

template <typename T, int D>
cudaError_t launch_t(PagedAttnArgs a, int num_sms, cudaStream_t st) {
    a.grid = kCtasPerSm * num_sms;
    CUtensorMap tmK, tmV;
    if (!paged_cache_maps(a.c, kStep, &tmK, &tmV, &a.d_tok, &a.d_head)) return cudaErrorInvalidValue;
    const int ring = 1024 + kWarps * kStages * 2 * kStep * D * 2;
    const int pre = (a.B + 1) * 8;
    auto kern = k_paged_attn<T, D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ring + pre);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(a.grid), dim3(kThreads), ring + pre, st, tmK, tmV, a);
    if (e != cudaSuccess) return e;
    const int wgt = a.grid * kRows * 4;
    return launch_pdl(k_paged_join<T, D>, dim3(a.grid), dim3(kJoinThreads), wgt, st, a);
}

}  // namespace

size_t paged_rows16_bytes(int D, int num_sms) {
    return static_cast<size_t>(kCtasPerSm) * num_sms * (2 * kRows * (D + 2) * 4 + sizeof(Join));
}

cudaError_t launch_paged_rows16(PagedAttnArgs a, int num_sms, cudaStream_t st) {
    if (a.c.dt == 1) return a.c.D == 128 ? launch_t<__nv_bfloat16, 128>(a, num_sms, st) : launch_t<__nv_bfloat16, 64>(a, num_sms, st);
    return a.c.D == 128 ? launch_t<__half, 128>(a, num_sms, st) : launch_t<__half, 64>(a, num_sms, st);
}

}  // namespace cider
