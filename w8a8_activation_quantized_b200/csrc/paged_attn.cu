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
// Loads: a fifth warp copies 64-key blocks of K and V (TMA, 128-byte swizzle,
// one box per page and 64 dims) into a ring of 96 KB, ahead of the four warps
// that use them, each 16 keys of a block, and on into the next tile; two CTAs
// per SM keep up to 192 KB in flight.  (The using warps' instructions set the
// pace where the bytes do not: with 16-byte cp.async of their own, and with TMA
// of their own, four requests of up to 32K keys took 49.5 and 45.2 us, with this
// warp 41.)  Pages that
// no query of the tile sees are not read; their boxes lie outside the tensor
// map, which makes them zeros.  Where only some keys of a step are seen by any
// query, the other rows of V are zeroed in shared memory: what the cache's
// unwritten slots hold may be NaN, and 0 x NaN is not 0.
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
//
// Measured (with the join, calls back to back): 64 requests of up to 8K keys, 32 / 8
// heads, D = 128: 208 to 212 us, 6.4 to 6.5 TB/s, the rate of a copy; 4 of up to
// 32K, 32 / 4 heads: 41 to 43 us, of which the 176 MB are 27 and the start and the
// join the rest; 16 windows of 4096 keys, 32 / 32 heads, D = 64: 96 us, 5.6 TB/s;
// one request of 1000 keys: 11.3 us, the two launches' chains of loads.
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
constexpr int kUsers = kWarps * 32;       // threads of the warps that compute; one more warp loads
constexpr int kThreads = kUsers + 32;
constexpr int kStep = 16;      // keys per warp and step
constexpr int kBlock = kWarps * kStep;  // keys per block of the line
template <int D>
constexpr int kRing = D == 128 ? 3 : 6;  // blocks in the ring: 96 KB
constexpr int kCtasPerSm = 2;
// Shortest share of a CTA, in blocks: with 2 or 3 there would be fewer pieces to
// join, but one short request (1000 keys) and four long ones were slower.
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

// Barrier of the warps that compute.
__device__ __forceinline__ void users_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(kUsers) : "memory");
}

__device__ __forceinline__ bool users_or(bool x) {  // true if any thread passes true
    uint32_t y;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, 1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(y)
        : "r"(static_cast<uint32_t>(x)), "n"(kUsers)
        : "memory");
    return y != 0;
}

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
    line.share = max(static_cast<int64_t>(kMinShare), div_nonneg(line.total + a.grid - 1, a.grid));
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
    const int64_t u = div_nonneg(x - pre[t.b], t.blocks);  // tile * H_kv + head
    t.begin = pre[t.b] + u * t.blocks;
    const int tile = static_cast<int>(div_nonneg(u, a.c.H_kv));
    t.head = static_cast<int>(u - static_cast<int64_t>(tile) * a.c.H_kv);
    t.row0 = tile * kRows;
    t.rows = min(kRows, t.r.n * a.G - t.row0);
    return t;
}

// A piece of a tile that a CTA computes: found, with its queries, by the warp that
// loads, while the others are busy with the one before.
struct Piece {
    Tile t;
    PagedSpan<kBlock> span;
    int vb0, vb1;  // its blocks of the span; vb1 < 0: no more pieces
    int slot;      // of its partial result; -1: it is the whole tile
};

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
    constexpr int kStages = kRing<D>;
    constexpr int kAtom = kBlock * 128;                  // bytes of 64 dims of a block
    constexpr int kHalf = kBlock * D * 2;                // bytes of K (or V) of a block
    constexpr int kPieces = kStep * (D / 8) / 32;        // 16-byte pieces of V per lane and step
    constexpr int kNd = D / 16;                          // d-steps of 16
    static_assert(kWarps * kRows * D * 4 <= 2 * kHalf, "the warps' exchange fits one stage");
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ uint32_t s_lost[kStages];                 // per 16 keys of a block: the page is missing
    __shared__ int s_abort;
    __shared__ int64_t s_warp[kThreads / 32];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    __shared__ Piece s_piece[2];
    __shared__ __align__(128) uint4 s_q[2][D / 64][kRows][8];  // queries of a piece: [64 dims][row][8 dims]
    __shared__ uint64_t piece_full[2], piece_empty[2];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int64_t* pre = reinterpret_cast<int64_t*>(ring + kStages * 2 * kHalf);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&piece_full[i], 1);
            mbar_init(&piece_empty[i], 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    pdl_wait();
    pdl_trigger();
    const Line line = make_line(a, pre, s_warp, blockIdx.x == 0);  // its barriers also publish the mbarriers
    const int64_t x1 = min(line.total, (blockIdx.x + 1) * line.share);
    bool ok = true;      // false: a wait has run out, and no other one is begun
    uint32_t blk = 0;    // blocks of the ring so far

    if (warp == kWarps) {
        // ------------------------------- loads -------------------------------
        const int box_keys = min(a.c.page_size, kBlock), boxes = kBlock / box_keys;  // 1, 2 or 4 pages per block
        const int box = lane % boxes, half = (lane / boxes) % (D / 64), kv = lane / boxes / (D / 64);
        if (lane == 0) part_join<D>(a)[blockIdx.x].pieces = 0;
        int64_t x = blockIdx.x * line.share;
        for (int n = 0; ok; ++n) {
            const int buf = n & 1;
            ok = mbar_wait(&piece_empty[buf], ((n >> 1) & 1) ^ 1, a.status, &s_abort);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            if (x >= x1) {  // no more pieces
                if (lane == 0) {
                    s_piece[buf].vb1 = -1;
                    mbar_arrive(&piece_full[buf]);
                }
                break;
            }
            const Tile t = find_tile(a, pre, x);
            const int64_t xe = min(x1, t.begin + t.blocks);
            PagedSpan<kBlock> span;
            span.set(t.r.L - t.r.n + t.row0 / a.G, t.r.L - t.r.n + (t.row0 + t.rows - 1) / a.G, a.window, a.sinks);
            const int vb0 = static_cast<int>(x - t.begin), vb1 = min(static_cast<int>(xe - t.begin), span.blocks);
            const int32_t* table = a.table + t.b * a.ld_table;
            // The page numbers of 32 / boxes blocks from vb on, one per lane, and a
            // bit per lane whose page is missing.
            int pages = 0;
            uint32_t bad = 0;
            auto fetch_pages = [&](int vb) {
                pages = a.c.num_pages;  // outside the map
                bool missing = false;
                const int b = vb + lane / boxes;
                const int key0 = b < vb1 ? span.block(b) * kBlock + box * box_keys : INT_MAX;
                // (below L <= width * page_size, because pmax is)
                if (key0 <= span.pmax && (a.window <= 0 || key0 + box_keys - 1 > span.pmin - a.window || key0 < a.sinks)) {
                    const int p = __ldg(table + (key0 >> a.c.ps_log2));
                    if (p >= 0 && p < a.c.num_pages)
                        pages = p;
                    else
                        missing = true;
                }
                if (missing) atomicOr(a.status, kStatusIndex);
                bad = __ballot_sync(0xffffffffu, missing);
            };
            // the piece and its queries, zero rows beyond the tile's
            {
                constexpr int kQ = kRows * (D / 8) / 32;
                uint4 q[kQ];
#pragma unroll
                for (int i = 0; i < kQ; ++i) {
                    const int e = i * 32 + lane, row = e / (D / 8);
                    q[i] = make_uint4(0, 0, 0, 0);
                    if (row < t.rows)
                        q[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + row_offset(a, t.r.start, t.head, t.row0 + row, a.ld_q)) + e % (D / 8));
                }
                fetch_pages(vb0);
#pragma unroll
                for (int i = 0; i < kQ; ++i) {
                    const int e = i * 32 + lane, row = e / (D / 8), c = e % (D / 8);
                    s_q[buf][c >> 3][row][(c & 7) ^ (row & 7)] = q[i];
                }
                if (lane == 0) {
                    const int slot = x == t.begin && xe == t.begin + t.blocks ? -1 : x == blockIdx.x * line.share ? 0 : 1;
                    s_piece[buf] = Piece{t, span, vb0, vb1, slot};
                    if (slot >= 0 && x == t.begin)  // this CTA's last piece: the tile goes on in the next ones
                        part_join<D>(a)[blockIdx.x] = Join{static_cast<int>(div_nonneg(t.begin + t.blocks - 1, line.share)) - static_cast<int>(blockIdx.x) + 1,
                                                           slot, t.r.start, t.head, t.row0, t.rows};
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&piece_full[buf]);
            }
            for (int vb = vb0; vb < vb1; ++vb, ++blk) {
                const int in_batch = (vb - vb0) % (32 / boxes);
                if (in_batch == 0 && vb > vb0) fetch_pages(vb);
                const int page = __shfl_sync(0xffffffffu, pages, in_batch * boxes + box);
                const int st = blk % kStages;
                if (ok) ok = mbar_wait(&empty[st], ((blk / kStages) & 1) ^ 1, a.status, &s_abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    uint32_t lost = 0;
                    if (bad)
                        for (int w = 0; w < kWarps; ++w) lost |= ((bad >> (in_batch * boxes + w * boxes / kWarps)) & 1u) << w;
                    s_lost[st] = lost;
                    mbar_arrive_expect_tx(&full[st], 2 * kHalf);
                }
                __syncwarp();
                if (kv < 2) {
                    int c[4] = {0, page, page, page};
#pragma unroll
                    for (int d = 1; d < 4; ++d) {
                        if (d == a.d_tok) c[d] = (span.block(vb) * kBlock) & (a.c.page_size - 1);
                        if (d == a.d_head) c[d] = t.head;
                    }
                    tma_load_4d(ring + st * (2 * kHalf) + kv * kHalf + half * kAtom + box * box_keys * 128, kv ? &tmV : &tmK, &full[st],
                                half * 64, c[1], c[2], c[3]);
                }
                __syncwarp();
            }
            x = xe;
        }
    } else {
        // ------------------------------ products ------------------------------
        const int g = lane >> 2, qd = lane & 3;
        // Where a lane's row of a ldmatrix begins in a stage, for the first 16 dims
        // of an atom; the swizzle turns the i-th 16 dims into an exclusive or.
        const int mm = lane >> 3, mr = lane & 7;
        const uint32_t k_off = warp * (kStep * 128) + ((mm >> 1) * 8 + mr) * 128 + (((mm & 1) ^ mr) << 4);
        const uint32_t q_off = ((mm & 1) * 8 + mr) * 128 + (((mm >> 1) ^ mr) << 4);
        const uint32_t v_off = kHalf + warp * (kStep * 128) + ((mm & 1) * 8 + mr) * 128 + (((mm >> 1) ^ mr) << 4);
        for (int n = 0;; ++n) {
            const int buf = n & 1;
            if (ok) ok = mbar_wait(&piece_full[buf], (n >> 1) & 1, a.status, &s_abort);
            if (users_or(!ok)) break;  // all go on, or none
            const PagedSpan<kBlock> span = s_piece[buf].span;
            const int vb0 = s_piece[buf].vb0, vb1 = s_piece[buf].vb1;
            if (vb1 < 0) break;
            int pos[2];
            {
                const Tile t = s_piece[buf].t;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) pos[hh] = t.r.L - t.r.n + (t.row0 + g + 8 * hh) / a.G;
            }
            // The queries stay in shared memory at D = 128: in registers, 32, they
            // would spill others (four requests of up to 32K keys, when that was tried: 49.0
            // and 46.3 us).
            const uint32_t q_row = smem_u32(s_q[buf]) + q_off;
            uint32_t q[kNd][4];
            if (D == 64)
#pragma unroll
                for (int kk = 0; kk < kNd; ++kk) ldsm4(q_row ^ ((kk & 3) << 5), q[kk]);

            float o[2 * kNd][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 2 * kNd; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;

            for (int vb = vb0; vb < vb1; ++vb, ++blk) {
                const int st = blk % kStages;
                if (ok) ok = mbar_wait(&full[st], (blk / kStages) & 1, a.status, &s_abort);
                __syncwarp();
                const uint32_t stage = smem_u32(ring) + st * (2 * kHalf);
                const int key0 = span.block(vb) * kBlock + warp * kStep;
                const bool lost = (s_lost[st] >> warp) & 1u;

                float sa[2][4], sc[2][4];  // two chains of products each
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sa[j][e] = sc[j][e] = 0.0f;
#pragma unroll
                for (int kk = 0; kk < kNd; ++kk) {
                    uint32_t b[4];
                    if (D != 64) ldsm4((q_row ^ ((kk & 3) << 5)) + (kk >> 2) * (kRows * 128), q[kk]);
                    ldsm4(((stage + k_off) ^ ((kk & 3) << 5)) + (kk >> 2) * kAtom, b);
                    mma16816<T>(kk & 1 ? sa[0] : sc[0], q[kk], b[0], b[1]);
                    mma16816<T>(kk & 1 ? sa[1] : sc[1], q[kk], b[2], b[3]);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[j][e] += sa[j][e];
                // Masks, unless every row sees every key of the step.  A row that has
                // seen a key has a finite maximum, even if its scores were all -inf
                // (-FLT_MAX, a mark; if that stays its result is 0 / 0, as the
                // formula's), and only one that has seen none keeps -inf (its result is 0).
                float low[2] = {-FLT_MAX, -FLT_MAX};
                const bool whole = !lost && key0 + kStep - 1 <= span.pmin &&
                                   (a.window <= 0 || key0 > span.pmax - a.window || key0 + kStep <= a.sinks);
                bool slow = false;
                if (!whole) {
                    low[0] = low[1] = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = key0 + j * 8 + 2 * qd + (e & 1);
                            if (!lost && paged_sees(key, pos[e >> 1], a.window, a.sinks))
                                low[e >> 1] = -FLT_MAX;
                            else
                                sc[j][e] = -INFINITY;
                        }
                    // Rows of V that no query of the tile sees become zeros.  If another
                    // one, which some of the queries see and some do not, holds NaN or an
                    // infinity, 0 x V would reach the queries that must not see it.
                    bool nf = false;
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const int e = i * 32 + lane, row = (e >> 3) & (kStep - 1);
                        uint4* piece = reinterpret_cast<uint4*>(ring + st * (2 * kHalf) + kHalf + (e >> 7) * kAtom + (warp * kStep + row) * 128) + (e & 7);
                        const int j = key0 + row;
                        if (j <= span.pmax && (a.window <= 0 || j > span.pmin - a.window || j < a.sinks))
                            nf |= any_nonfinite<T>(*piece);
                        else
                            *piece = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_shared();  // before the copies that will overwrite it
                    slow = __any_sync(0xffffffffu, nf) && span.pmin != span.pmax;
                    __syncwarp();
                }
                // running maximum, weights
                float mn[2];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    float y = fmaxf(fmaxf(sc[0][2 * hh], sc[0][2 * hh + 1]), fmaxf(sc[1][2 * hh], sc[1][2 * hh + 1]));
                    y = fmaxf(y, low[hh]);
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
                    mn[hh] = fmaxf(m[hh], y);
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
                    // The difference comes before the scale: m times the scale would be rounded
                    // to more than a unit of the exponent for large scores, and may overflow.
                    const float mu = m[hh] == -INFINITY ? 0.0f : m[hh];  // nothing seen yet: all p = 0
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            p[j][2 * hh + e] = ex2(fmaf(sc[j][2 * hh + e] - mu, a.qscale, kPOff<T>));
                            l[hh] += p[j][2 * hh + e];
                        }
                }
                // O += P V.  P is rounded to the 16-bit type, the operand's of the product:
                // off by half a unit per weight, as the result is once more.  (A second part
                // for the rest would double these products; against 64 bits the error is 2 to 11 %
                // above that of weights in fp32.)  l sums the weights before the rounding.
                if (!slow) {
                    uint32_t pa[4];
                    pa[0] = pack2_out<T>(p[0][0], p[0][1]);
                    pa[1] = pack2_out<T>(p[0][2], p[0][3]);
                    pa[2] = pack2_out<T>(p[1][0], p[1][1]);
                    pa[3] = pack2_out<T>(p[1][2], p[1][3]);
#pragma unroll
                    for (int jj = 0; jj < kNd; ++jj) {
                        uint32_t b[4];
                        ldsm4_t(((stage + v_off) ^ ((jj & 3) << 5)) + (jj >> 2) * kAtom, b);
                        mma16816<T>(o[2 * jj], pa, b[0], b[1]);
                        mma16816<T>(o[2 * jj + 1], pa, b[2], b[3]);
                    }
                } else {
                    const uint8_t* sv = ring + st * (2 * kHalf) + kHalf + warp * (kStep * 128);
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
                __syncwarp();
                if (vb + 1 < vb1 && lane == 0) mbar_arrive(&empty[st]);  // the piece's last stage is the exchange's
            }
            const bool any = vb1 > vb0;  // else nothing is seen: m = -inf, l = 0, and no stage to exchange in
            const int last = (blk + kStages - 1) % kStages;
            float* so = reinterpret_cast<float*>(ring + last * (2 * kHalf));  // [warp][row][D], 8-float groups swizzled by row
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
            users_sync();  // also: every warp is done with the last stage
            if (any) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int row = g + 8 * hh;
                    float mx = s_m[0][row];
#pragma unroll
                    for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][row]);
                    const float f = m[hh] == mx ? 1.0f : ex2((m[hh] - mx) * a.qscale);  // no keys in this warp: 2^-inf = 0
#pragma unroll
                    for (int j = 0; j < 2 * kNd; ++j)
                        *reinterpret_cast<float2*>(so + (warp * kRows + row) * D + ((j ^ (row & 3)) * 8) + 2 * qd) =
                            make_float2(o[j][2 * hh] * f, o[j][2 * hh + 1] * f);
                }
            }
            users_sync();
            const Tile t = s_piece[buf].t;
            const int slot = s_piece[buf].slot;
            for (int e = threadIdx.x; e < t.rows * (D / 4); e += kUsers) {
                const int row = e / (D / 4), d4 = (e % (D / 4)) * 4;
                float mx = s_m[0][row], ls = 0.0f;
#pragma unroll
                for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][row]);
                float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    ls += s_m[w][row] == mx ? s_l[w][row] : s_l[w][row] * ex2((s_m[w][row] - mx) * a.qscale);
                    if (!any) continue;
                    const float4 y = *reinterpret_cast<const float4*>(so + (w * kRows + row) * D + (d4 ^ ((row & 3) << 3)));
                    v.x += y.x;
                    v.y += y.y;
                    v.z += y.z;
                    v.w += y.w;
                }
                if (slot < 0) {
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
            users_sync();          // s_m, s_l, the piece and its queries are free, too
            if (any && lane == 0) mbar_arrive(&empty[last]);
            if (threadIdx.x == 0) mbar_arrive(&piece_empty[buf]);
        }
    }
    if (s_abort) {  // a wait ran out: give this CTA's copies in flight time to land
        const unsigned long long t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
}

// Joins the pieces of the tile in CTA c's record, c = blockIdx.x:
// out = sum_c O_c 2^(m_c - M) / sum_c l_c 2^(m_c - M), kJoinPieces at a time.  A
// tile may have as many pieces as there are CTAs, so the threads that a tile's
// rows leave over share the pieces.  Beside two CTAs of the kernel before it (168
// registers for each of 160 threads; D = 64: 158) an SM has no room for one of these
// (48 registers for each of 256); it enters when one of the two has left and waits
// for the others: 8.4 us by itself, about 4 behind that kernel.
constexpr int kJoinThreads = 256;
constexpr int kJoinPieces = 32;
constexpr int kJoinSplit = 4;  // CTAs per record, each for a quarter of the dims
constexpr int kJoinAhead = 2;  // pieces loaded before their weights are known
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 5) k_paged_join(const __grid_constant__ PagedAttnArgs a) {
    constexpr int kQuads = D / 4 / kJoinSplit;  // groups of four dims per row
    static_assert(kRows * kQuads <= kJoinThreads, "four dims of a row per thread");
    __shared__ float2 s_ml[kJoinPieces][kRows];  // maximum and sum, then the weight
    __shared__ float s_m[kRows], s_l[kRows], s_f[kRows];
    __shared__ float4 s_sum[kJoinThreads];
    pdl_wait();
    pdl_trigger();
    const Join t = part_join<D>(a)[blockIdx.x];
    if (t.pieces == 0) return;
    const int64_t c0 = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int items = t.rows * kQuads, groups = kJoinThreads / items;
    const int e = static_cast<int>(threadIdx.x) % items, grp = static_cast<int>(threadIdx.x) / items;
    const int row = e / kQuads, d4 = (static_cast<int>(blockIdx.y) * kQuads + e % kQuads) * 4;
    float4 v = make_float4(0, 0, 0, 0);
    if (threadIdx.x < kRows) {
        s_m[threadIdx.x] = -INFINITY;
        s_l[threadIdx.x] = 0.0f;
    }
    for (int p0 = 0; p0 < t.pieces; p0 += kJoinPieces) {
        const int np = min(kJoinPieces, t.pieces - p0);
        auto slot_of = [&](int i) { return p0 + i == 0 ? t.slot : 0; };
        // the first pieces' sums are on their way while the weights are found
        float4 y[kJoinAhead];
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            const int i = grp + k * groups;
            if (grp < groups && i < np) y[k] = *reinterpret_cast<const float4*>(part_o<D>(a, c0 + p0 + i, slot_of(i)) + row * D + d4);
        }
        __syncthreads();
        for (int x = threadIdx.x; x < np * kRows; x += kJoinThreads)
            if (x % kRows < t.rows) s_ml[x / kRows][x % kRows] = part_ml<D>(a, c0 + p0 + x / kRows, slot_of(x / kRows))[x % kRows];
        __syncthreads();
        for (int r = warp; r < t.rows; r += kJoinThreads / 32) {
            const float2 ml = lane < np ? s_ml[lane][r] : make_float2(-INFINITY, 0.0f);
            float mx = fmaxf(ml.x, s_m[r]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float w = ml.x == mx ? 1.0f : ex2((ml.x - mx) * a.qscale);
            float l = ml.y * w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (lane < np) s_ml[lane][r].x = w;
            if (lane == 0) {
                const float f = s_m[r] == mx ? 1.0f : ex2((s_m[r] - mx) * a.qscale);
                s_f[r] = f;
                s_l[r] = s_l[r] * f + l;
                s_m[r] = mx;
            }
        }
        __syncthreads();
        if (grp < groups) {
            const float f = s_f[row];
            v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
            auto add = [&](int i, const float4& z) {
                const float w = s_ml[i][row].x;
                v.x = fmaf(z.x, w, v.x);
                v.y = fmaf(z.y, w, v.y);
                v.z = fmaf(z.z, w, v.z);
                v.w = fmaf(z.w, w, v.w);
            };
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k)
                if (grp + k * groups < np) add(grp + k * groups, y[k]);
#pragma unroll 2
            for (int i = grp + kJoinAhead * groups; i < np; i += groups)
                add(i, *reinterpret_cast<const float4*>(part_o<D>(a, c0 + p0 + i, slot_of(i)) + row * D + d4));
        }
    }
    s_sum[threadIdx.x] = v;
    __syncthreads();
    if (grp > 0) return;
    for (int i = 1; i < groups; ++i) {
        const float4 y = s_sum[i * items + e];
        v = make_float4(v.x + y.x, v.y + y.y, v.z + y.z, v.w + y.w);
    }
    const float inv = s_m[row] == -INFINITY ? 0.0f : 1.0f / s_l[row];
    uint2 w2;
    w2.x = pack2_out<T>(v.x * inv, v.y * inv);
    w2.y = pack2_out<T>(v.z * inv, v.w * inv);
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row_offset(a, t.start, t.head, t.row0 + row, a.ld_out) + d4) = w2;
}

template <typename T, int D>
cudaError_t launch_t(PagedAttnArgs a, int num_sms, cudaStream_t st) {
    a.grid = kCtasPerSm * num_sms;
    CUtensorMap tmK, tmV;
    if (!paged_cache_maps(a.c, std::min(a.c.page_size, kBlock), &tmK, &tmV, &a.d_tok, &a.d_head)) return cudaErrorInvalidValue;
    const int ring = 1024 + kRing<D> * 2 * kBlock * D * 2;
    const int pre = (a.B + 1) * 8;
    auto kern = k_paged_attn<T, D>;
    // The limit is the function's, for all host threads: the most that any call
    // takes, since one call's own size could be in force at another's launch.
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ring + (kPagedMaxRequests + 1) * 8);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(a.grid), dim3(kThreads), ring + pre, st, tmK, tmV, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_paged_join<T, D>, dim3(a.grid, kJoinSplit), dim3(kJoinThreads), 0, st, a);
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
