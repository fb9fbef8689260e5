// paged_attn_tc.cu -- attention of chunks of new tokens over a paged key/value
// cache on the tensor cores (tcgen05): what paged_attn.cu computes, for
// requests that bring more rows than one of its tiles holds.
//
//   out = sum_j p_j V[j] / sum_j p_j,   p_j = 2^((s_j - m) scale log2 e)
//
// A unit of work is up to 256 rows -- two tiles of 128 / G tokens with their G
// query heads of one KV head -- against a run of 128-key blocks.  One CTA per
// SM works through its units:
//  * warps 0 and 3 copy (TMA, 128-byte swizzle) the unit's queries and, block by
//    block, K and V through rings of 128-key tiles.  A tile is
//    gathered from its pages, one box of 64 dims x page_size keys per page and
//    half, the page numbers read one block ahead.  Pages that no query of the
//    unit sees are not read: their boxes lie outside the tensor map, which
//    fills them with zeros.
//  * one thread of warp 1 issues the products.  Per block and tile t:
//    O_t += P_t V, then S_t = Q_t K^T of the next block, so that each tile's
//    softmax runs while the tensor pipe works for the other tile.
//  * two warpgroups do the softmax, one per tile, one thread per row (no
//    shuffles): S_t from tensor memory, mask, maximum, weights, sum; P_t goes
//    back in 16 bits, over S_t's first 64 columns or (D = 64) beside, and is the
//    product's operand from there.  O_t stays in tensor memory.
//    The maximum is a reference, not the exact one: it moves (and O_t and the
//    sum are rescaled) only when a row's maximum has grown by a factor of 2^8
//    or more, which after the first blocks hardly happens.  Weights then reach
//    2^8 times 2^kOff at most, and the fp32 sums lose nothing by it.
//  * Slots behind the request's end, which may hold anything, become zeros in
//    shared memory before the product that would multiply V there by zero
//    weights.  Other rows of V are tokens' values: finite, as a rule.  If one that
//    some query does not see is not, 0 x V makes that query's output NaN; a row
//    whose output is not finite although its weights' sum is gets computed again
//    by its warp (redo_row), from the keys that it sees alone.  So is a row with scores
//    of 2^16 or more (scaled, in base two).
//
// What bounds it: per 128 x 128 block of scores the two products take 1024
// cycles of the tensor pipe at D = 128 (8192 fp16 operations per cycle and SM),
// and the 16384 exponentials 1024 cycles of the special-function units (16 per
// cycle and SM).  Both tiles' block takes 3430 to 3560 cycles (D = 64: 3280) and
// not 2048: a tile's scores, weights and products follow one another, and the two
// tiles do not fill all the gaps; both pipes are at 57 %.  (A third tile does not fit
// in tensor memory; two warps per 32 rows, which halves the softmax's length, gained
// nothing.)
// Measured, 32 / 8 heads, D = 128, calls back to back: a prompt of 2048 48 us, four
// chunks of 500 tokens over up to 16K keys 260 us (985 TFLOP/s), 4096 tokens over 16K
// 890 to 925 us (1040 to 1080; the board's power limit lowers the clock); 2 x 2048
// tokens with a window of 1024, 32 / 4 heads, D = 64: 99 to 115 us.
//
// The work list is made by a one-CTA kernel that reads the lengths on the
// device: it lists the units longest first (each CTA takes them in snake
// order, so the SMs finish together) and, when they are too few for the SMs,
// cuts their key blocks into pieces whose fp32 results another kernel joins.
// Every wait is bounded (tile_wait).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "gemm_common.cuh"
#include "paged_common.cuh"

namespace cider {
namespace {

constexpr int kKeys = 128;                     // keys per block
constexpr int kTcThreads = 384;                // warps 0-3: TMA, MMA, idle, TMA; then a softmax warpgroup per tile
constexpr int kPlanThreads = 256;  // fewer threads, cheaper barriers: a prompt of 2048 52.8 us with 1024, 48.9 with 256
constexpr int kMaxGrid = 256;                  // CTAs of the tile kernel: one per SM
static_assert(kPlanThreads >= kMaxGrid, "the planner has a thread per CTA");
constexpr int kMaxCut = 2560;                  // units up to which they may be cut
constexpr int kUnitCost = 2;                   // the start and end of a unit, in blocks
constexpr int kMinShare = 2 + kUnitCost;       // length per CTA where the line is cut
constexpr float kLazy = 8.0f;                  // log2 of the growth of a maximum that is put off
// The exponents are s q - m q (q the scale, in base two), one operation per score; below this
// |m q| the rounding of m q, which is the same for all keys until m moves, is 2^-9 at
// most.  Rows beyond it are computed again with (s - m) q.
constexpr float kFar = 65536.0f;

// One unit: tokens [token0, token0 + ntok) of q's rows, the first at position
// pmin, against blocks [vb0, vb0 + nblk) of its span; slot -1: the whole span.
struct __align__(16) TcUnit {
    int b, token0, ntok, pmin, vb0, nblk, slot, head;  // head: where the list is cut
    int len, pad[3];  // the request's keys
};
// A unit of several pieces: the first in `slot`, the others in slot 2 c of the
// CTAs c behind cta.
struct TcJoin {
    int token0, ntok, head, slot, cta, pieces;
};
struct TcPlan {
    int units, cut, joins;  // whole: records, each for H_kv heads
};

struct TcArgs {
    PagedAttnArgs p;
    int tok;              // tokens per 128-row tile: 128 / G
    int max_tiles;        // records that the workspace holds: enough for offsets that do not decrease
    int boxes;            // pages per block (at least 1)
    int box_keys;         // keys per box: min(page_size, 128)
    int grid;
    TcPlan* plan;
    TcUnit* units;
    TcJoin* joins;
    int2* ranges;         // cut: each CTA's first record and their number
    float* part;          // [slot][256][D], then [slot][256] maximum and sum
    int slots;
    int wide;             // out's rows begin at 32-byte boundaries
    int64_t l2_keys;      // keys whose K and V (all heads) fill 3/5 of the L2
};

__device__ __forceinline__ float ex2(float x) {  // 2^x, PTX ex2.approx (relative error near 2^-22)
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Weights are made as 2^(x + kOff).  fp16: 2^7, with the lazy maximum up to
// 2^15 < 65504, so weights down to 2^-21 of the reference keep all 11 bits;
// bf16 has the range of fp32.  The factor cancels in O / l.
template <typename T>
constexpr float kOff = std::is_same<T, __half>::value ? 7.0f : 0.0f;

// ---- the work list ------------------------------------------------------------

// Blocks that the queries [pmin, pmin + ntok) read.
__device__ __forceinline__ int span_blocks(const PagedAttnArgs& a, int pmin, int ntok) {
    PagedSpan<kKeys> s;
    s.set(pmin, pmin + ntok - 1, a.window, a.sinks);
    return s.blocks;
}

// Two ways to share the units out.  Whole: the list is sorted, longest first,
// and each CTA takes its units in snake order.  Cut: the units form one line, in
// order, each as long as its blocks and kUnitCost (half in front, half behind), of
// which each CTA takes an equal share; a unit that several share leaves fp32 partial
// results, at most two per CTA, for the join.  (With the blocks alone the CTA with
// the first, short tiles of a prompt got many of them: 4096 tokens, 8 / 2 heads, 79
// us; now 58, and whole units 73.)  The cheaper one is taken, in blocks: whole, the
// longest CTA; cut, the share, the start and end of a unit once more per CTA, and
// eight for writing and joining the partial results.  With units for every SM the cut
// also needs the keys and values to stay in the L2: whole units of the same
// head walk through its keys together and read them from HBM once, the cut ones
// start all over the place (four chunks of 500 over 268 MB of keys and values:
// 278 us whole, 305 us cut; 4096 tokens over 67 MB: 940 us whole, 917 us cut).
__global__ void __launch_bounds__(kPlanThreads) k_paged_plan(TcArgs t) {
    extern __shared__ int32_t pre[];  // [B + 1] tiles before each request, then [B] of each request's row, tokens and keys
    __shared__ int64_t s_warp[kPlanThreads / 32];
    __shared__ int s_hist[kPlanThreads], s_sorted[kMaxCut];
    __shared__ int s_first[kMaxGrid], s_last[kMaxGrid];
    __shared__ int s_max, s_joins;
    __shared__ unsigned long long s_keys;
    const PagedAttnArgs& a = t.p;
    const int per_unit = 2 * t.tok, tid = threadIdx.x, lane = tid & 31;
    int32_t* start = pre + a.B + 1;
    int32_t* fresh = start + a.B;
    int32_t* keys = fresh + a.B;
    pdl_wait();
    pdl_trigger();
    s_hist[tid] = 0;
    if (tid == 0) {
        s_max = s_joins = 0;
        s_keys = 0;
    }
    if (tid < kMaxGrid) {
        s_first[tid] = INT_MAX;
        s_last[tid] = -1;
    }
    const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int sum = 0;
    int64_t len = 0;
    bool any_bad = false;
    for (int b = b0; b < b1; ++b) {
        bool bad;
        const PagedRequest r = paged_request(a, b, &bad);
        any_bad |= bad;
        len += r.n > 0 ? r.L : 0;
        pre[b] = sum;
        start[b] = r.start;
        fresh[b] = r.n;
        keys[b] = r.L;
        sum += (r.n + per_unit - 1) / per_unit;
    }
    if (any_bad) atomicOr(a.status, kStatusIndex);
    int64_t total;
    const int64_t base = block_prefix<kPlanThreads>(sum, s_warp, &total);
    for (int b = b0; b < b1; ++b) pre[b] = static_cast<int>(min(pre[b] + base, static_cast<int64_t>(INT_MAX)));
    if (tid == 0) pre[a.B] = static_cast<int>(min(total, static_cast<int64_t>(INT_MAX)));
    __syncthreads();
    // Offsets that decrease can give the same rows to many requests; the list has
    // room for each row once, and ends there.
    const int tiles = static_cast<int>(min(total, static_cast<int64_t>(t.max_tiles)));
    auto unit = [&](int i) {
        TcUnit u;
        u.b = find_request(pre, a.B, i);
        const int first = (i - pre[u.b]) * per_unit;
        u.token0 = start[u.b] + first;
        u.ntok = min(per_unit, fresh[u.b] - first);
        u.pmin = keys[u.b] - fresh[u.b] + first;
        u.vb0 = 0;
        u.nblk = span_blocks(a, u.pmin, u.ntok);
        u.slot = -1;
        u.head = 0;
        u.len = keys[u.b];
        u.pad[0] = u.pad[1] = u.pad[2] = 0;
        return u;
    };
    // this thread's tiles, in order, and the blocks before them
    const int each = (tiles + kPlanThreads - 1) / kPlanThreads;
    const int i0 = min(tiles, tid * each), i1 = min(tiles, i0 + each);
    int mx = 0;
    int64_t blocks = 0;
    for (int i = i0; i < i1; ++i) {
        const int n = unit(i).nblk;
        mx = max(mx, n);
        blocks += n + kUnitCost;
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (lane == 0) atomicMax(&s_max, mx);
    if (len) atomicAdd(&s_keys, static_cast<unsigned long long>(len));
    int64_t work;
    int64_t before = block_prefix<kPlanThreads>(blocks, s_warp, &work);
    mx = s_max;
    // whole: places by counting per class of length
    const float scale = (kPlanThreads - 1.0f) / max(1, mx);
    auto bin = [&](int n) { return kPlanThreads - 1 - min(kPlanThreads - 1, static_cast<int>(n * scale)); };
    // A class's length (rounded up; where a class holds one length, that).  The units of
    // a class come in any order, and what is chosen below may not depend on it.
    auto length = [&](int bin) { return ((kPlanThreads - 1 - bin) * mx + kPlanThreads - 2) / (kPlanThreads - 1); };
    for (int i = i0; i < i1; ++i) atomicAdd(&s_hist[bin(unit(i).nblk)], 1);
    __syncthreads();
    const int64_t place = block_prefix<kPlanThreads>(s_hist[tid], s_warp, &total);
    s_hist[tid] = static_cast<int>(place);
    __syncthreads();
    const int64_t units = static_cast<int64_t>(tiles) * a.c.H_kv;
    const bool may_cut = units <= kMaxCut;  // beyond, the rounds are many and even out
    for (int i = i0; i < i1; ++i) {
        const TcUnit u = unit(i);
        const int at = atomicAdd(&s_hist[bin(u.nblk)], 1);
        t.units[at] = u;
        if (may_cut) s_sorted[at] = length(bin(u.nblk));
    }
    __syncthreads();
    work *= a.c.H_kv;
    const int64_t share = max(static_cast<int64_t>(kMinShare), (work + t.grid - 1) / t.grid);
    bool cut = false;
    if (may_cut) {
        int load = 0;
        if (tid < t.grid)
            for (int r = 0; r * t.grid < units; ++r) {
                const int x = r * t.grid + ((r & 1) ? t.grid - 1 - tid : tid);
                if (x < units) load += s_sorted[x / a.c.H_kv] + kUnitCost;
            }
        load = __reduce_max_sync(0xffffffffu, load);
        __syncthreads();
        if (tid == 0) s_max = 0;
        __syncthreads();
        if (lane == 0) atomicMax(&s_max, load);
        __syncthreads();
        cut = share + kUnitCost + 8 < s_max &&
              (units < t.grid || static_cast<int64_t>(s_keys) <= t.l2_keys);
    }
    if (cut) {
        // Record j + c is unit j's piece in CTA c's share (so a CTA's records are
        // next to one another); a unit without blocks has one all the same.
        for (int i = i0; i < i1; ++i) {
            TcUnit u = unit(i);
            const int n = u.nblk;
            const int w = n + kUnitCost;
            auto block_at = [&](int64_t y) { return static_cast<int>(min(max(y - kUnitCost / 2, int64_t(0)), static_cast<int64_t>(n))); };
            for (int head = 0; head < a.c.H_kv; ++head) {
                const int64_t x0 = before * a.c.H_kv + static_cast<int64_t>(head) * w, x1 = x0 + w;
                const int j = i * a.c.H_kv + head;
                int c0 = static_cast<int>(x0 / share), c1 = n > 0 ? static_cast<int>((x1 - 1) / share) : c0;
                bool at_start = x0 == c0 * share;  // of c0's share
                if (n > 0 && block_at((c0 + 1) * share - x0) == 0) {  // nothing but the front
                    ++c0;
                    at_start = true;
                }
                if (c1 > c0 && block_at(c1 * share - x0) == n) --c1;  // nothing but what is behind
                u.head = head;
                const int slot0 = 2 * c0 + (at_start ? 0 : 1);
                for (int c = c0; c <= c1; ++c) {
                    u.vb0 = block_at(c == c0 ? 0 : c * share - x0);
                    u.nblk = block_at(c == c1 ? w : (c + 1) * share - x0) - u.vb0;
                    u.slot = c1 == c0 ? -1 : c == c0 ? slot0 : 2 * c;
                    t.units[j + c] = u;
                    atomicMin(&s_first[c], j + c);
                    atomicMax(&s_last[c], j + c);
                }
                if (c1 > c0) t.joins[atomicAdd(&s_joins, 1)] = TcJoin{u.token0, u.ntok, head, slot0, c0, c1 - c0 + 1};
            }
            before += w;
        }
        __syncthreads();
        if (tid < t.grid) t.ranges[tid] = make_int2(s_first[tid], s_last[tid] < 0 ? 0 : s_last[tid] - s_first[tid] + 1);
    }
    if (tid == 0) *t.plan = TcPlan{tiles, cut ? 1 : 0, s_joins};
}

// ---- tensor-core pieces ---------------------------------------------------------

// Shared-memory operand descriptors, 128-byte swizzle, as two words: the low
// one is the start address and the leading byte offset (both >> 4), the high
// one the stride between 8-row groups (1024 bytes), the version and the layout,
// which are constants here.  K-major: rows of 64 K elements; the leading offset
// is not used.  MN-major: rows of 64 MN elements, the leading offset between
// 64-element atoms along MN.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return ((addr >> 4) & 0x3FFFu) | (lbo >> 4) << 16; }

// kind::f16 instruction descriptor: D = F32, A = B = fp16 (bf = 0) or bf16 (bf
// = 1); b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_16(int M, int N, int bf, int b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(bf) << 7) | (static_cast<uint32_t>(bf) << 10) |
           (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %5};\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi)
        : "memory");
}
// A from tensor memory: row = lane, two 16-bit values of K per column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi)
        : "memory");
}
// The waits of this kernel.  Their limit is longer than elsewhere, because a warp
// in redo_row keeps the others waiting: 20 s, some ten million keys of a unit.
constexpr unsigned long long kTileWaitNs = 20000000000ull;
__device__ __forceinline__ bool tile_wait(uint64_t* bar, uint32_t parity, unsigned* status, volatile int* abort_flag) {
    return mbar_wait_for(bar, parity, status, abort_flag, kTileWaitNs);
}

__device__ __forceinline__ bool elect_one() {
    uint32_t x;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
    return x != 0;
}

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
// Waits for the loads so far; r is given, so that no use of it moves in front.
__device__ __forceinline__ void ld_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i])::"memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {  // NaN if any is
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// Barrier of the 128 threads of softmax warpgroup wg; true if any passes x.
__device__ __forceinline__ bool group_or(int wg, bool x) {
    uint32_t y;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, %2, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(y)
        : "r"(static_cast<uint32_t>(x)), "r"(1 + wg)
        : "memory");
    return y != 0;
}

// 32 bytes to a 32-byte boundary: a thread writes whole sectors of its row, where
// two 16-byte stores would take the warp twice as many passes over its 32 rows.
__device__ __forceinline__ void store32(void* p, const uint32_t* r) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

template <int D>
__device__ __forceinline__ float* part_row(const TcArgs& t, int slot, int row) {
    return t.part + (static_cast<int64_t>(slot) * 256 + row) * D;
}
template <int D>
__device__ __forceinline__ float2* part_ml(const TcArgs& t, int slot, int row) {
    return reinterpret_cast<float2*>(t.part + static_cast<int64_t>(t.slots) * 256 * D) + static_cast<int64_t>(slot) * 256 + row;
}

// One row of a unit on the CUDA cores, by one warp: each lane has D / 32 dims, 16
// keys (of one page) at a time, and only keys that the row sees reach the result.
// Rare (see the top of the file).  It keeps to few registers, which the tile
// kernel around it would otherwise spill.  A warp whose 32 rows all need it takes
// 1 to 2 us per key of the unit (a prompt of 2048 with NaN everywhere: 4 ms).
template <typename T, int D>
__device__ __noinline__ void redo_row(const TcArgs& t, TcUnit u, int row) {
    constexpr int E = D / 32, N = 16;
    using Vec = std::conditional_t<E == 4, uint2, uint32_t>;
    const PagedAttnArgs& a = t.p;
    const int lane = threadIdx.x & 31;
    const int tok = (row >> 7) * t.tok + (row & 127) / a.G, pos = u.pmin + tok;
    const int64_t q_row = u.token0 + tok, col = static_cast<int64_t>(u.head * a.G + (row & 127) % a.G) * D + lane * E;
    PagedSpan<kKeys> span;
    span.set(u.pmin, u.pmin + u.ntok - 1, a.window, a.sinks);
    const int32_t* table = a.table + u.b * a.ld_table;
    const T* kh = reinterpret_cast<const T*>(a.c.k) + u.head * a.c.sh + lane * E;
    const T* vh = reinterpret_cast<const T*>(a.c.v) + u.head * a.c.sh + lane * E;
    auto load = [](const T* p) { return __ldg(reinterpret_cast<const Vec*>(p)); };
    float q[E], o[E], m = -INFINITY, l = 0.0f;
    const Vec qv = load(static_cast<const T*>(a.q) + q_row * a.ld_q + col);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = to_f32<T>(reinterpret_cast<const T*>(&qv)[e]);
        o[e] = 0.0f;
    }
    for (int vb = u.vb0; vb < u.vb0 + u.nblk; ++vb) {
        const int block = span.block(vb) * kKeys;
        for (int key0 = block; key0 < block + kKeys && key0 <= pos; key0 += N) {  // pages hold 16 keys or more
            const int page = __ldg(table + (key0 >> a.c.ps_log2));
            if (page < 0 || page >= a.c.num_pages) continue;
            const int64_t off = page * a.c.sp + (key0 & (a.c.page_size - 1)) * a.c.st;
            Vec k[N], v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) k[i] = load(kh + off + i * a.c.st);
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = load(vh + off + i * a.c.st);
            float s[N], mn = m;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                s[i] = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) s[i] = fmaf(q[e], to_f32<T>(reinterpret_cast<const T*>(&k[i])[e]), s[i]);
#pragma unroll
                for (int w = 16; w > 0; w >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], w);
                if (paged_sees(key0 + i, pos, a.window, a.sinks)) mn = fmaxf(fmaxf(mn, s[i]), -FLT_MAX);
            }
            const float f = mn == m ? 1.0f : ex2((m - mn) * a.qscale);
            m = mn;
            l *= f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (!paged_sees(key0 + i, pos, a.window, a.sinks)) continue;
                const float p = ex2(fmaf(s[i] - mn, a.qscale, kOff<T>));
                l += p;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(p, to_f32<T>(reinterpret_cast<const T*>(&v[i])[e]), o[e]);
            }
        }
    }
    if (u.slot >= 0) {
        float* part = part_row<D>(t, u.slot, row) + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) part[e] = o[e];
        if (lane == 0) *part_ml<D>(t, u.slot, row) = make_float2(m, l);
    } else {
        const float inv = m == -INFINITY ? 0.0f : 1.0f / l;
        T* out = static_cast<T*>(a.out) + q_row * a.ld_out + col;
#pragma unroll
        for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(out + e) = pack2<T>(o[e] * inv, o[e + 1] * inv);
    }
}

template <int D>
constexpr int kTileBytes = kKeys * D * 2;  // one K or V tile; one tile of queries is the same
// The rings' tiles of keys and of values.  A block's keys are done with when its
// scores are made, its values a block later.
template <int D>
constexpr int kKStages = D == 128 ? 2 : 4;
template <int D>
constexpr int kVStages = D == 128 ? 3 : 4;
constexpr int kTmemCols = 512;
// Whether P has columns of its own (S 2 x 128, O 2 x D, P 2 x 64).  Then the next
// block's scores are made as soon as the last one's have been read, and a tile's
// softmax waits for no product; where P lies over S, they wait for the product
// that reads it.
template <int D>
constexpr bool kApart = D == 64;

template <typename T, int D>
__global__ void __launch_bounds__(kTcThreads, 1) k_paged_tc(const __grid_constant__ CUtensorMap tmQ,
                                                            const __grid_constant__ CUtensorMap tmK,
                                                            const __grid_constant__ CUtensorMap tmV,
                                                            const __grid_constant__ TcArgs t) {
    constexpr int BF = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
    constexpr int KS = kKStages<D>, VS = kVStages<D>;
    constexpr int TB = kTileBytes<D>;
    constexpr int AB = kKeys * 128;  // one 64-dim atom of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;               // two tiles of queries
    uint8_t* sK = smem + 2 * TB;      // KS tiles of keys
    uint8_t* sV = sK + KS * TB;       // VS tiles of values
    __shared__ uint64_t qfull, qempty, kfull[KS], kempty[KS], vfull[VS], vempty[VS], sfull[2], pfull[2][2], sfree[2], odone[2][2], turn[4][2], ufull[2], uempty[2];
    __shared__ TcUnit s_unit[2];    // the units, one after the other, from the loading warp; nblk < 0: no more
    __shared__ uint32_t s_lost[8];  // of the last 8 blocks: a bit per box whose page is missing;
    __shared__ uint32_t tmem_slot;
    __shared__ int s_abort;
    volatile int* abort_flag = &s_abort;
    const PagedAttnArgs& a = t.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        s_abort = 0;
        mbar_init(&qfull, 1);
        mbar_init(&qempty, 2);
        for (int s = 0; s < KS; ++s) {
            mbar_init(&kfull[s], 1);
            mbar_init(&kempty[s], 2);  // each tile's products
        }
        for (int s = 0; s < VS; ++s) {
            mbar_init(&vfull[s], 1);
            mbar_init(&vempty[s], kApart<D> ? 1 : 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i][0], 4);  // one arrival per warp
            mbar_init(&pfull[i][1], 4);
            mbar_init(&sfree[i], 4);
            for (int w = 0; w < 4; ++w) mbar_init(&turn[w][i], 1);
            mbar_init(&odone[i][0], 1);
            mbar_init(&odone[i][1], 1);
            mbar_init(&ufull[i], 1);
            mbar_init(&uempty[i], 4);  // the values' loader, the issuer and the softmax of each tile
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) tmem_alloc(&tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();
    pdl_trigger();
    unsigned* status = a.status;
    const bool cut = t.plan->cut;
    const int nunits = t.plan->units * a.c.H_kv;
    const int2 range = cut ? t.ranges[blockIdx.x] : make_int2(0, 0);
    const int rounds = cut ? range.y : (nunits + t.grid - 1) / t.grid;
    // this CTA's unit of round r; false: it has none
    auto fetch = [&](int r, TcUnit& u) {
        if (cut) {
            u = t.units[range.x + r];
            return true;
        }
        const int i = static_cast<int>(blockIdx.x);
        const int x = r * t.grid + ((r & 1) ? t.grid - 1 - i : i);
        if (x >= nunits) return false;
        u = t.units[x / a.c.H_kv];
        u.head = x % a.c.H_kv;
        return true;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (warp == 0 || warp == 3) {
            // ------------------------------ TMA producers -----------------------------
            // Warp 0 loads queries and keys, warp 3 values: a lane's copy takes some
            // 100 cycles to issue, and a block of 16-key pages has 32 of them.
            const bool keys = warp == 0;
            int blk = 0, nq = 0;  // blocks and units with queries so far
            bool ok = true;
            for (int n = 0, r = 0; ok; ++n) {
                TcUnit u{};
                if (keys) {  // posts the units to the other warps
                    while (r < rounds && !fetch(r, u)) ++r;
                    if (r++ >= rounds) u.nblk = -1;
                    ok = tile_wait(&uempty[n & 1], ((n >> 1) & 1) ^ 1, status, abort_flag);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    if (lane == 0) {
                        s_unit[n & 1] = u;
                        mbar_arrive(&ufull[n & 1]);
                    }
                } else {
                    ok = tile_wait(&ufull[n & 1], (n >> 1) & 1, status, abort_flag);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    u = s_unit[n & 1];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&uempty[n & 1]);
                }
                if (u.nblk < 0) break;
                PagedSpan<kKeys> span;
                span.set(u.pmin, u.pmin + u.ntok - 1, a.window, a.sinks);
                const int32_t* table = a.table + u.b * a.ld_table;
                // page of this lane's box of block vb; num_pages (outside the map:
                // zeros) where no query sees any of its keys, or the page is bad
                bool missing = false;
                auto page_of = [&](int vb) {
                    int page = a.c.num_pages;
                    missing = false;
                    if (lane < t.boxes && vb < u.vb0 + u.nblk) {
                        const int key0 = span.block(vb) * kKeys + lane * t.box_keys;
                        const bool used = key0 <= span.pmax && (a.window <= 0 || key0 + t.box_keys - 1 > span.pmin - a.window || key0 < a.sinks);
                        if (used) {
                            const int p = __ldg(table + (key0 >> a.c.ps_log2));
                            if (p >= 0 && p < a.c.num_pages)
                                page = p;
                            else
                                missing = true;
                        }
                    }
                    if (missing) atomicOr(status, kStatusIndex);
                    return page;
                };
                const CUtensorMap* map = keys ? &tmK : &tmV;
                // one box per page and 64-dim half, a lane each
                const int box = lane % t.boxes, half = lane / t.boxes;
                int next = page_of(u.vb0);
                for (int i = 0; i < u.nblk && ok; ++i, ++blk) {
                    const int page = __shfl_sync(0xffffffffu, next, box);
                    const uint32_t lost = __ballot_sync(0xffffffffu, missing);
                    next = page_of(u.vb0 + i + 1);
                    const int st = keys ? blk % KS : blk % VS, ph = (keys ? blk / KS : blk / VS) & 1;
                    uint64_t* full = keys ? &kfull[st] : &vfull[st];
                    ok = tile_wait(keys ? &kempty[st] : &vempty[st], ph ^ 1, status, abort_flag);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    if (lane == 0) {
                        if (keys) s_lost[blk & 7] = lost;
                        mbar_arrive_expect_tx(full, TB);
                    }
                    __syncwarp();
                    if (half < D / 64) {
                        int c[4] = {half * 64, page, page, page};
#pragma unroll
                        for (int d = 1; d < 4; ++d) {
                            if (d == a.d_tok) c[d] = (span.block(u.vb0 + i) * kKeys) & (a.c.page_size - 1);  // pages of 256: 0 or 128
                            if (d == a.d_head) c[d] = u.head;
                        }
                        tma_load_4d((keys ? sK : sV) + st * TB + half * AB + box * t.box_keys * 128, map, full, c[0], c[1], c[2], c[3]);
                    }
                    __syncwarp();
                    if (keys && i == 0) {  // the queries, once the last unit's products are done with theirs
                        ok = tile_wait(&qempty, (nq & 1) ^ 1, status, abort_flag);
                        ok = __all_sync(0xffffffffu, ok);
                        const int tiles = u.ntok > t.tok ? 2 : 1;
                        const int bytes = t.tok * a.G * 128;
                        if (ok && lane == 0) {
                            mbar_arrive_expect_tx(&qfull, tiles * (D / 64) * bytes);
                            for (int h = 0; h < tiles; ++h)
                                for (int d = 0; d < D / 64; ++d)
                                    tma_load_3d(sQ + h * TB + d * AB, &tmQ, &qfull, d * 64, u.head * a.G, u.token0 + h * t.tok);
                        }
                        __syncwarp();
                        ++nq;
                    }
                }
            }
        } else if (warp == 1) {
            // ------------------------------ MMA issuer --------------------------------
            // The whole warp runs the loop, so that addresses stay in uniform
            // registers; one lane issues.
            constexpr uint32_t idesc_s = idesc_16(128, kKeys, BF, 0);
            constexpr uint32_t idesc_o = idesc_16(128, D, BF, 1);
            const uint32_t q_lo = desc_lo(smem_u32(sQ), 0), k_lo = desc_lo(smem_u32(sK), 0), v_lo = desc_lo(smem_u32(sV), AB);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const bool leader = elect_one();
            int gb = 0, nq = 0, blk[2] = {0, 0};  // the rings' blocks and units so far, and the blocks of each tile
            bool ok = true;
            for (int n = 0; ok; ++n) {
                ok = tile_wait(&ufull[n & 1], (n >> 1) & 1, status, abort_flag);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const int nblk = s_unit[n & 1].nblk, tiles = s_unit[n & 1].ntok > t.tok ? 2 : 1;
                __syncwarp();
                if (lane == 0) mbar_arrive(&uempty[n & 1]);
                if (nblk < 0) break;
                if (nblk == 0) continue;
                auto scores = [&](int h, int s) {  // S_h = Q_h K^T
                    if (leader) {
                        const uint32_t a0 = q_lo + h * (TB >> 4), b0 = k_lo + s * (TB >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * AB + (kk & 3) * 32) >> 4;
                            mma_ss(tm + h * 128, a0 + off, b0 + off, idesc_s, kk > 0);
                        }
                        umma_commit(&sfull[h]);
                    }
                };
                ok = tile_wait(&kfull[gb % KS], (gb / KS) & 1, status, abort_flag) && tile_wait(&qfull, nq & 1, status, abort_flag);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
                // O_h (+)= P_h V of 64 keys, V in stage sv
                auto values = [&](int h, int half, int sv, bool first) {
                    if (leader) {
                        const uint32_t v0 = v_lo + sv * (TB >> 4), p0 = kApart<D> ? 384 + h * 64 : h * 128;
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4) {  // 16 keys: 8 columns of P, 2 KB of each atom of V
                            const int kk = half * 4 + k4;
                            mma_ts(tm + 256 + h * D, tm + p0 + kk * 8, v0 + (kk * 2048 >> 4), idesc_o, !first || k4 > 0);
                        }
                    }
                };
                for (int h = 0; h < tiles && ok; ++h) {
                    if (kApart<D> && blk[h] > 0) {
                        ok = tile_wait(&sfree[h], (blk[h] - 1) & 1, status, abort_flag);
                        ok = __all_sync(0xffffffffu, ok);
                        tc_fence_after();
                    }
                    if (ok) scores(h, gb % KS);
                }
                ++nq;
                for (int i = 0; i < nblk && ok; ++i, ++gb) {
                    const int sv = gb % VS, sk = (gb + 1) % KS;
                    const bool more = i + 1 < nblk;
                    if (kApart<D> && more) {  // the next scores first: they need only the last ones read
                        ok = tile_wait(&kfull[sk], ((gb + 1) / KS) & 1, status, abort_flag);
                        for (int h = 0; h < tiles; ++h) {
                            ok = ok && tile_wait(&sfree[h], blk[h] & 1, status, abort_flag);
                            ok = __all_sync(0xffffffffu, ok);
                            tc_fence_after();
                            if (ok) scores(h, sk);
                        }
                    }
                    for (int h = 0; h < tiles; ++h) {
                        if (h == 0) ok = ok && tile_wait(&vfull[sv], (gb / VS) & 1, status, abort_flag);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            ok = ok && tile_wait(&pfull[h][half], blk[h] & 1, status, abort_flag);
                            ok = __all_sync(0xffffffffu, ok);
                            tc_fence_after();
                            if (ok) values(h, half, sv, i == 0 && half == 0);
                        }
                        if (!ok) break;
                        if (leader && (kApart<D> || !more)) umma_commit(&odone[h][kApart<D> ? blk[h] & 1 : 0]);
                        ++blk[h];
                        if (!kApart<D> && more) {
                            if (h == 0) {
                                ok = tile_wait(&kfull[sk], ((gb + 1) / KS) & 1, status, abort_flag);
                                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                                tc_fence_after();
                            }
                            scores(h, sk);
                        }
                    }
                    if (ok && kApart<D> && leader) umma_commit(&vempty[sv]);
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------ softmax and output ----------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int h = (warp - 4) >> 2;  // this warpgroup's tile
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_addr + h * 128, tO = tmem + lane_addr + 256 + h * D;
        const uint32_t tP = kApart<D> ? tmem + lane_addr + 384 + h * 64 : tS;
        int nb = 0, nu = 0;  // blocks and units of this tile so far
        uint32_t turns = 0;  // of this warp at the exponentials
        int gb = 0;    // the rings' blocks before this unit
        bool ok = true;
        for (int n = 0;; ++n) {
            if (ok) ok = tile_wait(&ufull[n & 1], (n >> 1) & 1, status, abort_flag);
            const TcUnit u = s_unit[n & 1];
            if (group_or(h, !ok || u.nblk < 0)) break;  // the group's warps go on, or end, together (and have read it)
            if (row == 0) mbar_arrive(&uempty[n & 1]);
            const int head = u.head;
            const int tok0 = h * t.tok, ntok = min(t.tok, u.ntok - tok0);  // this tile's tokens
            if (ntok <= 0) {
                gb += u.nblk;
                continue;
            }
            PagedSpan<kKeys> span;
            span.set(u.pmin, u.pmin + u.ntok - 1, a.window, a.sinks);
            const int pmin = u.pmin + tok0, pmax = pmin + ntok - 1;
            const int tok = row / a.G;
            const int pos = pmin + tok;
            const bool live = tok < ntok && row < t.tok * a.G;
            float m = -INFINITY, l = 0.0f;
            // One thread tells the producer what this tile's products are done with
            // (and for the second tile, where the unit has none).
            const int frees = row != 0 ? 0 : u.ntok > t.tok ? 1 : 2;
            // Where no product keeps the tiles apart in time, the two warps that share a
            // scheduler take turns at the exponentials: at the same time each would take
            // twice as long, and then leave the special-function unit idle together.
            const bool paired = kApart<D> && u.ntok > t.tok && u.nblk > 0;
            uint64_t* my_turn = &turn[warp & 3][h];
            uint64_t* other_turn = &turn[warp & 3][h ^ 1];
            if (paired && h == 1 && lane == 0) mbar_arrive(other_turn);
            for (int i = 0; i < u.nblk; ++i, ++nb) {
                const int key0 = span.block(u.vb0 + i) * kKeys;
                ok = tile_wait(&sfull[h], nb & 1, status, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int e = 0; e < frees; ++e) {  // QK^T of this block and PV of the last one are done
                    mbar_arrive(&kempty[(gb + i) % KS]);
                    if (!kApart<D> && i > 0) mbar_arrive(&vempty[(gb + i - 1) % VS]);
                    if (i + 1 == u.nblk) mbar_arrive(&qempty);
                }
                __syncwarp();  // the loads from tensor memory are the whole warp's; so below, behind one lane's arrivals
                float low = -FLT_MAX;  // a row that has seen a key has a finite maximum: this mark, if its scores were all -inf
                const uint32_t lost = s_lost[(gb + i) & 7];
                const bool whole = !lost && key0 + kKeys - 1 <= pmin &&
                                   (a.window <= 0 || key0 > pmax - a.window || key0 + kKeys <= a.sinks);
                if (!whole) {
                    if (key0 + kKeys > u.len) {  // slots behind the request's end: V becomes zeros there
                        const int s = (gb + i) % VS;
                        ok = tile_wait(&vfull[s], ((gb + i) / VS) & 1, status, abort_flag);
                        if (!__all_sync(0xffffffffu, ok)) {
                            ok = false;
                            break;
                        }
                        for (int e = row; e < kKeys * (D / 8); e += 128)
                            if (key0 + ((e >> 3) & (kKeys - 1)) >= u.len) reinterpret_cast<uint4*>(sV + s * TB)[e] = make_uint4(0, 0, 0, 0);
                        fence_async_smem();
                    }
                    // S: -inf where the row does not see the key, 32 columns at a time
                    // and back to tensor memory, so that the registers hold the 128
                    // scores only once (a spill goes to L2: shared memory leaves no L1).
                    // Columns that all rows of the warp see stay as they are, and those
                    // that none sees are not read: of a block on the diagonal or at a
                    // window's start three of the four chunks are one or the other.
                    const int last = pos - key0;                                             // seen: x <= last
                    const int first = a.window > 0 ? max(pos - a.window, -1) - key0 : -1;    // and x > first
                    const int sink = a.window > 0 ? max(min(a.sinks - key0, kKeys), 0) : 0;  // or x < sink
                    uint32_t any = 0;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        const int lo = c * 32;
                        const uint32_t below = last - lo >= 31 ? ~0u : last < lo ? 0u : (2u << (last - lo)) - 1;
                        const uint32_t after = first < lo ? ~0u : first - lo >= 31 ? 0u : ~((2u << (first - lo)) - 1);
                        const uint32_t sinks = sink <= lo ? 0u : sink - lo >= 32 ? ~0u : (1u << (sink - lo)) - 1;
                        uint32_t see = below & (after | sinks);  // the row's seen columns as bits
                        if (lost)
                            for (int e = 0; e < 32; e += 16)  // pages hold 16 keys or more
                                if ((lost >> ((lo + e) / t.box_keys)) & 1u) see &= ~(0xffffu << e);
                        any |= see;
                        if (__all_sync(0xffffffffu, see == ~0u)) continue;
                        uint32_t x[32];
                        if (__any_sync(0xffffffffu, see)) {
                            tmem_ld_32x32b_x32(tS + lo, x);
                            ld_wait(x);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((see >> e) & 1u)) x[e] = 0xff800000u;  // -inf
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = 0xff800000u;
                        }
                        tmem_st_32x32b_x32(tS + lo, x);
                    }
                    tmem_st_wait();
                    if (!any) low = -INFINITY;
                }
                // Maximum of the row (the reference moves only if it grew by 2^kLazy),
                // in four chains.  Where P lies over S, the upper 64 columns come first and
                // are read again for their weights: that leaves registers.
                uint32_t sr[kApart<D> ? 4 : 2][32];
                float mc[4] = {low, low, low, low};
                auto maxima = [&](const uint32_t (&x)[32], int c) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        mc[2 * c + (e >> 4)] = max3_nan(mc[2 * c + (e >> 4)], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                };
                if constexpr (kApart<D>) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(tS + c * 32, sr[c]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) ld_wait(sr[c]);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sfree[h]);  // S may be overwritten
#pragma unroll
                    for (int c = 0; c < 4; ++c) maxima(sr[c], c & 1);
                } else {
#pragma unroll
                    for (int half = 1; half >= 0; --half) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) tmem_ld_32x32b_x32(tS + half * 64 + c * 32, sr[c]);
                        ld_wait(sr[0]);
                        ld_wait(sr[1]);
                        maxima(sr[0], 0);
                        maxima(sr[1], 1);
                    }
                }
                const float mx = max3_nan(max3_nan(mc[0], mc[1], mc[2]), mc[3], mc[3]);
                // From -inf it always moves.  A NaN score makes the row NaN, and so
                // does +inf (inf - inf), as in the formula.
                const bool grow = !(mx <= m) && (m <= -FLT_MAX || !((mx - m) * a.qscale <= kLazy));
                const float f = grow ? ex2((m - mx) * a.qscale) : 1.0f;
                m = !grow ? m : mx == INFINITY ? NAN : mx;
                l *= f;
                if (kApart<D> && i > 0) {  // the last block's product is done: with P, and O is complete
                    if (ok) ok = tile_wait(&odone[h][(nb - 1) & 1], ((nb - 1) >> 1) & 1, status, abort_flag);
                    __syncwarp();
                    tc_fence_after();
                }
                if (i > 0 && __any_sync(0xffffffffu, grow)) {  // O is complete up to the last block
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(tO + c * 32, o);
                        ld_wait(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st_32x32b_x32(tO + c * 32, o);
                    }
                    tmem_st_wait();
                }
                // no score above -inf yet: all weights 0 (the mark times the scale may overflow)
                const float ms = kOff<T> - (m <= -FLT_MAX ? 0.0f : m) * a.qscale;
                const uint64_t qs2 = pack_f32x2(a.qscale, a.qscale), ms2 = pack_f32x2(ms, ms);
                uint64_t l2[4] = {0, 0, 0, 0};
                // 64 keys' weights, from the scores in x[0] and x[1].  They are rounded to the
                // 16-bit type, the operand's of the product with V: off by half a unit each, as
                // the result is once more.  (A second part for the rest would double that product
                // and P's room; against 64 bits the error is 28 to 40 % above that of weights in
                // fp32.)  l sums them before the rounding.
                auto weights = [&](const uint32_t (*x)[32], uint32_t (&p)[32]) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint32_t* s2 = &x[e >> 4][(2 * e) & 31];
                        const uint64_t y = fma_f32x2((static_cast<uint64_t>(s2[1]) << 32) | s2[0], qs2, ms2);
                        const uint64_t w = pack_f32x2(ex2(lo_f32(y)), ex2(hi_f32(y)));
                        l2[e & 3] = add_f32x2(l2[e & 3], w);
                        p[e] = pack2<T>(lo_f32(w), hi_f32(w));
                    }
                };
                if constexpr (kApart<D>) {
                    uint32_t p[2][32];
                    if (paired) {
                        if (ok) ok = tile_wait(my_turn, turns++ & 1, status, abort_flag);
                        __syncwarp();
                    }
                    weights(sr, p[0]);
                    weights(sr + 2, p[1]);
                    tmem_st_32x32b_x32(tP, p[0]);
                    tmem_st_32x32b_x32(tP + 32, p[1]);
                    if (paired && lane == 0 && !(h == 1 && i + 1 == u.nblk)) mbar_arrive(other_turn);
                    __syncwarp();
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&pfull[h][0]);
                        mbar_arrive(&pfull[h][1]);
                    }
                } else {
                    uint32_t p[32];
                    weights(sr, p);
                    tmem_st_32x32b_x32(tS, p);
                    tmem_ld_32x32b_x32(tS + 64, sr[0]);
                    tmem_ld_32x32b_x32(tS + 96, sr[1]);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pfull[h][0]);  // 64 keys' weights: their half of the product may start
                    __syncwarp();
                    ld_wait(sr[0]);
                    ld_wait(sr[1]);
                    weights(sr, p);
                    tmem_st_32x32b_x32(tS + 32, p);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pfull[h][1]);
                }
                const uint64_t ls = add_f32x2(add_f32x2(l2[0], l2[1]), add_f32x2(l2[2], l2[3]));
                l += lo_f32(ls) + hi_f32(ls);
            }
            gb += u.nblk;
            if (u.nblk > 0 && ok) {
                ok = kApart<D> ? tile_wait(&odone[h][(nb - 1) & 1], ((nb - 1) >> 1) & 1, status, abort_flag)
                               : tile_wait(&odone[h][0], nu & 1, status, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
                for (int e = 0; !kApart<D> && e < frees; ++e) mbar_arrive(&vempty[(gb - 1) % VS]);
                ++nu;
            }
            if (!ok) continue;  // ends above, with the group's other warps
            const int slot = u.slot;
            const int64_t q_row = u.token0 + tok0 + tok;
            const int64_t q_col = static_cast<int64_t>(head * a.G + (row - tok * a.G)) * D;
            T* out = static_cast<T*>(a.out) + q_row * a.ld_out + q_col;
            const float inv = m == -INFINITY ? 0.0f : 1.0f / l;  // nothing seen: zeros
            if (slot >= 0 && live) *part_ml<D>(t, slot, h * 128 + row) = make_float2(m, l);
            bool odd = false;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                __syncwarp();  // rows that are not live leave the loop's body early
                if (u.nblk > 0) {
                    tmem_ld_32x32b_x32(tO + c * 32, o);
                    ld_wait(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0;
                }
                if (!live) continue;
#pragma unroll
                for (int e = 0; e < 32; ++e) odd |= (o[e] & 0x7f800000u) == 0x7f800000u;
                if (slot >= 0) {
                    float* p = part_row<D>(t, slot, h * 128 + row) + c * 32;
#pragma unroll
                    for (int e = 0; e < 4; ++e) store32(p + 8 * e, o + 8 * e);
                } else {
                    uint32_t y[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        y[e] = m == -INFINITY ? 0u : pack2<T>(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                    if (t.wide) {
                        store32(out + c * 32, y);
                        store32(out + c * 32 + 16, y + 8);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            reinterpret_cast<uint4*>(out + c * 32)[e] = make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                    }
                }
            }
            // NaN or an infinity in O although the weights' sum is finite: it came from V,
            // perhaps from a row of it that this query does not see.  Or scores too large for
            // the product of the maximum and the scale (m is neither NaN nor a mark).
            odd = odd && l < INFINITY;
            odd |= m > -FLT_MAX && fabsf(m * a.qscale) >= kFar;
            for (uint32_t rows = __ballot_sync(0xffffffffu, odd && live); rows; rows &= rows - 1) {
                __syncwarp();  // its lane's stores are overwritten
                redo_row<T, D>(t, u, h * 128 + (warp & 3) * 32 + __ffs(rows) - 1);
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (s_abort) {  // a wait ran out: give this CTA's copies in flight time to land
        const unsigned long long t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the pieces of the units that were cut, a warp per row:
// out = sum_c O_c 2^(m_c - M) / sum_c l_c 2^(m_c - M).
template <typename T, int D>
__global__ void __launch_bounds__(256) k_paged_tc_join(const TcArgs t) {
    constexpr int E = D / 32;  // dims per lane
    pdl_wait();
    pdl_trigger();
    const PagedAttnArgs& a = t.p;
    const int lane = threadIdx.x & 31;
    const int rows = t.plan->joins * 256;  // at most 256 per CTA of the tile kernel
    for (int x = static_cast<int>(blockIdx.x * 256 + threadIdx.x) >> 5; x < rows; x += gridDim.x * 8) {
        const int row = x & 255;
        const TcJoin j = t.joins[x >> 8];
        const int tok = (row >> 7) * t.tok + (row & 127) / a.G;
        if ((row & 127) >= t.tok * a.G || tok >= j.ntok) continue;
        float mx = -INFINITY, l = 0.0f, o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.0f;
        for (int c0 = 0; c0 < j.pieces; c0 += 4) {  // four pieces' loads at a time
            float2 ml[4];
            float v[4][E];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + i, slot = c == 0 ? j.slot : 2 * (j.cta + c);
                ml[i] = make_float2(-INFINITY, 0.0f);
                if (c < j.pieces) {
                    ml[i] = *part_ml<D>(t, slot, row);
                    const float* p = part_row<D>(t, slot, row) + lane * E;
                    if constexpr (D == 128)
                        *reinterpret_cast<float4*>(v[i]) = *reinterpret_cast<const float4*>(p);
                    else
                        *reinterpret_cast<float2*>(v[i]) = *reinterpret_cast<const float2*>(p);
                }
            }
            float mn = mx;
#pragma unroll
            for (int i = 0; i < 4; ++i) mn = fmaxf(mn, ml[i].x);
            const float f = mn == mx ? 1.0f : ex2((mx - mn) * a.qscale);
            l *= f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] *= f;
            mx = mn;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (c0 + i >= j.pieces) break;
                const float w = ml[i].x == mx ? 1.0f : ex2((ml[i].x - mx) * a.qscale);
                l = fmaf(ml[i].y, w, l);
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(v[i][e], w, o[e]);
            }
        }
        const float inv = mx == -INFINITY ? 0.0f : 1.0f / l;
        T* out = static_cast<T*>(a.out) + (static_cast<int64_t>(j.token0) + tok) * a.ld_out +
                 static_cast<int64_t>(j.head * a.G + (row & 127) % a.G) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(out + e) = pack2<T>(o[e] * inv, o[e + 1] * inv);
    }
}

// ---- host -------------------------------------------------------------------------

int64_t max_tiles(int64_t T, int64_t B, int tok) { return T / (2 * tok) + B; }
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct TcLayout {
    size_t ranges, units, joins, part, total;
};
TcLayout tc_layout(int64_t T, int64_t B, int G, int D, int num_sms) {
    const int tok = 128 / G;
    const int grid = std::min(num_sms, kMaxGrid);
    const int64_t slots = 2 * grid;
    TcLayout l;
    l.ranges = 256;
    l.units = l.ranges + align256(grid * sizeof(int2));
    l.joins = l.units + align256((std::max<int64_t>(max_tiles(T, B, tok), kMaxCut) + grid) * sizeof(TcUnit));
    l.part = l.joins + align256(grid * sizeof(TcJoin));  // a cut unit ends at some CTA's share
    l.total = l.part + slots * 256 * (D + 2) * sizeof(float) + 16;  // the workspace may begin 16 bytes before a multiple of 32
    return l;
}

template <typename T, int D>
cudaError_t launch_tc(const PagedAttnArgs& p, int num_sms, cudaStream_t st) {
    TcArgs t{};
    t.p = p;
    t.tok = 128 / p.G;
    t.max_tiles = static_cast<int>(max_tiles(p.T, p.B, t.tok));
    t.box_keys = std::min(p.c.page_size, kKeys);
    t.boxes = kKeys / t.box_keys;
    t.grid = std::min(num_sms, kMaxGrid);
    t.slots = 2 * t.grid;
    t.wide = ((reinterpret_cast<uintptr_t>(p.out) | static_cast<uintptr_t>(p.ld_out) * 2) & 31) == 0;
    int dev = 0, l2 = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (e = cudaDeviceGetAttribute(&l2, cudaDevAttrL2CacheSize, dev)) != cudaSuccess) return e;
    t.l2_keys = static_cast<int64_t>(l2) * 3 / 5 / (int64_t(4) * D * p.c.H_kv);
    const TcLayout l = tc_layout(p.T, p.B, p.G, D, num_sms);
    char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(p.part) + 31) & ~uintptr_t(31));  // for store32
    t.plan = reinterpret_cast<TcPlan*>(ws);
    t.units = reinterpret_cast<TcUnit*>(ws + l.units);
    t.joins = reinterpret_cast<TcJoin*>(ws + l.joins);
    t.ranges = reinterpret_cast<int2*>(ws + l.ranges);
    t.part = reinterpret_cast<float*>(ws + l.part);

    CUtensorMap tmQ, tmK, tmV;
    if (!paged_cache_maps(p.c, t.box_keys, &tmK, &tmV, &t.p.d_tok, &t.p.d_head)) return cudaErrorInvalidValue;
    const auto type = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint32_t ones[3] = {1, 1, 1};
    const cuuint64_t qd[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p.H_q), static_cast<cuuint64_t>(p.T)};
    const cuuint64_t qs[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(p.ld_q) * 2};
    const cuuint32_t qb[3] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(t.tok)};
    if (!encode_tensor_map(&tmQ, type, 3, const_cast<void*>(p.q), qd, qs, qb, ones, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;

    const int smem = 1024 + (2 + kKStages<D> + kVStages<D>) * kTileBytes<D>;
    auto kern = k_paged_tc<T, D>;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    const int plan_smem = (4 * p.B + 1) * 4;
    // the most that any call takes: the limit is the function's, for all host threads
    e = cudaFuncSetAttribute(k_paged_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, (4 * kPagedMaxRequests + 1) * 4);
    if (e != cudaSuccess) return e;
    if ((e = launch_pdl(k_paged_plan, dim3(1), dim3(kPlanThreads), plan_smem, st, t)) != cudaSuccess) return e;
    if ((e = launch_pdl(kern, dim3(t.grid), dim3(kTcThreads), smem, st, tmQ, tmK, tmV, t)) != cudaSuccess) return e;
    // as many CTAs as are resident: a row is a few dependent loads
    return launch_pdl(k_paged_tc_join<T, D>, dim3(6 * t.grid), dim3(256), 0, st, t);
}

}  // namespace

bool paged_tc_applies(int G) { return G <= 128; }

size_t paged_tc_bytes(int64_t T, int64_t B, int G, int D, int num_sms) { return tc_layout(T, B, G, D, num_sms).total; }

cudaError_t launch_paged_tc(const PagedAttnArgs& a, int num_sms, cudaStream_t st) {
    if (a.c.dt == 1) return a.c.D == 128 ? launch_tc<__nv_bfloat16, 128>(a, num_sms, st) : launch_tc<__nv_bfloat16, 64>(a, num_sms, st);
    return a.c.D == 128 ? launch_tc<__half, 128>(a, num_sms, st) : launch_tc<__half, 64>(a, num_sms, st);
}

}  // namespace cider
