// Attention of runs of rows (prompts, chunks, drafted tokens) over a paged cache, causal, with a sliding window and sinks.
//
//   row i of a sequence stands at place p = len - count + i and sees tokens t <= p with t > p - window or t < sinks
//   out[row][hq] = sum_t softmax_t(scale q . k_t) v_t over what it sees; zeros if that is nothing
//
// 16-bit caches: on the tensor cores (tcgen05). 4 d flop per (row, query head, visible token) against a few bytes per row and
// token bind long prompts to the matrix unit's rate, and 128 x 128 exponentials a tile come next; a few rows behind a long
// context are bound by HBM. One CTA an SM goes through units: a block of 256 rows (tokens by the group's query heads, which share
// a kv head) against key tiles of 128 tokens. Its rows are two tiles of 128: while one's products run, the other's softmax does.
//   S = Q K^T (128 x 128, Q and K from shared memory), scores and O in tensor memory: 2 x 128 + 2 x d columns, all 512 at d = 128
//   P over S's place in 16 bits, O += P V with P from tensor memory, V from shared memory as it lies in its pages
// Warp roles: 8 warps softmax (a thread for each row, so that a row's maximum and sum need no shuffle), one issues the products,
// one copies keys and values page by page into a ring, one looks units up ahead and copies their queries, one keeps the clock.
// Where rows fill one tile only, both tiles hold them and take the key tiles in turn; where a call has few units, their keys are
// shared out over the idle CTAs and the last to arrive joins the parts in order, so results do not depend on timing. Where it has
// many, the grid has a CTA for each and those that run take over the next ones that have not begun (clusterlaunchcontrol), so that
// unequal units even out without a counter in memory: against every CTA taking each 152nd unit, 15 runs of 2 .. 5 rows (32 heads,
// d = 64) 66 -> 56 us, five prompts 97 -> 89, 15 runs of 33 .. 64 rows behind 3,000 .. 4,096 tokens 94 -> 56. (With a counter in a
// workspace, which captured graphs clear: 4 us more a call. The longest sequences first: prompts 92.)
//
// The running maximum is a reference that moves when it has risen by 2^8, so the accumulator in tensor memory is seldom scaled.
// Sums in fp32. A probability enters the product rounded to the row's type: half a step of it (2^-8 in bf16, 2^-11 in f16) beside
// an output that is rounded likewise; two parts as in the one-token kernel would double the product's work. f16 probabilities
// are kept 2^7 times larger: normal numbers down to 2^-21 of the largest, 2^-32 of it at worst below.
//
// What a row does not see meets a probability of zero in the product, so a value there that is not finite would spoil rows
// that must not see it: slots behind a sequence's last token are cleared in the ring, pages that do not exist arrive as zeros, and
// a row whose values' sums are not finite is computed again by one warp in the order of the definition (attend_row), up to where
// all of them are not finite.
//
// Measured (8 kv heads x 4 query heads, d = 128, bf16): 8,191 tokens under a window of 2,048: 198 us = 1.22 PFLOP/s of what is
// visible; five prompts of 601 .. 1,851 tokens 89 us; 16,384 tokens without a window 1,340 us = 1.64 PFLOP/s; four rows behind
// 131,068 tokens 110 us = 4.9 TB/s. The first with units dealt in turn 209 us, of which the products and hand-overs without the
// softmax's arithmetic are 184; with the two tiles' products issued by two warps, which fall into step, 245; with two threads a
// row 238. One instruction of the issuing warp costs about ten cycles beside two softmax warps on its scheduler, so its loop is
// short: one barrier for a tile's values and the next one's keys, products issued from single statements (one by one: 282 us).
//
// 8-bit caches: the pages that the rows see are widened into the workspace first (exact for the scales that appends give), since
// many rows read them: five prompts over int8 or e4m3 pages 124 us, of which about 33 are the copies.
//
// Every wait is bounded, by a clock that a warp keeps for the block (2 s in which no key tile was copied and no row that is done
// again moved on): then all waits return at once, the loops run to their end, copies in flight are waited for, and the status word
// says so.
#include <cstdlib>

#include "pages_attend.cuh"
#include "pages_prompt.cuh"
#include "rows_index.cuh"

namespace polykv {
namespace {

// ------------------------------------------------------------------ the tensor-core kernel
constexpr int kSoftWarps = 8;                 // two warpgroups, one for each row tile
constexpr int kWarpMma = kSoftWarps, kWarpTma = kSoftWarps + 1, kWarpUnits = kSoftWarps + 2, kWarpClock = kSoftWarps + 3;
constexpr int kThreadsTc = 32 * (kSoftWarps + 4);
// registers a thread after the split; at launch 168 each: 256 x 208 + 128 x 88 = 384 x 168
constexpr int kRegSoft = 208, kRegOther = 88;
constexpr int kTile = 128;                    // rows of a row tile, tokens of a key tile
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kRise = 8.0f;                 // log2 units that the maximum may rise before sums are scaled down
constexpr int kMaxSplitUnits = 128;           // units of a call whose keys are shared out over blocks: eight counts each in 4 KiB
constexpr int kPartTiles = 4;                 // key tiles that a part has at least

template <int D>
constexpr int tile_bytes() { return kTile * D * 2; }
template <int D>
constexpr int stages() { return rows::ring_stages(D); }

constexpr int kNearly = 2;    // key tiles of a unit that are still to be copied when its block takes the next
using rows::kPairs;                           // barriers of the ring: a tile's values and the next one's keys have one together
using rows::pair_barrier;
using rows::pair_parity;
using rows::Turns;

// One CTA's work at a time: a block of one sequence's rows for one kv head, over all of its key tiles or a part of them.
struct UnitSh {
    int p0, len, row0;   // place of the first row; the sequence's tokens; the first row
    int seq, ntok;       // ntok rows' tokens; 0: the end
    int l, h, g0, gn;    // layer, kv head, its query heads [g0, g0 + gn)
    int j0, j1;          // key tiles of the list
    int index, part, parts;   // among the call's units; which part of how many
};
struct SharedTc {
    uint64_t full[kPairs], empty[kPairs], unit_full[2], unit_free[2], q_ready, q_free, s_full[2], p_most[2], p_ready[2], o_done[2], half_ready, half_free, nearly, claimed, done;
    alignas(16) uint4 claim;   // the answer to a block's request for another block's unit
    float2 half_ml[kTile];     // the second half's maxima and sums, where both tiles hold the same rows
    uint32_t pages_ok[8];      // of the last stages' tiles, a bit per 16-token step whose page exists
    UnitSh unit[2];
    uint32_t tmem;
    int abort;
    uint32_t tiles;            // key tiles whose copies are under way: what the block's clock goes by, and
    uint64_t moved;            // when rows that are done again last moved on
};

// The key tiles that a run of places [p0, p1] sees, in order: those of the sinks, then from the window's first on.
// (Places are below 2^31 and tiles begin at multiples of 128, so t + 127 fits as well.)
struct Tiles {
    int begin;         // the first row's window
    int lead, from, n; // tiles of sinks; the first behind them; in all
    __device__ __forceinline__ Tiles(int p0, int p1, int window, int sinks) {
        begin = window > 0 && p0 >= window ? p0 - window + 1 : 0;
        const int first = min(begin, sinks);   // tokens before the window that are seen
        const int last = p1 / kTile;
        lead = min((first + kTile - 1) / kTile, last + 1);
        from = max(begin / kTile, lead);
        n = lead + max(last - from + 1, 0);
    }
    __device__ __forceinline__ int at(int j) const { return j < lead ? j : from + j - lead; }
};
// What the places [a, b] see of a key tile.
struct Sight {
    int a, b, low_a, low_b, sinks;   // the first token in the first and the last place's window
    __device__ __forceinline__ Sight(int a_, int b_, int window, int sinks_) : a(a_), b(b_) {
        low_a = window > 0 && a >= window ? a - window + 1 : 0;
        low_b = window > 0 && b >= window ? b - window + 1 : 0;
        sinks = window > 0 ? sinks_ : 0;
    }
    __device__ __forceinline__ bool any(int jt) const {
        const int t = jt * kTile;
        return a <= b && t <= b && (t + (kTile - 1) >= low_a || t < sinks);
    }
    __device__ __forceinline__ bool all(int jt) const {
        const int t = jt * kTile;
        return t + (kTile - 1) <= a && (t >= low_b || t + (kTile - 1) < sinks);
    }
};

__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&r)[32]) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]),
          "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]),
          "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]),
          "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(addr));
}

// Waits for the loads of these registers: the arithmetic on them depends on it.
__device__ __forceinline__ void landed(float (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]),
                   "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
                 :
                 : "memory");
    asm volatile(""
                 : "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]), "+f"(r[24]),
                   "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void landed(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                   "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// kind::f16 with fp32 sums; both operands bf16 or both f16.
template <bool BF16>
constexpr uint32_t idesc(uint32_t n, bool b_mn) {
    return tc::idesc_f16(kTile, n, false, b_mn) | (BF16 ? (1u << 7) | (1u << 10) : 0u);
}

// Two fp32 values in one register pair.
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 parts_of(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// The lowest n bits, 0 <= n <= 32 after clamping.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u); }

// The products of one row tile, each issued by one elected lane of the converged warp from a single statement, with all
// operands formed from a few values: written as a loop over one instruction at a time, the issuing thread and not the tensor
// core set the pace (100 and 75 cycles an instruction instead of 64).
//
// Scores: S (128 columns at d) = Q K^T over D / 16 steps; both operands K-major, 32 bytes on a step, 16 KB on 64 columns.
template <int D>
__device__ __forceinline__ void issue_scores(uint32_t d, uint64_t q, uint64_t k, uint32_t id, uint32_t bar) {
#define PKV_STEP(N, OFF) " add.u64 q" #N ", %1, " #OFF ";\n add.u64 k" #N ", %2, " #OFF ";\n"
#define PKV_MMA(N) " @P tcgen05.mma.cta_group::1.kind::f16 [%0], q" #N ", k" #N ", %3, T;\n"
    if constexpr (D == 128) {
        asm volatile(
            "{\n .reg .pred P, T, F;\n .reg .b64 q1, q2, q3, q4, q5, q6, q7, k1, k2, k3, k4, k5, k6, k7;\n"
            " elect.sync _|P, 0xffffffff;\n setp.ne.u32 T, 1, 0;\n setp.ne.u32 F, 0, 0;\n"
            PKV_STEP(1, 2) PKV_STEP(2, 4) PKV_STEP(3, 6) PKV_STEP(4, 1024) PKV_STEP(5, 1026) PKV_STEP(6, 1028) PKV_STEP(7, 1030)
            " @P tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, F;\n"
            PKV_MMA(1) PKV_MMA(2) PKV_MMA(3) PKV_MMA(4) PKV_MMA(5) PKV_MMA(6) PKV_MMA(7)
            " @P tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n}" ::"r"(d),
            "l"(q), "l"(k), "r"(id), "r"(bar)
            : "memory");
    } else {
        asm volatile(
            "{\n .reg .pred P, T, F;\n .reg .b64 q1, q2, q3, k1, k2, k3;\n"
            " elect.sync _|P, 0xffffffff;\n setp.ne.u32 T, 1, 0;\n setp.ne.u32 F, 0, 0;\n"
            PKV_STEP(1, 2) PKV_STEP(2, 4) PKV_STEP(3, 6)
            " @P tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, F;\n"
            PKV_MMA(1) PKV_MMA(2) PKV_MMA(3)
            " @P tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n}" ::"r"(d),
            "l"(q), "l"(k), "r"(id), "r"(bar)
            : "memory");
    }
#undef PKV_STEP
#undef PKV_MMA
}
// Values: O (D columns at d) += P V over steps of 16 tokens: P in tensor memory, 8 columns a step; V MN-major, 2 KB a step. Six
// steps, and two.
__device__ __forceinline__ void issue_values6(uint32_t d, uint32_t p, uint64_t v, uint32_t id, uint32_t add) {
    asm volatile(
        "{\n .reg .pred P, T, A;\n .reg .b32 p1, p2, p3, p4, p5;\n .reg .b64 v1, v2, v3, v4, v5;\n"
        " elect.sync _|P, 0xffffffff;\n setp.ne.u32 T, 1, 0;\n setp.ne.u32 A, %4, 0;\n"
        " add.u32 p1, %1, 8;\n add.u32 p2, %1, 16;\n add.u32 p3, %1, 24;\n add.u32 p4, %1, 32;\n add.u32 p5, %1, 40;\n"
        " add.u64 v1, %2, 128;\n add.u64 v2, %2, 256;\n add.u64 v3, %2, 384;\n add.u64 v4, %2, 512;\n add.u64 v5, %2, 640;\n"
        " @P tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, A;\n"
        " @P tcgen05.mma.cta_group::1.kind::f16 [%0], [p1], v1, %3, T;\n"
        " @P tcgen05.mma.cta_group::1.kind::f16 [%0], [p2], v2, %3, T;\n"
        " @P tcgen05.mma.cta_group::1.kind::f16 [%0], [p3], v3, %3, T;\n"
        " @P tcgen05.mma.cta_group::1.kind::f16 [%0], [p4], v4, %3, T;\n"
        " @P tcgen05.mma.cta_group::1.kind::f16 [%0], [p5], v5, %3, T;\n}" ::"r"(d),
        "r"(p), "l"(v), "r"(id), "r"(add)
        : "memory");
}
__device__ __forceinline__ void issue_values2(uint32_t d, uint32_t p, uint64_t v, uint32_t id) {
    asm volatile(
        "{\n .reg .pred P, T;\n .reg .b32 p1;\n .reg .b64 v1;\n"
        " elect.sync _|P, 0xffffffff;\n setp.ne.u32 T, 1, 0;\n add.u32 p1, %1, 8;\n add.u64 v1, %2, 128;\n"
        " @P tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, T;\n"
        " @P tcgen05.mma.cta_group::1.kind::f16 [%0], [p1], v1, %3, T;\n}" ::"r"(d),
        "r"(p), "l"(v), "r"(id)
        : "memory");
}
__device__ __forceinline__ void commit_elected(uint32_t bar) {
    asm volatile(
        "{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n"
        " @P tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar)
        : "memory");
}

// Partials of units whose keys several CTAs share out: per part of a unit 256 rows, as [2 tiles][4 quarters][D / 4][32 rows] of four
// columns each, and the rows' maximum and sum. A warp of the softmax joins the 32 rows of its quarter if it came last.
struct RowParts {
    uint32_t* counts;   // [kMaxSplitUnits][8], zero between calls
    float4* acc;
    float2* ml;         // [slot][2][128]
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreadsTc, 1) rows_tc_kernel(const __grid_constant__ PagesRowsArgs a, const __grid_constant__ attend::PageMaps maps,
                                                                const __grid_constant__ CUtensorMap q_map, const int q_boxes, const int none, const int items,
                                                                const int split, const __grid_constant__ RowParts rp, const bool queued, const bool stall) {
    constexpr int NS = stages<D>(), HV = D / 64;
    constexpr int kTileB = tile_bytes<D>(), kHalf = kTile * 128;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* const q_sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);   // [2 row tiles][HV][128][128 B]
    unsigned char* const ring = q_sm + 2 * kTileB;                                                // [NS][HV][128][128 B]
    SharedTc& sh = *reinterpret_cast<SharedTc*>(ring + NS * kTileB);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagesView& p = a.p;
    const int GT = min(a.G, kTile);           // query heads of a kv head that a unit takes
    const int RG = (a.G + GT - 1) / GT, TM = kTile / GT;   // tokens of a row tile
    volatile int* abort = &sh.abort;

    if (tid == 0) {
        for (int s = 0; s < kPairs; ++s) {
            tc::mbar_init(tc::smem_u32(&sh.full[s]), 1);
            tc::mbar_init(tc::smem_u32(&sh.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(tc::smem_u32(&sh.unit_full[i]), 1);
            tc::mbar_init(tc::smem_u32(&sh.unit_free[i]), kSoftWarps + 2);
            tc::mbar_init(tc::smem_u32(&sh.s_full[i]), 1);
            tc::mbar_init(tc::smem_u32(&sh.p_most[i]), 4);
            tc::mbar_init(tc::smem_u32(&sh.p_ready[i]), 4);
            tc::mbar_init(tc::smem_u32(&sh.o_done[i]), 1);
        }
        tc::mbar_init(tc::smem_u32(&sh.q_ready), 1);
        tc::mbar_init(tc::smem_u32(&sh.q_free), 1);
        tc::mbar_init(tc::smem_u32(&sh.half_ready), 4);
        tc::mbar_init(tc::smem_u32(&sh.half_free), 4);
        tc::mbar_init(tc::smem_u32(&sh.nearly), 1);
        tc::mbar_init(tc::smem_u32(&sh.claimed), 1);
        tc::mbar_init(tc::smem_u32(&sh.done), kThreadsTc / 32 - 1);
        tc::mbar_init_fence();
        sh.abort = 0;
        sh.moved = sh.tiles = 0;
    }
    if (warp == kWarpMma) tc::tmem_alloc(tc::smem_u32(&sh.tmem), 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = sh.tmem;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on

    // A warp's wait; all lanes get the same answer. Its limit is the block's clock's: once that has given up they all return.
    auto wait = [&](uint64_t& bar, uint32_t parity) {
        const uint32_t b = tc::smem_u32(&bar);
        bool ok = tc::mbar_try(b, parity);
        while (!ok) {
            ok = tc::mbar_try_suspend(b, parity, 2000u);
            if (!ok && *abort) break;
        }
        return __all_sync(0xffffffffu, ok) != 0;
    };
    // Until copies have landed, or 50 ms after a wait has given up.
    auto wait_landed = [&](uint64_t& bar, uint32_t parity) {
        const uint64_t t0 = tc::globaltimer();
        uint64_t limit = kWaitNs;
        while (!tc::mbar_try(tc::smem_u32(&bar), parity)) {
            const uint64_t now = tc::globaltimer() - t0;
            if (limit == kWaitNs && *abort) limit = now + 50000000ull;
            if (now > limit) {
                *abort = 1;
                break;
            }
        }
    };
    // The k-th unit, or none: every role takes them in turn, and says when it is through with one.
    auto take = [&](int k, UnitSh* u) {
        if (!wait(sh.unit_full[k & 1], (k >> 1) & 1)) return false;
        *u = sh.unit[k & 1];
        return u->ntok > 0;
    };
    auto through = [&](int k) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.unit_free[k & 1]));
    };
    // Where both row tiles would not be filled, they hold the same rows and take the key tiles in turn.
    auto halved = [&](const UnitSh& u) { return u.ntok <= TM; };
    auto sight = [&](const UnitSh& u, int i) {
        const int first = halved(u) ? 0 : i * TM, last = min(u.ntok, first + TM) - 1;
        return Sight(u.p0 + first, u.p0 + last, a.window, a.sinks);
    };
    auto turns_of = [&](const UnitSh& u, const Tiles& tiles, const Sight& see, int i) {
        const int nj = u.j1 - u.j0;
        Turns t = rows::every_other(nj, i);
        if (!halved(u)) {
            t = {0, nj, 0};
            while (t.lo < nj && !see.any(tiles.at(u.j0 + t.lo))) ++t.lo;
            while (t.hi > t.lo && !see.any(tiles.at(u.j0 + t.hi - 1))) --t.hi;
        }
        return t;
    };
    auto tiles_of = [&](const UnitSh& u) { return Tiles(u.p0, u.p0 + u.ntok - 1, a.window, a.sinks); };
    // A unit's queries into the two row tiles: boxes of 64 columns, the unit's heads and a tile's tokens (what a box holds beside
    // its rows belongs to nobody's result). Where a stride is none that a tensor map takes, 16 bytes at a time, two (D = 64: four)
    // rows a turn.
    auto load_rows = [&](const UnitSh& u) {
        if (q_boxes) {
            if (lane == 0) {
                const uint32_t ready = tc::smem_u32(&sh.q_ready);
                tc::mbar_arrive_expect_tx(ready, 2 * HV * GT * TM * 128);
#pragma unroll
                for (int tile = 0; tile < 2; ++tile)
#pragma unroll
                    for (int hf = 0; hf < HV; ++hf)
                        asm volatile(
                            "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
                                tc::smem_u32(q_sm) + tile * kTileB + hf * kHalf),
                            "l"(reinterpret_cast<uint64_t>(&q_map)), "r"(64 * hf), "r"(u.h * a.G + u.g0), "r"(u.row0 + (tile && !halved(u) ? TM : 0)),
                            "r"(a.qs.layer ? u.l : 0), "r"(ready)
                            : "memory");
            }
            __syncwarp();
            return;
        }
        constexpr int LR = D / 8, STEP = 32 / LR;   // lanes of a row, rows of a turn
        const int ch = lane % LR;
#pragma unroll 1
        for (int r = lane / LR; r < 2 * kTile; r += STEP) {
            const int tile = r / kTile, rr = r - tile * kTile, tok = rr / GT, g = rr - tok * GT, at = tok + (tile && !halved(u) ? TM : 0);
            const bool is = tok < TM && at < u.ntok && g < u.gn;
            const uint16_t* src = a.q + u.l * a.qs.layer + (int64_t)(u.row0 + at) * a.qs.row + (int64_t)(u.h * a.G + u.g0 + g) * a.qs.head + 8 * ch;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(q_sm) + tile * kTileB + (ch >> 3) * kHalf + tc::sw128(rr, (ch & 7) * 16)),
                         "l"(is ? src : a.q), "r"(is ? 16 : 0)
                         : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.q_ready));
    };

    if (warp >= kSoftWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegOther));
        if (warp == kWarpUnits) {
            // ============================================================ units, one ahead of the others, and their queries
            const int HR = p.H * RG;
            uint32_t bad = 0;
            int k = 0;
            // A sequence's rows as the call has them; false if it takes no part.
            auto rows_of = [&](int s, int64_t* start, int64_t* count, int* len) {
                *start = a.starts[s], *count = (int64_t)a.starts[s + 1] - *start;
                const int64_t n = a.s.lens[s];
                if (*count < 0 || *start < 0 || *start + *count > a.rows) {
                    bad |= kPagesBadLength;
                } else if (n >= 0 && *count > 0) {
                    *len = (int)clamp_len(n, a.s.max_pages, p.page, &bad);
                    if (*len == n && n >= *count) return true;
                    bad |= kPagesBadLength;
                }
                return false;
            };
            // Up to 32 sequences: a lane for each, so that no turn is without rows and none looks its sequence up in memory. The
            // others' items are counted by `starts` alone, as many as the host counted, and some have no rows.
            const bool few = a.s.A <= 32;
            int64_t start1 = 0, count1 = 0, base1 = 0, blocks1 = 0, n_items = items;
            int len1 = 0, seq1 = lane;
            auto number = [&]() {   // base1: the blocks of the lanes before; all of them, at most what the host counted
                int64_t sum = blocks1;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += x;
                }
                base1 = sum - blocks1;
                return min((int64_t)items, __shfl_sync(0xffffffffu, sum, 31));
            };
            if (few) {
                if (lane < a.s.A && rows_of(lane, &start1, &count1, &len1)) blocks1 = (count1 + 2 * TM - 1) / (2 * TM);
                bad = __reduce_or_sync(0xffffffffu, bad);
                n_items = number();
            }
            const int64_t per_layer = n_items * HR * split, total = per_layer * a.s.nl;
            // More units than the card runs blocks (queued): the grid has a block for each, and one that runs takes over one that has
            // not begun, when the copies of its unit are nearly all under way (the ring covers the time to look the next one up;
            // taken earlier, it would wait here while other blocks are idle).
            constexpr int64_t kNone = INT64_MAX;
            uint32_t claims = 0;
            bool left = queued;   // blocks that have not begun, as far as this one knows: none is asked for after a refusal
            auto claim = [&]() {
                const uint32_t to = tc::smem_u32(&sh.claim), bar = tc::smem_u32(&sh.claimed);
                tc::fence_proxy_async();   // the last answer has been read
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(bar, 16);
                    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(to), "r"(bar) : "memory");
                }
                __syncwarp();
                wait_landed(sh.claimed, claims & 1);
                uint32_t got = 0, id = 0;
                if (__all_sync(0xffffffffu, tc::mbar_try(bar, claims & 1)))
                    asm volatile(
                        "{\n .reg .b128 r;\n .reg .pred p;\n ld.shared.b128 r, [%2];\n"
                        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
                        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}"
                        : "=&r"(got), "=&r"(id)
                        : "r"(to)
                        : "memory");
                ++claims;
                left = got != 0;
                return got ? (int64_t)id : kNone;
            };
            auto next = [&](int64_t x) {
                if (!queued) return x + gridDim.x;
                if (k >= 1) wait(sh.nearly, (k - 1) & 1);
                return __any_sync(0xffffffffu, *abort != 0) ? kNone : claim();
            };
            for (int64_t x = blockIdx.x;; x = next(x)) {
                UnitSh u;
                u.ntok = 0;
                if (x < total) {
                    u.l = (int)(x / per_layer);
                    const int64_t rest = x - u.l * per_layer;
                    const int64_t item = n_items - 1 - rest / (HR * split);   // the last rows of a sequence, which see most, come first
                    const int in = (int)(rest % (HR * split)), hr = in % HR;
                    u.part = in / HR;
                    u.h = hr / RG;
                    u.g0 = (hr - u.h * RG) * GT;
                    u.gn = min(GT, a.G - u.g0);
                    u.index = (int)((x - (int64_t)u.part * HR) / (HR * split)) * HR + hr;   // below kMaxSplitUnits where it counts
                    int64_t start = 0, count = 0, first = -1;
                    if (few) {
                        const int owner = __popc(__ballot_sync(0xffffffffu, base1 <= item)) - 1;
                        u.seq = __shfl_sync(0xffffffffu, seq1, owner);
                        u.len = __shfl_sync(0xffffffffu, len1, owner);
                        start = __shfl_sync(0xffffffffu, start1, owner);
                        count = __shfl_sync(0xffffffffu, count1, owner);
                        first = (item - __shfl_sync(0xffffffffu, base1, owner)) * 2 * TM;
                    } else {
                        // the item's sequence: s owns the items [starts[s] / (2 TM) + s, starts[s + 1] / (2 TM) + s + 1)
                        int lo = 0, n = a.s.A;
                        while (n > 1) {
                            const int stride = (n + 31) / 32, i = lane * stride;
                            const bool le = i < n && a.starts[lo + i] / (2 * TM) + lo + i <= item;
                            const int cnt = max(1, __popc(__ballot_sync(0xffffffffu, le)));
                            lo += (cnt - 1) * stride;
                            n = min(stride, n - (cnt - 1) * stride);
                        }
                        u.seq = lo;
                        if (rows_of(lo, &start, &count, &u.len)) first = (item - (start / (2 * TM) + lo)) * 2 * TM;
                    }
                    if (first >= 0 && first < count) {
                        u.p0 = (int)(u.len - count + first);
                        u.row0 = (int)(start + first);
                        u.ntok = (int)min((int64_t)(2 * TM), count - first);
                    }
                    if (u.ntok == 0) continue;
                    const int n_tiles = tiles_of(u).n;
                    u.parts = min(split, max(1, n_tiles / kPartTiles));
                    if (u.part >= u.parts) continue;
                    u.j0 = (int)((int64_t)n_tiles * u.part / u.parts);
                    u.j1 = (int)((int64_t)n_tiles * (u.part + 1) / u.parts);
                } else if (queued && x != kNone) {
                    continue;   // a block of no unit
                }
                if (k >= 2 && !wait(sh.unit_free[k & 1], ((k >> 1) - 1) & 1)) break;
                if (lane == 0) {
                    sh.unit[k & 1] = u;
                    tc::mbar_arrive(tc::smem_u32(&sh.unit_full[k & 1]));
                }
                __syncwarp();
                if (u.ntok == 0) break;
                if (k >= 1 && !wait(sh.q_free, (k - 1) & 1)) break;
                if (__all_sync(0xffffffffu, *abort == 0)) load_rows(u);
                ++k;
            }
            if (bad && p.status && lane == 0) atomicOr(p.status, bad);
            if (k >= 1) wait_landed(sh.q_ready, (k - 1) & 1);
            while (left && __any_sync(0xffffffffu, *abort != 0)) claim();   // after a wait has given up no block begins any more
        } else if (warp == kWarpTma) {
            // ============================================================ producer: keys and values of a tile in turn
            uint32_t bad = 0;
            const int shift = page_shift(p.page), spb = p.page < 64 ? p.page / kPageStep : 4;   // steps of a box
            // Stages are used in the order K(0), V(0), K(1), V(1), ...; K(0) of a unit has a barrier to itself, V(j) and K(j + 1)
            // share one. Lane s keeps which barrier's turn filled stage s last.
            uint32_t issued = 0, tile = 0, pair = 0, filled = 0;
            UnitSh u;
            for (int k = 0; take(k, &u); ++k) {
                const Tiles tiles = tiles_of(u);
                const int p1 = u.p0 + u.ntok - 1, sinks = a.window > 0 ? a.sinks : 0;
                const int64_t head_row = ((int64_t)(a.s.layer0 + u.l) * p.n_pages * p.H + u.h) * p.page;
                for (int j = u.j0; j < u.j1; ++j, ++tile) {
                    if (j == max(u.j0, u.j1 - kNearly) && lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.nearly));
                    const int t = tiles.at(j) * kTile + (lane & 7) * kPageStep;
                    int row = none;               // behind the cache's last row: arrives as zeros
                    bool ok = true, has = false;
                    if (t <= p1 && (t + kPageStep > tiles.begin || t < sinks)) {
                        const int64_t id = check_page(a.s.table[(int64_t)u.seq * a.s.max_pages + (t >> shift)], p.n_pages, &bad);
                        ok = has = id >= 0;
                        if (has) row = (int)(head_row + id * p.H * p.page + (t & (p.page - 1)));
                    }
                    const uint32_t oks = __ballot_sync(0xffffffffu, ok) & 0xffu;
                    const uint32_t there = __ballot_sync(0xffffffffu, has);
                    const uint32_t box = ((1u << spb) - 1u) << ((lane & 7) & ~(spb - 1));
                    const bool boxed = (there & box) == box;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t s = issued % NS;
                        if (issued >= NS) {
                            const uint32_t before = __shfl_sync(0xffffffffu, filled, s);
                            wait(sh.empty[pair_barrier(before)], pair_parity(before));
                        }
                        if (lane == s) filled = pair;
                        ++issued;
                        const bool first = kv || j == u.j0;   // of its barrier's turn
                        if (__all_sync(0xffffffffu, *abort == 0) && !stall) {
                            const uint32_t full = tc::smem_u32(&sh.full[pair_barrier(pair)]);
                            if (lane == 0) {
                                if (kv == 0) {
                                    sh.pages_ok[tile & 7] = oks;
                                    sh.tiles = tile + 1;
                                }
                                if (first) tc::mbar_arrive_expect_tx(full, kv && j + 1 < u.j1 ? 2 * kTileB : kTileB);
                            }
                            __syncwarp();
                            if (lane < 8 && (!boxed || (lane & (spb - 1)) == 0)) {
                                const uint32_t dst = tc::smem_u32(ring) + s * kTileB + lane * (kPageStep * 128);
                                const void* m = kv ? (boxed ? &maps.v_box : &maps.v_step) : (boxed ? &maps.k_box : &maps.k_step);
#pragma unroll
                                for (int hf = 0; hf < HV; ++hf) tc::tma_2d_g2s(dst + hf * kHalf, m, 64 * hf, row, full);
                            }
                        }
                        __syncwarp();
                        if (kv == 0 || j + 1 == u.j1) ++pair;   // keys end a turn, and so do a unit's last values
                    }
                }
                through(k);
            }
            if (bad && p.status) atomicOr(p.status, bad);
            for (uint32_t n = pair > kPairs ? pair - kPairs : 0; n < pair; ++n) wait_landed(sh.full[pair_barrier(n)], pair_parity(n));
        } else if (warp == kWarpClock) {
            // ============================================================ the limit of all waits: no key tile copied for 2 s, and no
            // sign of life from rows that are done again (which take as long as they take). One clock for the block: a clock in
            // every wait that looks for that sign too made the five prompts 91 us instead of 89.
            const uint32_t bar = tc::smem_u32(&sh.done);
            uint64_t since = tc::globaltimer();
            uint32_t seen = 0;
            while (!tc::mbar_try_suspend(bar, 0, 20000u)) {
                const uint64_t moved = *reinterpret_cast<volatile uint64_t*>(&sh.moved), now = tc::globaltimer();
                const uint32_t tiles = *reinterpret_cast<volatile uint32_t*>(&sh.tiles);
                if (tiles != seen) {
                    seen = tiles;
                    since = now;
                }
                if (moved > since) since = moved;
                if (now > since + kWaitNs) {
                    if (*abort == 2) break;   // nor has it ended since
                    *abort = 2;
                    since = now;
                }
            }
            if (*abort && p.status && lane == 0) atomicOr(p.status, kPagesTimeout);
        } else if (warp == kWarpMma) {
            // ============================================================ matrix products, in the order S0(0), S1(0), then for each key
            // tile j: O0 += P0(j) V(j), S0(j + 1), O1 += P1(j) V(j), S1(j + 1). They run one after the other, so a tile's scores and
            // probabilities may share their place, and while one row tile's run, the other's softmax does.
            const uint32_t ring_u = tc::smem_u32(ring);
            const uint64_t q_desc = tc::sdesc(tc::smem_u32(q_sm), 16, 1024);
            uint32_t pp[2] = {0, 0}, s = 0, pair = 0;   // parities of the probabilities; the ring's next stage, its next barrier
            bool ok = true;
            UnitSh u;
            for (int k = 0; take(k, &u); ++k) {
                const Tiles tiles = tiles_of(u);
                const int nj = u.j1 - u.j0;
                const Turns turns[2] = {turns_of(u, tiles, sight(u, 0), 0), turns_of(u, tiles, sight(u, 1), 1)};
                // key tiles [f0, f1) that both row tiles take, and the next one too
                const int f0 = max(turns[0].lo, turns[1].lo), f1 = turns[0].by ? 0 : min(turns[0].hi, turns[1].hi) - 1;
                // slots behind the sequence's last token hold anything: the key tile that has them
                int tail = -1;
                if (u.len & (kPageStep - 1))
                    for (int j = nj - 1; j >= 0 && tail < 0 && tiles.at(u.j0 + j) >= (u.len - 1) / kTile; --j) tail = j;
                uint32_t started[2] = {0, 0};
                auto scores = [&](int i, uint32_t st) {
                    issue_scores<D>(tmem + i * kTile, q_desc + i * (kTileB >> 4), tc::sdesc(ring_u + st * kTileB, 16, 1024), idesc<BF16>(kTile, false),
                                    tc::smem_u32(&sh.s_full[i]));
                };
                auto values = [&](int i, uint64_t v) {
                    ok = wait(sh.p_most[i], pp[i]) && ok;
                    tc::fence_after();
                    if (ok) issue_values6(tmem + 256 + i * kTile, tmem + i * kTile, v, idesc<BF16>(D, true), started[i]);
                    ok = wait(sh.p_ready[i], pp[i]) && ok;
                    tc::fence_after();
                    if (ok) issue_values2(tmem + 256 + i * kTile, tmem + i * kTile + 48, v + 768, idesc<BF16>(D, true));
                    pp[i] ^= 1;
                    started[i] = 1;
                };
                auto arrived = [&]() { ok = wait(sh.full[pair_barrier(pair)], pair_parity(pair)) && ok; };
                auto release = [&]() {
                    commit_elected(tc::smem_u32(&sh.empty[pair_barrier(pair)]));
                    ++pair;
                };
                auto stage = [&]() {
                    const uint32_t now = s;
                    s = s + 1 == NS ? 0 : s + 1;
                    return now;
                };
                ok = wait(sh.q_ready, k & 1) && ok;
                tc::fence_proxy_async();
                arrived();
                const uint32_t first = stage();
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (ok && turns[i].has(0)) scores(i, first);
                release();
                if (nj == 1) commit_elected(tc::smem_u32(&sh.q_free));
                for (int j = 0; j < nj; ++j) {
                    const bool more = j + 1 < nj;
                    const uint32_t kv = stage(), kn = more ? stage() : 0;
                    const uint64_t v = tc::sdesc(ring_u + kv * kTileB, kHalf, 1024);
                    arrived();
                    if (j == tail && ok) {   // their values must not meet a probability of zero
                        const int left = (u.len - 1) % kTile + 1, r1 = (left + kPageStep - 1) & ~(kPageStep - 1);
                        for (int c = lane; c < (r1 - left) * HV * 8; c += 32) {
                            const int r = left + c / (HV * 8), ch = c % (HV * 8);
                            *reinterpret_cast<uint4*>(ring + kv * kTileB + (ch >> 3) * kHalf + r * 128 + (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        tc::fence_proxy_async();
                        __syncwarp();
                    }
                    if (j >= f0 && j < f1) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            values(i, v);
                            if (ok) scores(i, kn);
                        }
                    } else {
                        // a tile that rests now has its next scores first
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (ok && more && !turns[i].has(j) && turns[i].has(j + 1)) scores(i, kn);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (!turns[i].has(j)) continue;
                            values(i, v);
                            if (ok && more && turns[i].has(j + 1)) scores(i, kn);
                            if (j + 1 == turns[i].hi) commit_elected(tc::smem_u32(&sh.o_done[i]));
                        }
                    }
                    release();
                    if (j + 2 == nj) commit_elected(tc::smem_u32(&sh.q_free));
                }
                through(k);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoft));
        // ================================================================ softmax: a thread for each row
        const int i = warp >> 2, rr = (warp & 3) * 32 + lane, tok = rr / GT, g = rr - tok * GT;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // the warp's quarter of the tensor memory's lanes
        const uint32_t tS = tmem + i * kTile + lanes, tO = tmem + 256 + i * kTile + lanes;
        constexpr float kUp = BF16 ? 0.0f : 7.0f;   // f16 probabilities are kept 2^7 larger, for its exponents
        uint32_t ph = 0, sums = 0, halves = 0, tile = 0;
        UnitSh u;
        for (int k = 0; take(k, &u); ++k) {
            const Tiles tiles = tiles_of(u);
            const Sight see = sight(u, i);
            const Turns turns = turns_of(u, tiles, see, i);
            const bool both = halved(u);
            const int at = tok + (both ? 0 : i * TM);
            const int place = u.p0 + at;
            float M = -INFINITY, L = 0.0f;
            bool started = false, ok = true;
            for (int j = u.j0; j < u.j1; ++j, ++tile) {
                if (!turns.has(j - u.j0)) continue;
                const int jt = tiles.at(j);
                ok = wait(sh.s_full[i], ph) && ok;
                ph ^= 1;
                tc::fence_after();
                float s0[32], s1[32], s2[32], s3[32];
                tmem_ld32(tS, s0);
                tmem_ld32(tS + 32, s1);
                tmem_ld32(tS + 64, s2);
                tmem_ld32(tS + 96, s3);
                landed(s0);
                landed(s1);
                landed(s2);
                landed(s3);
                const uint32_t pages = sh.pages_ok[tile & 7];
                if (!see.all(jt) || pages != 0xffu) {   // what the row does not see, a bit each, so that no element branches
                    const int t = jt * kTile, hi = place - t + 1, lo = a.window > 0 ? place - a.window - t + 1 : 0, sk = see.sinks - t;
                    auto hide = [&](float (&s)[32], int c0) {
                        const uint32_t ok2 = pages >> (c0 >> 4);
                        const uint32_t m = low_bits(hi - c0) & (~low_bits(lo - c0) | low_bits(sk - c0)) & ((ok2 & 1u ? 0xffffu : 0u) | (ok2 & 2u ? 0xffff0000u : 0u));
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[e] = m & (1u << e) ? s[e] : -INFINITY;
                    };
                    hide(s0, 0);
                    hide(s1, 32);
                    hide(s2, 64);
                    hide(s3, 96);
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto largest = [&](const float (&s)[32]) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], s[e], s[e + 1]);
                };
                largest(s0);
                largest(s1);
                largest(s2);
                largest(s3);
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
                // the reference stays until the maximum has risen by 2^kRise, so that sums are seldom scaled
                const bool rise = started ? top > M + kRise : true;
                const float ref = rise ? fmaxf(top, M) : M;
                if (started && __any_sync(0xffffffffu, rise)) {
                    const float f = M == -INFINITY ? 0.0f : attend::ex2a(M - ref);
                    L *= f;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tc::tmem_ld16(tO + c, o);
                        landed(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc::tmem_st16(tO + c, o);
                    }
                }
                M = ref;
                started = true;
                const float sub = kUp - (M == -INFINITY ? 0.0f : M);
                const uint64_t scale2 = pair_of(a.scale_log2, a.scale_log2), sub2 = pair_of(sub, sub);
                uint64_t sum[4] = {0, 0, 0, 0};
                auto weigh = [&](float (&s)[32], int c0) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 x = parts_of(fma2(pair_of(s[e], s[e + 1]), scale2, sub2));
                        const float u = attend::ex2a(x.x), v = attend::ex2a(x.y);
                        sum[(e >> 1) & 3] = add2(sum[(e >> 1) & 3], pair_of(u, v));
                        w[e >> 1] = pack_rn<BF16>(u, v);
                    }
                    tc::tmem_st16(tS + c0 / 2, w);   // over scores that have been read: columns c0 / 2 .. + 16
                };
                // the first 96 tokens' products begin while the last 32 are weighed
                auto give = [&](uint64_t& bar) {
                    tc::wait_st();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(tc::smem_u32(&bar));
                };
                weigh(s0, 0);
                weigh(s1, 32);
                weigh(s2, 64);
                give(sh.p_most[i]);
                weigh(s3, 96);
                give(sh.p_ready[i]);
                const float2 la = parts_of(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
                L += la.x + la.y;
            }
            // Four lanes exchange the 16-byte chunks of their four rows, so that what goes out together is 64 bytes of a row and
            // not one chunk of 32 rows: lane 4a + b then has chunk b of rows 4a .. 4a + 3.
            uint16_t* out[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int r2 = (warp & 3) * 32 + (lane & ~3) + t, tok2 = r2 / GT, g2 = r2 - tok2 * GT, at2 = tok2 + (both ? 0 : i * TM);
                out[t] = tok2 < TM && at2 < u.ntok && g2 < u.gn 
                             ? a.out + (((int64_t)u.l * a.rows + u.row0 + at2) * a.Hq + u.h * a.G + u.g0 + g2) * D + 8 * (lane & 3)
                             : nullptr;
            }
            if (turns.any()) {
                ok = wait(sh.o_done[i], sums) && ok;
                sums ^= 1;
            }
            tc::fence_after();
            bool mine = tok < TM && at < u.ntok && g < u.gn;
            float f0 = 1.0f, f1 = 0.0f;   // factors of this tile's sums, and of the other half's
            if (both) {
                if (i == 1) {
                    sh.half_ml[rr] = make_float2(M, L);
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.half_ready));
                    wait(sh.half_free, halves & 1);   // until the other warpgroup has read them
                    ++halves;
                    through(k);
                    continue;
                }
                ok = wait(sh.half_ready, halves & 1) && ok;
                ++halves;
                tc::fence_after();
                const float2 x = sh.half_ml[rr];
                const float m = fmaxf(M, x.x), ms = m == -INFINITY ? 0.0f : m;
                f0 = attend::ex2a(M - ms);
                f1 = u.j1 - u.j0 > 1 ? attend::ex2a(x.x - ms) : 0.0f;
                L = fmaf(L, f0, u.j1 - u.j0 > 1 ? x.y * f1 : 0.0f);
                M = m;
            }
            // a row tile's sums, 32 columns at a time, with the other half's
            auto columns = [&](int c, float (&o)[32]) {
                tmem_ld32(tO + c, o);
                landed(o);
                if (both) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] *= f0;
                    if (u.j1 - u.j0 > 1) {
                        float o1[32];
                        tmem_ld32(tO + kTile + c, o1);
                        landed(o1);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = fmaf(o1[e], f1, o[e]);
                    }
                }
                if (!started) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.0f;
                }
            };
            bool joins = true;   // this warp writes its rows
            if (u.parts > 1) {
                const int64_t slot = (int64_t)u.index * split + u.part;
                float4* acc = rp.acc + ((slot * 2 + i) * 4 + (warp & 3)) * (D / 4) * 32 + lane;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    columns(c, o);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) __stcg(acc + ((c + e) >> 2) * 32, make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]));
                }
                __stcg(rp.ml + (slot * 2 + i) * kTile + rr, make_float2(M, L));
                __syncwarp();
                uint32_t before = 0;
                if (lane == 0)
                    asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
                                 : "=r"(before)
                                 : "l"(rp.counts + u.index * 8 + i * 4 + (warp & 3)), "r"((uint32_t)u.parts - 1)
                                 : "memory");
                before = __shfl_sync(0xffffffffu, before, 0);
                joins = before == (uint32_t)u.parts - 1;
                __syncwarp();
            }
            bool again = false;
            if (joins) {
                float2 ml[1];
                const float4* acc = rp.acc + (((int64_t)u.index * split * 2 + i) * 4 + (warp & 3)) * (D / 4) * 32 + lane;
                const float2* mls = rp.ml + ((int64_t)u.index * split * 2 + i) * kTile + rr;
                if (u.parts > 1) {
                    M = -INFINITY;
                    for (int q = 0; q < u.parts; ++q) M = fmaxf(M, __ldcg(mls + (int64_t)q * 2 * kTile).x);
                    const float ms = M == -INFINITY ? 0.0f : M;
                    L = 0.0f;
                    for (int q = 0; q < u.parts; ++q) {
                        ml[0] = __ldcg(mls + (int64_t)q * 2 * kTile);
                        L = fmaf(ml[0].y, attend::ex2a(ml[0].x - ms), L);
                    }
                }
                // a sum that is NaN: the row sees a logit that is NaN or +inf, and is NaN
                const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L), ms = M == -INFINITY ? 0.0f : M;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    if (u.parts == 1) {
                        columns(c, o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0.0f;
                        for (int q = 0; q < u.parts; ++q) {
                            const float f = attend::ex2a(__ldcg(mls + (int64_t)q * 2 * kTile).x - ms);
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 x = __ldcg(acc + (int64_t)q * 2 * 4 * (D / 4) * 32 + ((c + e) >> 2) * 32);
                                o[e] = fmaf(x.x, f, o[e]);
                                o[e + 1] = fmaf(x.y, f, o[e + 1]);
                                o[e + 2] = fmaf(x.z, f, o[e + 2]);
                                o[e + 3] = fmaf(x.w, f, o[e + 3]);
                            }
                        }
                    }
                    float zero = 0.0f;   // a NaN if one of them is not finite
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        o[e] *= inv;
                        zero = fmaf(o[e], 0.0f, zero);
                    }
                    again = again || (zero != 0.0f && L == L);
                    uint32_t w[4][4];   // [chunk][word]
#pragma unroll
                    for (int e = 0; e < 32; e += 2) w[e >> 3][(e >> 1) & 3] = pack_rn<BF16>(o[e], o[e + 1]);
                    // a 4 x 4 transposition in two steps: with the lane beside, then with the one two away
#pragma unroll
                    for (int d = 1; d < 4; d <<= 1) {
                        const bool odd = lane & d;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            if (x & d) continue;
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const uint32_t send = odd ? w[x][y] : w[x | d][y], got = __shfl_xor_sync(0xffffffffu, send, d);
                                if (odd) w[x][y] = got;
                                else w[x | d][y] = got;
                            }
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        if (out[t] && ok) *reinterpret_cast<uint4*>(out[t] + c) = make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
                }
            }
            tc::fence_before();
            __syncwarp();
            if (both && lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.half_free));
            // a row that is not finite is done again, one by one: a value that is not finite has met its zeros, or it has seen one
            uint32_t todo = __ballot_sync(0xffffffffu, again && mine && ok), bad = 0;
            while (todo) {
                const int from = __ffs(todo) - 1;
                todo &= todo - 1;
                const int at2 = __shfl_sync(0xffffffffu, at, from), g2 = __shfl_sync(0xffffffffu, g, from);
                const RowOf row = {u.seq, u.p0 + at2};
                attend_row<D, BF16>(a, u.l, row, u.row0 + at2, u.h * a.G + u.g0 + g2, lane, &bad, &sh.moved);
            }
            through(k);
        }
    }
    if (warp != kWarpClock) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.done));
    }
    // the products in flight end before the tensor memory goes: every unit's last ones have been waited for, unless a wait gave up
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == kWarpMma) {
        const uint64_t t0 = tc::globaltimer();
        while (*abort && tc::globaltimer() - t0 < 50000000ull) {
        }
        tc::tmem_dealloc(tmem, 512);
    }
}

// Blocks of rows that a call's items are, at most.
template <int D>
struct RowsPlan {
    int items, split;
    int64_t units;
    RowsPlan(const PagesRowsArgs& a) {
        const int GT = a.G < kTile ? a.G : kTile, RG = (a.G + GT - 1) / GT, TM = kTile / GT;
        items = (int)(a.rows / (2 * TM) + a.s.A);
        units = (int64_t)items * a.p.H * RG * a.s.nl;
        // Few units: the keys of each are shared out over as many blocks as there are idle ones, four key tiles each at least
        // (what a call can see at most is known here, how long its sequences are is not).
        int64_t seen = a.s.max_pages * a.p.page;
        if (a.window > 0 && seen > (int64_t)a.window + a.sinks + 4 * kTile) seen = (int64_t)a.window + a.sinks + 4 * kTile;
        int64_t want = units <= kMaxSplitUnits ? device_sm_count() / units : 1;
        if (want > seen / (kTile * kPartTiles)) want = seen / (kTile * kPartTiles);
        split = (int)(want > 1 ? want : 1);
    }
    size_t ml() const { return 4096; }
    size_t acc() const { return ml() + (split > 1 ? (size_t)units * split * 2 * kTile * sizeof(float2) : 0); }
    size_t total() const { return split > 1 ? acc() + (size_t)units * split * 2 * kTile * D * sizeof(float) : 0; }
};

// The queries as a tensor of columns, heads, rows and layers; false if a stride is none that a tensor map takes.
template <int D, bool BF16>
bool make_q_map(const PagesRowsArgs& a, CUtensorMap* m) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = attend::tensor_map_encoder();
    const int GT = a.G < kTile ? a.G : kTile, TM = kTile / GT;
    auto bytes = [](int64_t stride, int64_t n) { return n > 1 ? stride * 2 : (int64_t)D * 2; };
    const int64_t layers = a.qs.layer ? a.s.nl : 1;
    const int64_t st[3] = {bytes(a.qs.head, a.Hq), bytes(a.qs.row, a.rows), bytes(a.qs.layer, layers)};
    for (int64_t x : st)
        if (x <= 0 || x % 16 != 0 || x >= ((int64_t)1 << 40)) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)a.Hq, (cuuint64_t)a.rows, (cuuint64_t)layers};
    const cuuint64_t strides[3] = {(cuuint64_t)st[0], (cuuint64_t)st[1], (cuuint64_t)st[2]};
    const cuuint32_t box[4] = {64, (cuuint32_t)GT, (cuuint32_t)TM, 1}, one[4] = {1, 1, 1, 1};
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<uint16_t*>(a.q), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF16>
polykv_status run_tc(const PagesRowsArgs& a, const attend::PageMaps& maps, void* ws, cudaStream_t st) {
    const RowsPlan<D> plan(a);
    auto kern = rows_tc_kernel<D, BF16>;
    constexpr size_t smem = 1024 + (2 + stages<D>()) * tile_bytes<D>() + sizeof(SharedTc);
    static_assert(smem <= 232448, "shared memory of a block");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_attend_rows: smem attribute: %s", cudaGetErrorString(e));
    // Test hook for the bounded waits: POLYKV_TEST_STALL=1 makes the producer copy nothing.
    const char* env = getenv("POLYKV_TEST_STALL");
    const bool stall = env && env[0] == '1';
    const int none = (int)((int64_t)a.p.L * a.p.n_pages * a.p.H * a.p.page);   // below 2^31: checked with the maps
    char* base = static_cast<char*>(ws);
    const RowParts rp = {reinterpret_cast<uint32_t*>(base), reinterpret_cast<float4*>(base + plan.acc()), reinterpret_cast<float2*>(base + plan.ml())};
    const int64_t units = plan.units * plan.split;
    const bool queued = units > device_sm_count() && units <= 0x7FFFFFFF;   // as many blocks as a grid may have
    const unsigned grid = (unsigned)(queued || units < device_sm_count() ? units : device_sm_count());
    CUtensorMap q_map = {};
    const int q_boxes = make_q_map<D, BF16>(a, &q_map);
    e = launch_after(kern, dim3(grid), kThreadsTc, smem, st, a, maps, q_map, q_boxes, none, plan.items, plan.split, rp, queued, stall);
    return e == cudaSuccess ? POLYKV_OK : set_error(POLYKV_E_CUDA, "pages_attend_rows launch: %s", cudaGetErrorString(e));
}

// A call over pages of codes widens the pages that its rows see first: they are read by many rows, and the products take 16 bits.
// The widened pages lie in the workspace behind the call's own part: by page id, with the call's own tables, where the cache has no
// more pages than the tables have entries (the copies are then never more than the cache's layers themselves, twice as wide, and a
// page that sequences share has one place); by place in the tables, with a table that says so, where the tables are the smaller.
struct Widened {
    bool by_id;
    int64_t places;   // of a layer, in pages
    size_t table, k, v, total;
    Widened(const PagesRowsArgs& a, size_t own) {
        const int64_t entries = (int64_t)a.s.A * a.s.max_pages;
        by_id = a.p.n_pages <= entries;
        places = by_id ? a.p.n_pages : entries;
        auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
        const size_t pages = (size_t)places * a.s.nl * a.p.H * a.p.page * a.p.d * 2;
        table = up(own > 4096 ? own : 4096);
        k = up(table + (by_id ? 0 : (size_t)places * sizeof(int32_t)));
        v = up(k + pages);
        total = v + pages;
    }
};
size_t own_workspace(const PagesRowsArgs& a) { return a.p.d == 128 ? RowsPlan<128>(a).total() : RowsPlan<64>(a).total(); }

polykv_status run_wide(const PagesRowsArgs& a, const attend::PageMaps& m, bool bf, void* ws, cudaStream_t st) {
    if (a.p.d == 128) return bf ? run_tc<128, true>(a, m, ws, st) : run_tc<128, false>(a, m, ws, st);
    return bf ? run_tc<64, true>(a, m, ws, st) : run_tc<64, false>(a, m, ws, st);
}

}  // namespace

size_t pages_rows_workspace(const PagesRowsArgs& a) {
    if (a.rows == 0) return 0;
    const size_t own = own_workspace(a);
    return a.p.code == kPagesWide ? own : Widened(a, own).total;
}

polykv_status launch_pages_rows(const PagesRowsArgs& a, polykv_dtype dt, void* ws, cudaStream_t st) {
    const bool bf = dt == POLYKV_BF16;
    if (a.p.code == kPagesWide) {
        const attend::PageMaps* maps;
        const polykv_status s = pages_wide_maps(a.p, &maps);
        return s == POLYKV_OK ? run_wide(a, *maps, bf, ws, st) : s;
    }
    const Widened w(a, own_workspace(a));
    char* base = static_cast<char*>(ws);
    int32_t* table = w.by_id ? nullptr : reinterpret_cast<int32_t*>(base + w.table);
    PagesRowsArgs b = a;
    b.p.code = kPagesWide;
    b.p.scales = nullptr;
    b.p.k = reinterpret_cast<uint16_t*>(base + w.k);
    b.p.v = reinterpret_cast<uint16_t*>(base + w.v);
    b.p.L = a.s.nl;
    b.p.n_pages = w.places;
    b.s.layer0 = 0;
    if (table) b.s.table = table;
    attend::PageMaps maps;   // refuses 2^31 token slots and more, as for the one-token kernels: no card holds such a cache and its copies
    polykv_status s = attend::make_maps(b.p, CU_TENSOR_MAP_DATA_TYPE_UINT16, b.p.d, 1, 64, 2, &maps);
    if (s == POLYKV_OK) s = launch_pages_expand(a, dt, b.p.k, b.p.v, w.places, table, st);
    return s == POLYKV_OK ? run_wide(b, maps, bf, ws, st) : s;
}

}  // namespace polykv
