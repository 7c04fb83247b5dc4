// Attention of runs of rows (prompts, chunks, drafted tokens) over a paged cache, causal, with a sliding window and sinks.
//
//   row i of a sequence stands at place p = len - count + i and sees tokens t <= p with t > p - window or t < sinks
//   out[row][hq] = sum_t softmax_t(scale q . k_t) v_t over what it sees; zeros if that is nothing
#include <cstdlib>

#include "pages_attend.cuh"
#include "pages_prompt.cuh"

namespace polykv {
namespace {

constexpr int kThreads = 256;

template <int D, int CODE, bool BF16>
__global__ void __launch_bounds__(kThreads) rows_exact_kernel(const PagesRowsArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32), jobs = (int64_t)a.s.nl * a.rows * a.Hq;
    for (int64_t job = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); job < jobs; job += warps) {
        const int h = (int)(job % a.Hq);
        const int64_t r = job / a.Hq % a.rows;
        const int l = (int)(job / a.Hq / a.rows);
        uint32_t bad = 0;
        const RowOf at = row_of(a, r, lane, &bad);
        if (at.place >= 0) attend_row<D, CODE, BF16>(a, l, at, r, h, lane, &bad);
        if (bad && a.p.status && lane == 0) atomicOr(a.p.status, bad);
    }
}

// ------------------------------------------------------------------ the tensor-core kernel
constexpr int kSoftWarps = 8;                 // two warpgroups, one for each row tile
constexpr int kWarpMma = kSoftWarps, kWarpTma = kSoftWarps + 1;
constexpr int kThreadsTc = 32 * (kSoftWarps + 4);   // the last warpgroup: products, copies, and two idle warps
// registers a thread after the split; at launch 168 each: 256 x 208 + 128 x 88 = 384 x 168
constexpr int kRegSoft = 208, kRegOther = 88;
constexpr int kTile = 128;                    // rows of a row tile, tokens of a key tile
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kRise = 8.0f;                 // log2 units that the maximum may rise before sums are scaled down

template <int D>
constexpr int tile_bytes() { return kTile * D * 2; }
template <int D>
constexpr int stages() { return D == 128 ? 4 : 8; }

struct UnitSh {   // one CTA's work: a block of one sequence's rows, for one kv head
    int p0, len, row0;   // place of the first row; the sequence's tokens; the first row
    int seq, ntok;
};
struct SharedTc {
    uint64_t full[8], empty[8], q_ready, s_full[2], p_most[2], p_ready[2], done;
    uint32_t pages_ok[2][8];   // of the last stages' tiles, a bit per 16-token step whose page exists
    uint32_t tmem;
    int abort;
    UnitSh unit;
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

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreadsTc, 1) rows_tc_kernel(const __grid_constant__ PagesRowsArgs a, const __grid_constant__ attend::PageMaps maps,
                                                                const int64_t none, const bool stall) {
    constexpr int NS = stages<D>(), HV = D / 64;
    constexpr int kTileB = tile_bytes<D>(), kHalf = kTile * 128;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* const q_sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);   // [2 row tiles][HV][128][128 B]
    unsigned char* const ring = q_sm + 2 * kTileB;                                                // [NS][HV][128][128 B]
    SharedTc& sh = *reinterpret_cast<SharedTc*>(ring + NS * kTileB);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagesView& p = a.p;
    const int GT = min(a.G, kTile);           // query heads of a kv head that a CTA takes
    const int RG = (a.G + GT - 1) / GT, TM = kTile / GT;   // tokens of a row tile
    const int hr = blockIdx.x % (p.H * RG), h = hr / RG, g0 = (hr - h * RG) * GT;
    const int gn = min(GT, a.G - g0);
    const int l = blockIdx.z;

    if (tid == 64) {
        for (int s = 0; s < NS; ++s) {
            tc::mbar_init(tc::smem_u32(&sh.full[s]), 1);
            tc::mbar_init(tc::smem_u32(&sh.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(tc::smem_u32(&sh.s_full[i]), 1);
            tc::mbar_init(tc::smem_u32(&sh.p_most[i]), 4);
            tc::mbar_init(tc::smem_u32(&sh.p_ready[i]), 4);
        }
        tc::mbar_init(tc::smem_u32(&sh.q_ready), 32 * kSoftWarps);
        tc::mbar_init(tc::smem_u32(&sh.done), 1);
        tc::mbar_init_fence();
        sh.abort = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    if (warp == 0) {
        // the block's sequence: sequence s owns the items [starts[s] / (2 TM) + s, starts[s + 1] / (2 TM) + s + 1); the last
        // ones, which see most, come first
        const int64_t item = (int64_t)(gridDim.x / (p.H * RG)) - 1 - blockIdx.x / (p.H * RG);
        int lo = 0, n = a.s.A;
        while (n > 1) {
            const int stride = (n + 31) / 32, i = lane * stride;
            const bool le = i < n && a.starts[lo + i] / (2 * TM) + lo + i <= item;
            const int cnt = max(1, __popc(__ballot_sync(0xffffffffu, le)));
            lo += (cnt - 1) * stride;
            n = min(stride, n - (cnt - 1) * stride);
        }
        const int64_t start = a.starts[lo], count = (int64_t)a.starts[lo + 1] - start, len = a.s.lens[lo];
        const int64_t first = (item - (start / (2 * TM) + lo)) * 2 * TM;
        uint32_t bad = 0;
        UnitSh u = {0, 0, 0, lo, 0};
        if (count < 0 || start < 0 || start + count > a.rows) {
            bad |= kPagesBadLength;
        } else if (len >= 0 && first >= 0 && first < count) {
            u.len = (int)clamp_len(len, a.s.max_pages, p.page, &bad);
            if (u.len < len || len < count) {
                bad |= kPagesBadLength;
            } else {
                u.p0 = (int)(len - count + first);
                u.row0 = (int)(start + first);
                u.ntok = (int)min((int64_t)(2 * TM), count - first);
            }
        }
        if (lane == 0) {
            sh.unit = u;
            if (bad && p.status && hr == 0 && l == 0) atomicOr(p.status, bad);
        }
    }
    __syncthreads();
    const UnitSh u = sh.unit;
    if (u.ntok == 0) return;
    const int p1 = u.p0 + u.ntok - 1;
    const Tiles tiles(u.p0, p1, a.window, a.sinks);
    auto sight = [&](int i) { return Sight(u.p0 + i * TM, min(p1, u.p0 + (i + 1) * TM - 1), a.window, a.sinks); };
    volatile int* abort = &sh.abort;

    if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegOther));
    if (warp == kWarpTma) {
        // ================================================================ producer: keys and values of a tile in turn
        uint32_t bad = 0;
        const int shift = page_shift(p.page), spb = p.page < 64 ? p.page / kPageStep : 4;   // steps of a box
        const int64_t head_row = ((int64_t)(a.s.layer0 + l) * p.n_pages * p.H + h) * p.page;
        int issued = 0;
        for (int j = 0; j < tiles.n; ++j) {
            const int jt = tiles.at(j);
            const int t = jt * kTile + (lane & 7) * kPageStep;
            int row = (int)none;          // behind the cache's last row: arrives as zeros
            bool ok = true, has = false;
            if (t <= p1 && (t + kPageStep > tiles.begin || t < (a.window > 0 ? a.sinks : 0))) {
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
                const int s = issued % NS;
                if (issued >= NS) tc::mbar_wait(tc::smem_u32(&sh.empty[s]), (issued / NS - 1) & 1, abort, kWaitNs);
                ++issued;
                if (__all_sync(0xffffffffu, *abort == 0) && !stall) {
                    const uint32_t full = tc::smem_u32(&sh.full[s]);
                    if (lane == 0) {
                        sh.pages_ok[kv][j & 7] = oks;
                        tc::mbar_arrive_expect_tx(full, kTileB);
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
            }
        }
        if (bad && p.status) atomicOr(p.status, bad);
        // until its copies have landed, or 50 ms after a wait has given up
        const uint64_t t0 = tc::globaltimer();
        uint64_t limit = kWaitNs;
        for (int k = max(0, issued - NS); k < issued; ++k)
            while (!tc::mbar_try(tc::smem_u32(&sh.full[k % NS]), (k / NS) & 1)) {
                const uint64_t now = tc::globaltimer() - t0;
                if (limit == kWaitNs && *abort) limit = now + 50000000ull;
                if (now > limit) {
                    *abort = 1;
                    break;
                }
            }
        if (*abort && p.status && lane == 0) atomicOr(p.status, kPagesTimeout);
    } else if (warp == kWarpMma) {
        // ================================================================ matrix products
        const Sight see[2] = {sight(0), sight(1)};
        const uint32_t q_u = tc::smem_u32(q_sm), ring_u = tc::smem_u32(ring);
        tc::tmem_alloc(tc::smem_u32(&sh.tmem), 512);
        tc::fence_before();
        tc::named_bar(1, 32 * (kSoftWarps + 1));   // the tensor memory's address, to the softmax's warps
        tc::fence_after();
        const uint32_t tmem = sh.tmem;
        uint32_t pp[2] = {0, 0};
        uint32_t started[2] = {0, 0};
        auto wait_stage = [&](int k) {
            const bool ok = tc::mbar_wait(tc::smem_u32(&sh.full[k % NS]), (k / NS) & 1, abort, kWaitNs);
            return __all_sync(0xffffffffu, ok) != 0;
        };
        auto scores = [&](int i, int k) {   // S_i = Q_i K^T
            issue_scores<D>(tmem + i * kTile, tc::sdesc(q_u + i * kTileB, 16, 1024), tc::sdesc(ring_u + (k % NS) * kTileB, 16, 1024),
                            idesc<BF16>(kTile, false), tc::smem_u32(&sh.s_full[i]));
        };
        bool ok = __all_sync(0xffffffffu, tc::mbar_wait(tc::smem_u32(&sh.q_ready), 0, abort, kWaitNs)) != 0;
        tc::fence_proxy_async();
        ok = wait_stage(0) && ok;
        for (int i = 0; i < 2; ++i)
            if (ok && see[i].any(tiles.at(0))) scores(i, 0);
        commit_elected(tc::smem_u32(&sh.empty[0]));
        for (int j = 0; j < tiles.n; ++j) {
            const int jt = tiles.at(j), kv = 2 * j + 1, kk = 2 * j + 2;
            const bool more = j + 1 < tiles.n;
            ok = wait_stage(kv) && ok;
            // slots behind the sequence's last token hold anything: their values must not meet a probability of zero
            const int left = u.len - jt * kTile;
            if (left < kTile && (left & (kPageStep - 1)) && ok) {
                const int r1 = (left + kPageStep - 1) & ~(kPageStep - 1);
                for (int i = lane; i < (r1 - left) * HV * 8; i += 32) {
                    const int r = left + i / (HV * 8), ch = i % (HV * 8);
                    *reinterpret_cast<uint4*>(ring + (kv % NS) * kTileB + (ch >> 3) * kHalf + r * 128 + (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                tc::fence_proxy_async();
                __syncwarp();
            }
            if (more) ok = wait_stage(kk) && ok;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (see[i].any(jt)) {
                    const uint64_t v = tc::sdesc(ring_u + (kv % NS) * kTileB, kHalf, 1024);
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(tc::smem_u32(&sh.p_most[i]), pp[i], abort, kWaitNs)) && ok;
                    tc::fence_after();
                    if (ok) issue_values6(tmem + 256 + i * kTile, tmem + i * kTile, v, idesc<BF16>(D, true), started[i]);
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(tc::smem_u32(&sh.p_ready[i]), pp[i], abort, kWaitNs)) && ok;
                    tc::fence_after();
                    if (ok) issue_values2(tmem + 256 + i * kTile, tmem + i * kTile + 48, v + 768, idesc<BF16>(D, true));
                    pp[i] ^= 1;
                    started[i] = 1;
                    __syncwarp();
                }
                if (ok && more && see[i].any(tiles.at(j + 1))) scores(i, kk);
            }
            commit_elected(tc::smem_u32(&sh.empty[kv % NS]));
            if (more) commit_elected(tc::smem_u32(&sh.empty[kk % NS]));
            __syncwarp();
        }
        commit_elected(tc::smem_u32(&sh.done));
        __syncwarp();
        tc::mbar_wait(tc::smem_u32(&sh.done), 0, abort, kWaitNs);
        tc::fence_before();
        tc::named_bar(2, 32 * (kSoftWarps + 1));   // nobody reads the tensor memory any more
        tc::fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoft));
        // ================================================================ softmax: a thread for each row
        const int i = warp >> 2, rr = (warp & 3) * 32 + lane, tok = rr / GT, g = rr - tok * GT, at = i * TM + tok;
        // queries into the swizzled tiles, zeros where a tile has no row: all on their way at once
#pragma unroll 4
        for (int k = tid; k < 2 * kTile * (D / 8); k += 32 * kSoftWarps) {
            const int r = k / (D / 8), ch = k - r * (D / 8), r2 = r & (kTile - 1), tok2 = r2 / GT, g2 = r2 - tok2 * GT;
            const int at2 = (r / kTile) * TM + tok2;
            const bool is = tok2 < TM && at2 < u.ntok && g2 < gn;
            const uint16_t* src = is ? a.q + l * a.qs.layer + (int64_t)(u.row0 + at2) * a.qs.row + (int64_t)(h * a.G + g0 + g2) * a.qs.head + 8 * ch : a.q;
            const uint32_t dst = tc::smem_u32(q_sm) + (r / kTile) * kTileB + (ch >> 3) * kHalf + tc::sw128(r2, (ch & 7) * 16);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(is ? 16 : 0) : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        tc::fence_proxy_async();
        tc::mbar_arrive(tc::smem_u32(&sh.q_ready));
        tc::named_bar(1, 32 * (kSoftWarps + 1));
        tc::fence_after();
        const uint32_t tmem = sh.tmem;
        const Sight see = sight(i);
        const bool mine = tok < TM && at < u.ntok && g < gn;
        const int place = u.p0 + at;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // the warp's quarter of the tensor memory's lanes
        const uint32_t tS = tmem + i * kTile + lanes, tO = tmem + 256 + i * kTile + lanes;
        constexpr float kUp = BF16 ? 0.0f : 7.0f;   // f16 probabilities are kept 2^7 larger, for its exponents
        float M = -INFINITY, L = 0.0f;
        uint32_t ph = 0;
        bool started = false, ok = true;
        for (int j = 0; j < tiles.n && ok; ++j) {
            const int jt = tiles.at(j);
            if (!see.any(jt)) continue;
            ok = __all_sync(0xffffffffu, tc::mbar_wait(tc::smem_u32(&sh.s_full[i]), ph, abort, kWaitNs)) != 0;
            ph ^= 1;
            if (!ok) break;
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
            const uint32_t pages = sh.pages_ok[0][j & 7];
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
#pragma unroll
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
        ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(tc::smem_u32(&sh.done), 0, abort, kWaitNs)) != 0;
        tc::fence_after();
        // a row that is not finite is done again, one by one: a value that is not finite has met its zeros, or it has seen one
        bool again = false;
        const float inv = L > 0.0f ? 1.0f / L : 0.0f;
        if (!(L < INFINITY)) again = true;
        uint16_t* out = a.out + (((int64_t)l * a.rows + u.row0 + at) * a.Hq + h * a.G + g0 + g) * D;
        if (started) {
#pragma unroll
            for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tc::tmem_ld16(tO + c, o);
                landed(o);
                float f[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    f[e] = __uint_as_float(o[e]) * inv;
                    again = again || !(fabsf(f[e]) < INFINITY);
                }
                if (mine && ok) {
#pragma unroll
                    for (int e = 0; e < 16; e += 8)
                        *reinterpret_cast<uint4*>(out + c + e) = make_uint4(pack_rn<BF16>(f[e], f[e + 1]), pack_rn<BF16>(f[e + 2], f[e + 3]),
                                                                            pack_rn<BF16>(f[e + 4], f[e + 5]), pack_rn<BF16>(f[e + 6], f[e + 7]));
                }
            }
        }
        tc::fence_before();
        tc::named_bar(2, 32 * (kSoftWarps + 1));
        uint32_t todo = __ballot_sync(0xffffffffu, again && mine && ok), bad = 0;
        while (todo) {
            const int from = __ffs(todo) - 1;
            todo &= todo - 1;
            const int at2 = __shfl_sync(0xffffffffu, at, from), g2 = __shfl_sync(0xffffffffu, g, from);
            const RowOf row = {u.seq, u.p0 + at2, u.len};
            attend_row<D, kPagesWide, BF16>(a, l, row, u.row0 + at2, h * a.G + g0 + g2, lane, &bad);
        }
    }
}

template <int D, bool BF16>
polykv_status run_tc(const PagesRowsArgs& a, cudaStream_t st) {
    const attend::PageMaps* maps;
    const polykv_status ms = pages_wide_maps(a.p, &maps);
    if (ms != POLYKV_OK) return ms;
    const int GT = a.G < kTile ? a.G : kTile, RG = (a.G + GT - 1) / GT, TM = kTile / GT;
    const int64_t blocks = (a.rows / (2 * TM) + a.s.A) * a.p.H * RG;
    if (blocks > 0x7FFFFFFF) return set_error(POLYKV_E_UNSUPPORTED, "pages_attend_rows: %lld blocks in one call", (long long)blocks);
    auto kern = rows_tc_kernel<D, BF16>;
    constexpr size_t smem = 1024 + (2 + stages<D>()) * tile_bytes<D>() + sizeof(SharedTc);
    static_assert(smem <= 232448, "shared memory of a block");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_attend_rows: smem attribute: %s", cudaGetErrorString(e));
    // Test hook for the bounded waits: POLYKV_TEST_STALL=1 makes the producer copy nothing.
    const char* env = getenv("POLYKV_TEST_STALL");
    const bool stall = env && env[0] == '1';
    const int64_t none = (int64_t)a.p.L * a.p.n_pages * a.p.H * a.p.page;   // below 2^31: checked with the maps
    e = launch_after(kern, dim3((unsigned)blocks, 1, (unsigned)a.s.nl), kThreadsTc, smem, st, a, *maps, none, stall);
    return e == cudaSuccess ? POLYKV_OK : set_error(POLYKV_E_CUDA, "pages_attend_rows launch: %s", cudaGetErrorString(e));
}

template <int D, int CODE>
polykv_status run(const PagesRowsArgs& a, bool bf, cudaStream_t st) {
    const int64_t jobs = (int64_t)a.s.nl * a.rows * a.Hq, want = (jobs + kThreads / 32 - 1) / (kThreads / 32);
    const unsigned grid = (unsigned)(want < 0x7FFFFFFF ? want : 0x7FFFFFFF);
    const cudaError_t e = bf ? launch_after(rows_exact_kernel<D, CODE, true>, dim3(grid), kThreads, 0, st, a)
                             : launch_after(rows_exact_kernel<D, CODE, false>, dim3(grid), kThreads, 0, st, a);
    return e == cudaSuccess ? POLYKV_OK : set_error(POLYKV_E_CUDA, "pages_attend_rows launch: %s", cudaGetErrorString(e));
}

}  // namespace

size_t pages_rows_workspace(const PagesRowsArgs&) { return 0; }

polykv_status launch_pages_rows(const PagesRowsArgs& a, polykv_dtype dt, void*, cudaStream_t st) {
    const bool bf = dt == POLYKV_BF16;
    if (a.p.code == kPagesWide) {
        if (a.p.d == 128) return bf ? run_tc<128, true>(a, st) : run_tc<128, false>(a, st);
        return bf ? run_tc<64, true>(a, st) : run_tc<64, false>(a, st);
    }
    if (a.p.code == kPagesInt8) return a.p.d == 128 ? run<128, kPagesInt8>(a, bf, st) : run<64, kPagesInt8>(a, bf, st);
    return a.p.d == 128 ? run<128, kPagesE4m3>(a, bf, st) : run<64, kPagesE4m3>(a, bf, st);
}

}  // namespace polykv
