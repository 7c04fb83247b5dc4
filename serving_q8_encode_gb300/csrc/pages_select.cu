// Which pages a sparse attention reads: for each (layer, sequence, kv head) the n pages with the highest
// score, a page's score being an upper bound of its tokens' logits,
//
//   score = max over the group's query heads of sum_d max(q_d lo_d, q_d hi_d)
//
// with lo / hi the page's lowest and highest key per coordinate. The sum decides whole numbers, so it is
// defined in fp32 in a fixed order: eight neighbouring coordinates left to right, then halves onto halves
// over the D / 8 partial sums. Products of two 16-bit values are exact in fp32, so fused multiply-adds give
// the same sums; max(q lo, q hi) is q hi where q > 0 and q lo elsewhere. Ties go to the lowest page.
//
// The scores read two rows per page, so HBM binds long contexts; the rest is latency, hence one launch. A
// (layer, sequence, kv head) is a unit; a CTA scores a unit's pages or, where there are few units, a share of
// them (D / 8 lanes a page, one 16-byte asynchronous copy of each row into shared memory that only the lane
// itself reads, eight sets of pages a warp). The scores are kept as whole numbers of the same order. The
// unit's CTA, or the last of its CTAs to arrive (a count that wraps back to zero), counts each key's place where
// there are few, else finds the n-th largest two bits at a time, from the highest bit in which the keys differ
// until a threshold splits off exactly n, and writes the pages in order.
//
// Measured back to back: 5 sequences of up to 116 pages x 32 kv heads (d = 64) 4.3 us; 15 of up to 450 pages x 8 kv heads
// of 4 query heads (d = 128) 12.0 us; one of 4,096 pages 11.9 us; 16 of up to 512 pages, 4 layers (27.6 MB of bounds)
// 17.6 us. Scoring runs at the rate at which HBM delivers bounds once it has begun; the time is the chain before it
// (length, ids and queries together, then bounds: 2 us) and the search behind it (1 to 5 us). Clusters that sent their
// scores to one CTA's shared memory were slower (26 us for the 4,096 pages: their CTAs shared SMs).
#include "pages_internal.cuh"
#include "tc_ptx.cuh"

namespace polykv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxShared = 32768;   // pages whose scores a CTA keeps in shared memory (128 KB)
constexpr int kMaxSplit = 1024;     // units that may be shared out (their arrival counts are 4 KiB)
constexpr int kMinPages = 64;       // a CTA's least share of the pages
constexpr int kBlock = 32;          // pages that go to a CTA together
constexpr int kIds = 1024;          // pages whose ids are looked up at once
constexpr int kRing = 8;            // page sets in a warp's ring: 8 KB
constexpr uint32_t kForced = 0xFFFFFFFFu;   // the key of a page that is always taken
constexpr uint32_t kNoPage = 1u;            // the key of a page that does not exist (0 is padding)

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// a b + c of two 16-bit values in fp32: the product is exact, so this is the fused multiply-add of the converted
// values without the conversions. The halves of two words, low then high.
template <bool BF16>
__device__ __forceinline__ float fma_halves(uint32_t a, uint32_t b, float c) {
    const uint16_t a0 = (uint16_t)a, a1 = (uint16_t)(a >> 16), b0 = (uint16_t)b, b1 = (uint16_t)(b >> 16);
    if constexpr (BF16) {
        asm("fma.rn.f32.bf16 %0, %1, %2, %0;" : "+f"(c) : "h"(a0), "h"(b0));
        asm("fma.rn.f32.bf16 %0, %1, %2, %0;" : "+f"(c) : "h"(a1), "h"(b1));
    } else {
        asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(c) : "h"(a0), "h"(b0));
        asm("fma.rn.f32.f16 %0, %1, %2, %0;" : "+f"(c) : "h"(a1), "h"(b1));
    }
    return c;
}

// fp32 to a whole number of the same order (+0 and -0 alike), in (kNoPage, kForced)
__device__ __forceinline__ uint32_t key_of(float s) {
    const uint32_t u = __float_as_uint(s + 0.0f);
    return (u & 0x80000000u) ? max(~u, kNoPage + 1) : min(u | 0x80000000u, kForced - 1);
}

// Scores of a unit in the workspace: rows of 16-byte aligned keys.
__host__ __device__ __forceinline__ int64_t key_stride(int64_t max_pages) { return (max_pages + 3) / 4 * 4; }

struct PickShared {
    uint32_t red[2][kWarps][3];
    int last;
};

// The highest pair of bits (its lower one) in which keys of [lo, hi] differ, and what they share above it.
__device__ __forceinline__ int first_bits(uint32_t lo, uint32_t hi, uint32_t* T) {
    const int bit = lo == hi ? 0 : (31 - __clz(lo ^ hi)) & ~1;
    *T = bit >= 30 ? 0u : hi & ~((1u << (bit + 2)) - 1u);
    return bit;
}

// The pages with the n_sel largest of np keys, ascending, by the whole block. Thread t has keys [t KT, (t + 1) KT)
// of each chunk of 256 KT in registers. src is 16-byte aligned and readable up to a multiple of four keys.
template <int KT, bool SHARED>
__device__ void pick(const uint32_t* src, int np, int n_sel, int32_t* out, PickShared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kChunk = kThreads * KT;
    const int chunks = (np + kChunk - 1) / kChunk;
    const uint32_t want = (uint32_t)n_sel;
    uint32_t k[KT];
    auto load = [&](int c) {
#pragma unroll
        for (int i = 0; i < KT; i += 4) {
            const int at = c * kChunk + tid * KT + i;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (at < np) x = SHARED ? *reinterpret_cast<const uint4*>(src + at) : __ldcg(reinterpret_cast<const uint4*>(src + at));
            k[i] = x.x;
            k[i + 1] = at + 1 < np ? x.y : 0u;
            k[i + 2] = at + 2 < np ? x.z : 0u;
            k[i + 3] = at + 3 < np ? x.w : 0u;
        }
    };
    if (chunks == 1) load(0);
    // ---- the range of the keys but for the forced ones, which are above any threshold in it
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) load(c);
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            lo = min(lo, k[i] - 1u);   // padding wraps to the top
            if (k[i] != kForced) hi = max(hi, k[i]);
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        sh.red[1][warp][0] = lo;
        sh.red[1][warp][1] = hi;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        lo = min(lo, sh.red[1][w][0]);
        hi = max(hi, sh.red[1][w][1]);
    }
    lo += 1u;
    // ---- the largest T with at least n_sel keys >= T
    uint32_t T;
    {
        bool exact = false;
        int b = 0;
        for (int bit = first_bits(lo, hi, &T); bit >= 0 && !exact; bit -= 2, b ^= 1) {
            const uint32_t c1 = T | (1u << bit), c2 = T | (2u << bit), c3 = T | (3u << bit);
            uint32_t n1 = 0, n2 = 0, n3 = 0;
            for (int c = 0; c < chunks; ++c) {
                if (chunks > 1) load(c);
#pragma unroll
                for (int i = 0; i < KT; ++i) {
                    n1 += k[i] >= c1;
                    n2 += k[i] >= c2;
                    n3 += k[i] >= c3;
                }
            }
            if (chunks == 1 && 32 * KT <= 1023) {   // a warp's three counts fit into one word
                n1 = __reduce_add_sync(0xffffffffu, n1 | n2 << 10 | n3 << 20);
                if (lane == 0) sh.red[b][warp][0] = n1;
                __syncthreads();       // two buffers: one barrier a round is enough
                n1 = n2 = n3 = 0;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const uint32_t x = sh.red[b][w][0];
                    n1 += x & 1023u;
                    n2 += x >> 10 & 1023u;
                    n3 += x >> 20;
                }
            } else {
                n1 = __reduce_add_sync(0xffffffffu, n1);
                n2 = __reduce_add_sync(0xffffffffu, n2);
                n3 = __reduce_add_sync(0xffffffffu, n3);
                if (lane < 3) sh.red[b][warp][lane] = lane == 0 ? n1 : (lane == 1 ? n2 : n3);
                __syncthreads();
                n1 = n2 = n3 = 0;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    n1 += sh.red[b][w][0];
                    n2 += sh.red[b][w][1];
                    n3 += sh.red[b][w][2];
                }
            }
            const uint32_t m = n3 >= want ? n3 : (n2 >= want ? n2 : n1);
            if (m >= want) {
                T = n3 >= want ? c3 : (n2 >= want ? c2 : c1);
                exact = m == want;
            }
        }
        __syncthreads();
    }
    // ---- keys above T and the first of those equal to T, in page order: T >= kNoPage, so padding is never among them
    uint32_t all_gt = 0;
    if (chunks > 1) {
        for (int c = 0; c < chunks; ++c) {
            load(c);
#pragma unroll
            for (int i = 0; i < KT; ++i) all_gt += k[i] > T;
        }
        all_gt = __reduce_add_sync(0xffffffffu, all_gt);
        if (lane == 0) sh.red[0][warp][2] = all_gt;
    }
    uint32_t base_gt = 0, base_eq = 0;   // of the chunks before
    for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) load(c);
        uint32_t gt = 0, eq = 0;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            gt += k[i] > T;
            eq += k[i] == T;
        }
        uint32_t ig = gt, ie = eq;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, ig, o), y = __shfl_up_sync(0xffffffffu, ie, o);
            if (lane >= o) {
                ig += x;
                ie += y;
            }
        }
        if (lane == 31) {
            sh.red[0][warp][0] = ig;
            sh.red[0][warp][1] = ie;
        }
        __syncthreads();
        uint32_t bg = base_gt + ig - gt, be = base_eq + ie - eq;
        all_gt = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t g = sh.red[0][w][0], e = sh.red[0][w][1];
            if (w < warp) {
                bg += g;
                be += e;
            }
            base_gt += g;
            base_eq += e;
            all_gt += chunks > 1 ? sh.red[0][w][2] : g;
        }
        const uint32_t need = want - all_gt;   // keys equal to T that are taken
        const int at = c * kChunk + tid * KT;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            if (k[i] > T || (k[i] == T && be < need)) out[bg + min(be, need)] = at + i;
            bg += k[i] > T;
            be += k[i] == T;
        }
        __syncthreads();
    }
}

// The same for np <= 256, one key a thread: it is taken if fewer than n_sel keys come before it. One in front of it
// does if it is at least as large, one behind it if it is larger.
__device__ void pick_few(const uint32_t* src, int np, int n_sel, int32_t* out, PickShared& sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool take = false;
    const int own = 32 * warp;
    if (own < np) {
        const uint32_t k = tid < np ? src[tid] : 0u, reach = k - 1u;
        uint32_t before = 0;
#pragma unroll 4
        for (int j = 0; j < own; j += 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + j);
            before += (x.x > reach) + (x.y > reach) + (x.z > reach) + (x.w > reach);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const uint32_t x = __shfl_sync(0xffffffffu, k, j);
            before += x > (j < lane ? reach : k);
        }
#pragma unroll 4
        for (int j = own + 32; j < np; j += 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + j);
            before += (x.x > k) + (x.y > k) + (x.z > k) + (x.w > k);
        }
        take = tid < np && before < (uint32_t)n_sel;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, take);
    if (lane == 0) sh.red[0][warp][0] = __popc(m);
    __syncthreads();
    if (take) {
        uint32_t at = __popc(m & ((1u << lane) - 1u));
        for (int w = 0; w < warp; ++w) at += sh.red[0][w][0];
        out[at] = tid;
    }
}

// grid: units x X, X CTAs to a unit. NH query heads in registers (1, 2 or 4); MANY: the kv head has more, in
// blocks of NH = 4. gkeys: the scores' place where X > 1 or they do not fit into shared memory.
template <int D, bool BF16, int NH, bool MANY>
__global__ void __launch_bounds__(kThreads) pages_select_kernel(const PagesSelectArgs a, const int X,
                                                                uint32_t* __restrict__ count,
                                                                uint32_t* __restrict__ gkeys) {
    constexpr int LR = D / 8;              // lanes per page
    constexpr int PW = 32 / LR;            // pages of a set: what a warp scores at once
    constexpr int SPG = 4 / NH;            // sets of a group: four sums to fold
    constexpr int NG = NH == 4 ? 2 : 1;    // groups of an iteration
    constexpr int SI = SPG * NG;           // sets of an iteration
    constexpr int ST = kRing / SI;         // iterations in the ring
    extern __shared__ __align__(16) unsigned char smem[];
    uint4* ring = reinterpret_cast<uint4*>(smem);                                    // [warp][set][lo, hi][lane]
    uint32_t* keys_sh = reinterpret_cast<uint32_t*>(smem + kWarps * kRing * 1024);   // [max_pages, or 256 of them]
    __shared__ int32_t ids[kIds];
    __shared__ float score[kIds];
    __shared__ PickShared pick_sh;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    const PagesView& p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t unit = blockIdx.x / (uint32_t)X, rank = blockIdx.x - unit * X;
    const uint32_t ls = unit / (uint32_t)p.H;
    const int h = (int)(unit - ls * p.H);
    const int l = (int)(ls / (uint32_t)a.s.A), sq = (int)(ls - l * a.s.A);
    // Pages go to the unit's CTAs in blocks of kBlock, taken in turn: a CTA knows its pages before it knows the
    // sequence's length, so the length, the first page ids and the queries are on their way together.
    auto page_at = [&](int i) { return ((i / kBlock) * X + (int)rank) * kBlock + i % kBlock; };   // of the share's i-th
    const int32_t* table = a.s.table + (int64_t)sq * a.s.max_pages;
    int raw[kIds / kThreads];
    auto load_ids = [&](int c0) {
#pragma unroll
        for (int e = 0; e < kIds / kThreads; ++e) {
            const int lp = page_at(c0 + tid + e * kThreads);
            raw[e] = 0;   // volatile: the loads go out here, before the length is known
            if (lp < a.s.max_pages) asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(raw[e]) : "l"(table + lp));
        }
    };
    load_ids(0);
    const int ch = lane % LR, sub = lane / LR;
    const bool up1 = lane & (LR / 2), up2 = lane & (LR / 4);
    const uint16_t* qb = a.q + l * a.qs.layer + sq * a.qs.row + (int64_t)h * a.G * a.qs.head + 8 * ch;
    uint4* my_ring = ring + warp * kRing * 64 + lane;
    uint32_t q[NH][4];     // eight coordinates, two a word
    uint32_t pos[NH][4];   // all ones in the halves where q > 0
    auto load_q = [&](int g0) {
#pragma unroll
        for (int g = 0; g < NH; ++g) {
            // a head beyond the group repeats the last one, which leaves the maximum as it is
            uint4 w;
            asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "l"(qb + min(g0 + g, a.G - 1) * a.qs.head));
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2<BF16>(ww[i]);
                q[g][i] = ww[i];
                pos[g][i] = (f.x > 0.0f ? 0xFFFFu : 0u) | (f.y > 0.0f ? 0xFFFF0000u : 0u);
            }
        }
    };
    if (!MANY) load_q(0);
    uint32_t bad = 0;
    const int64_t len = clamp_len(a.s.lens[sq], a.s.max_pages, p.page, &bad);
    if (bad && p.status && rank == 0 && tid == 0) atomicOr(p.status, bad);
    const int np = (int)pages_of(len, p.page);
    int32_t* out = a.out + (int64_t)unit * a.n_sel;
    if (np <= a.n_sel) {   // all pages
        if (rank == 0)
            for (int i = tid; i < a.n_sel; i += kThreads) out[i] = i < np ? i : -1;
        return;
    }
    uint32_t* gk = gkeys ? gkeys + (int64_t)unit * key_stride(a.s.max_pages) : nullptr;
    uint32_t* keys = gk ? gk : keys_sh;

    // ---- scores of this CTA's share: whole blocks, the last one's end beyond np left out
    const int blocks = (np + kBlock - 1) / kBlock;
    const int share = rank < (uint32_t)blocks ? (blocks - (int)rank + X - 1) / X * kBlock : 0;
    const int writer_u = NH == 1 ? 2 * (up1 ? 1 : 0) + (up2 ? 1 : 0) : (NH == 2 ? (up1 ? 1 : 0) : 0);
    const bool writer = (ch & (NH == 1 ? LR / 4 - 1 : (NH == 2 ? LR / 2 - 1 : LR - 1))) == 0;
    // the head's bounds of page 0, and a page's in units of 16 bytes
    const uint4* bounds = reinterpret_cast<const uint4*>(p.bounds) +
                          ((int64_t)(a.s.layer0 + l) * p.n_pages * p.H + h) * (D / 4) + ch;
    const uint32_t page_step = (uint32_t)p.H * (D / 4);
    const uint32_t ring_u = tc::smem_u32(my_ring);
    for (int c0 = 0; c0 < share; c0 += kIds) {
        const int cn = min(kIds, share - c0);
        if (c0 > 0) {
            __syncthreads();
            load_ids(c0);
        }
#pragma unroll
        for (int e = 0; e < kIds / kThreads; ++e) {
            const int i = tid + e * kThreads;
            if (i < cn) ids[i] = page_at(c0 + i) < np ? (int)check_page(raw[e], p.n_pages, &bad) : -1;
        }
        __syncthreads();
        const int iters = (cn + PW * SI - 1) / (PW * SI);          // of the chunk; a warp takes every kWarps-th
        const int mine = (iters - warp + kWarps - 1) / kWarps;
        auto page_of = [&](int k, int u) { return ((warp + k * kWarps) * SI + u) * PW + sub; };
        auto issue = [&](int k) {
            if (k < mine) {
#pragma unroll
                for (int u = 0; u < SI; ++u) {
                    const int i = page_of(k, u);
                    const int id = i < cn ? ids[i] : -1;
                    const uint4* b = bounds + (uint64_t)(uint32_t)max(id, 0) * page_step;
                    const uint32_t dst = ring_u + ((k % ST) * SI + u) * 1024;
                    const int bytes = id >= 0 ? 16 : 0;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(b), "r"(bytes) : "memory");
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 512), "l"(b + D / 8), "r"(bytes)
                                 : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int k = 0; k < ST - 1; ++k) issue(k);
        for (int k = 0; k < mine; ++k) {
            issue(k + ST - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(ST - 1) : "memory");
            const uint4* at = my_ring + (k % ST) * SI * 64;
            float best[NG];
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) best[gr] = -INFINITY;
            for (int g0 = 0; g0 < (MANY ? a.G : 1); g0 += NH) {
                if (MANY) load_q(g0);
                float v[NG];
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                    float s[4];
#pragma unroll
                    for (int u = 0; u < SPG; ++u) {
                        const uint4 wl = at[(gr * SPG + u) * 64], wh = at[(gr * SPG + u) * 64 + 32];
                        const uint32_t lw[4] = {wl.x, wl.y, wl.z, wl.w}, hw[4] = {wh.x, wh.y, wh.z, wh.w};
#pragma unroll
                        for (int g = 0; g < NH; ++g) {
                            float t = 0.0f;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                t = fma_halves<BF16>(q[g][i], (hw[i] & pos[g][i]) | (lw[i] & ~pos[g][i]), t);
                            s[u * NH + g] = t;
                        }
                    }
                    // halves onto halves; the first two folds also share the four sums out over the lanes, so
                    // that a lane ends with sum 2 up1 + up2
                    const float s0 = (up1 ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, up1 ? s[0] : s[2], LR / 2);
                    const float s1 = (up1 ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, up1 ? s[1] : s[3], LR / 2);
                    v[gr] = (up2 ? s1 : s0) + __shfl_xor_sync(0xffffffffu, up2 ? s0 : s1, LR / 4);
                }
#pragma unroll
                for (int o = LR / 8; o > 0; o >>= 1)
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) v[gr] += __shfl_xor_sync(0xffffffffu, v[gr], o);
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                    if (NH >= 2) v[gr] = fmaxf(v[gr], __shfl_xor_sync(0xffffffffu, v[gr], LR / 4));
                    if (NH >= 4) v[gr] = fmaxf(v[gr], __shfl_xor_sync(0xffffffffu, v[gr], LR / 2));
                    best[gr] = fmaxf(best[gr], v[gr]);
                }
            }
            // one of the lanes that hold a set's sum writes it
            if (writer) {
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                    const int i = page_of(k, gr * SPG + writer_u);
                    if (i < cn) score[i] = best[gr];
                }
            }
        }
        __syncthreads();
        for (int i = tid; i < cn; i += kThreads) {
            const int lp = page_at(c0 + i);
            if (lp >= np) continue;
            uint32_t key = ids[i] >= 0 ? key_of(score[i]) : kNoPage;
            if (lp < a.keep_first || lp >= np - a.keep_last) key = kForced;
            keys[lp] = key;
        }
    }
    if (bad && p.status) atomicOr(p.status, bad);
    if (X > 1) {
        __syncthreads();   // the share's scores are written: one thread releases them and acquires the others'
        if (tid == 0) {
            uint32_t before;
            asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
                         : "=r"(before)
                         : "l"(count + unit), "r"((uint32_t)X - 1)
                         : "memory");
            pick_sh.last = before == (uint32_t)X - 1;
        }
        __syncthreads();
        if (!pick_sh.last) return;
    }
    if (np <= kThreads) {   // in shared memory, padded to whole groups of four
        const int end = (np + 3) & ~3;
        if (gk && tid < end) keys_sh[tid] = tid < np ? __ldcg(gk + tid) : 0u;
        if (!gk && tid < end - np) keys_sh[np + tid] = 0u;
        __syncthreads();
        pick_few(keys_sh, np, a.n_sel, out, pick_sh);
        return;
    }
    if (X == 1) {
        if (gk) __threadfence();
        __syncthreads();
    }
    if (gk) {
        if (np <= 4 * kThreads) pick<4, false>(gk, np, a.n_sel, out, pick_sh);
        else pick<16, false>(gk, np, a.n_sel, out, pick_sh);
    } else {
        if (np <= 4 * kThreads) pick<4, true>(keys_sh, np, a.n_sel, out, pick_sh);
        else pick<16, true>(keys_sh, np, a.n_sel, out, pick_sh);
    }
}

// CTAs per unit: one a SM in all where there are few units, no share below kMinPages pages.
int split_of(int64_t units, int64_t max_pages) {
    if (units > kMaxSplit) return 1;
    const int64_t fit = (int64_t)device_sm_count() / units, most = max_pages / kMinPages;
    const int64_t x = fit < most ? fit : most;
    return x < 1 ? 1 : (int)x;
}

template <int D, bool BF16>
polykv_status run(const PagesSelectArgs& a, void* ws, cudaStream_t st) {
    auto kern = a.G > 4   ? pages_select_kernel<D, BF16, 4, true>
                : a.G > 2 ? pages_select_kernel<D, BF16, 4, false>
                : a.G > 1 ? pages_select_kernel<D, BF16, 2, false>
                          : pages_select_kernel<D, BF16, 1, false>;
    const int64_t units = (int64_t)a.s.A * a.p.H * a.s.nl;
    const int X = split_of(units, a.s.max_pages);
    if (units * X > 0x7FFFFFFF) return set_error(POLYKV_E_UNSUPPORTED, "pages_select: %lld units", (long long)units);
    const bool shared = a.s.max_pages <= kMaxShared;
    const size_t keys = X > 1 || !shared ? kThreads : (size_t)key_stride(a.s.max_pages);   // few are picked there anyway
    const size_t smem = kWarps * kRing * 1024 + keys * sizeof(uint32_t);
    // the limit stands for the process: always the most that a call needs, so that calls of other sizes from other host
    // threads do not lower it before the launch
    constexpr int most = kWarps * kRing * 1024 + kMaxShared * (int)sizeof(uint32_t);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_select: smem attribute: %s", cudaGetErrorString(e));
    uint32_t* count = static_cast<uint32_t*>(ws);
    e = launch_after(kern, dim3((unsigned)(units * X)), kThreads, smem, st, a, X, count,
                     X > 1 || !shared ? count + kMaxSplit : (uint32_t*)nullptr);
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_select launch: %s", cudaGetErrorString(e));
    return POLYKV_OK;
}

}  // namespace

size_t pages_select_workspace(const PagesView& p, int A, int nl, int64_t max_pages) {
    const int64_t units = (int64_t)A * p.H * nl;
    if (max_pages <= kMaxShared && split_of(units, max_pages) == 1) return 0;
    return (kMaxSplit + (size_t)units * (size_t)key_stride(max_pages)) * sizeof(uint32_t);
}

polykv_status launch_pages_select(const PagesSelectArgs& a, polykv_dtype dt, void* ws, cudaStream_t st) {
    const bool bf = dt == POLYKV_BF16;
    if (a.p.d == 128) return bf ? run<128, true>(a, ws, st) : run<128, false>(a, ws, st);
    return bf ? run<64, true>(a, ws, st) : run<64, false>(a, ws, st);
}

}  // namespace polykv
