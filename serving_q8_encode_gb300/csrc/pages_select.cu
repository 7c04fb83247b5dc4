// Which pages a sparse attention reads: for each (layer, sequence, kv head) the n pages with the highest
// score, a page's score being an upper bound of its tokens' logits,
//
//   score = max over the group's query heads of sum_d max(q_d lo_d, q_d hi_d)
//
// with lo / hi the page's lowest and highest key per coordinate. The sum decides whole numbers, so it is
// defined in fp32 in a fixed order: eight neighbouring coordinates left to right, then halves onto halves
// over the D / 8 partial sums. Products of two 16-bit values are exact in fp32, so fused multiply-adds give
// the same sums, and so does adding both q+ hi and q- lo (q+ = max(q, 0), q- = min(q, 0)): one of them is 0.
// Ties go to the lowest page.
//
// The scores read two rows per page, so HBM binds long contexts; short ones are bound by latency, hence one
// launch. A cluster of CTAs takes one (layer, sequence, kv head): each scores a share of the pages (D / 8
// lanes a page, one 16-byte load of each row) and sends the scores as ordered whole numbers to the first CTA's
// shared memory, which then finds the n-th largest two bits at a time, stops as soon as a threshold splits
// off exactly n, and writes the pages in order.
#include "pages_internal.cuh"
#include "tc_ptx.cuh"

namespace polykv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxShared = 49152;   // pages whose scores the first CTA keeps in shared memory (192 KB)
constexpr int kMinPages = 64;       // a CTA's least share of the pages
constexpr int kHeads = 4;           // query heads in registers at once
constexpr int kSets = 2;            // page sets whose loads a warp has in flight

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// fp32 to a whole number of the same order (+0 and -0 alike), above 0 for every number
__device__ __forceinline__ uint32_t key_of(float s) {
    const uint32_t u = __float_as_uint(s + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// One head's partial sums over this lane's eight coordinates.
__device__ __forceinline__ float lane_sum(const float (&qp)[8], const float (&qm)[8], const float (&lo)[8],
                                          const float (&hi)[8]) {
    float s = fmaf(qm[0], lo[0], qp[0] * hi[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) s = fmaf(qm[i], lo[i], fmaf(qp[i], hi[i], s));
    return s;
}

// grid: units x CS in clusters of CS; gkeys: the scores' place where they do not fit into shared memory.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) pages_select_kernel(const PagesSelectArgs a, const int CS,
                                                                uint32_t* __restrict__ gkeys) {
    constexpr int LR = D / 8;          // lanes per page
    constexpr int PW = 32 / LR;        // pages of a set: what a warp scores at once
    extern __shared__ uint32_t keys_sh[];
    __shared__ uint32_t cnt[2][kWarps][4];
    __shared__ uint32_t tot_gt[kWarps], tot_eq[kWarps];
    const PagesView& p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t unit = blockIdx.x / CS;
    const uint32_t rank = CS > 1 ? cluster_rank() : 0;
    const int h = (int)(unit % p.H);
    const int64_t ls = unit / p.H;
    const int sq = (int)(ls % a.s.A), l = (int)(ls / a.s.A);
    uint32_t bad = 0;
    const int64_t len = clamp_len(a.s.lens[sq], a.s.max_pages, p.page, &bad);
    if (bad && p.status && rank == 0 && tid == 0) atomicOr(p.status, bad);
    const int np = (int)((len + p.page - 1) / p.page);
    int32_t* out = a.out + unit * a.n_sel;
    if (np <= a.n_sel) {   // all pages
        if (rank == 0)
            for (int i = tid; i < a.n_sel; i += kThreads) out[i] = i < np ? i : -1;
        return;
    }
    if (CS > 1) cluster_sync();   // the first CTA runs before anything is sent to it
    uint32_t* gk = gkeys ? gkeys + unit * a.s.max_pages : nullptr;

    // ---- scores of this CTA's share
    const int p0 = (int)((int64_t)np * rank / CS), p1 = (int)((int64_t)np * (rank + 1) / CS);
    {
        const int ch = lane % LR, sub = lane / LR;
        const uint16_t* qb = a.q + l * a.qs.layer + sq * a.qs.row + (int64_t)h * a.G * a.qs.head + 8 * ch;
        const int32_t* table = a.s.table + (int64_t)sq * a.s.max_pages;
        const uint16_t* bounds = p.bounds + ((int64_t)(a.s.layer0 + l) * p.n_pages * p.H + h) * 2 * D + 8 * ch;
        const uint32_t first = tc::smem_u32(keys_sh);
        uint32_t remote = first;       // the first CTA's array
        if (CS > 1) asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(first));
        for (int g0 = 0; g0 < a.G; g0 += kHeads) {
            float qp[kHeads][8], qm[kHeads][8];
#pragma unroll
            for (int g = 0; g < kHeads; ++g) {
                // a head beyond the group repeats the last one, which leaves the maximum as it is
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(qb + min(g0 + g, a.G - 1) * a.qs.head));
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack2<BF16>(ww[i]);
                    qp[g][2 * i] = fmaxf(f.x, 0.0f);
                    qm[g][2 * i] = fminf(f.x, 0.0f);
                    qp[g][2 * i + 1] = fmaxf(f.y, 0.0f);
                    qm[g][2 * i + 1] = fminf(f.y, 0.0f);
                }
            }
            for (int pb = p0 + warp * kSets * PW; pb < p1; pb += kWarps * kSets * PW) {
                int64_t id[kSets];
                uint4 wl[kSets], wh[kSets];
#pragma unroll
                for (int u = 0; u < kSets; ++u) {
                    const int lp = pb + u * PW + sub;
                    id[u] = lp < p1 ? check_page(__ldg(table + lp), p.n_pages, &bad) : -1;
                }
#pragma unroll
                for (int u = 0; u < kSets; ++u) {
                    wl[u] = wh[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (id[u] >= 0) {
                        const uint16_t* b = bounds + id[u] * p.H * 2 * D;
                        wl[u] = __ldg(reinterpret_cast<const uint4*>(b));
                        wh[u] = __ldg(reinterpret_cast<const uint4*>(b + D));
                    }
                }
#pragma unroll
                for (int u = 0; u < kSets; ++u) {
                    const uint32_t lw[4] = {wl[u].x, wl[u].y, wl[u].z, wl[u].w}, hw[4] = {wh[u].x, wh[u].y, wh[u].z, wh[u].w};
                    float lo[8], hi[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 fl = unpack2<BF16>(lw[i]), fh = unpack2<BF16>(hw[i]);
                        lo[2 * i] = fl.x;
                        lo[2 * i + 1] = fl.y;
                        hi[2 * i] = fh.x;
                        hi[2 * i + 1] = fh.y;
                    }
                    float s[kHeads];
#pragma unroll
                    for (int g = 0; g < kHeads; ++g) s[g] = lane_sum(qp[g], qm[g], lo, hi);
                    // halves onto halves; the first two folds also share the four heads out over the lanes, so
                    // that a lane ends with one head's sum
                    const bool up1 = lane & (LR / 2), up2 = lane & (LR / 4);
                    const float s0 = (up1 ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, up1 ? s[0] : s[2], LR / 2);
                    const float s1 = (up1 ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, up1 ? s[1] : s[3], LR / 2);
                    float v = (up2 ? s1 : s0) + __shfl_xor_sync(0xffffffffu, up2 ? s0 : s1, LR / 4);
#pragma unroll
                    for (int o = LR / 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, LR / 2));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, LR / 4));
                    const int lp = pb + u * PW + sub;
                    if (lp < p1 && ch == 0) {
                        uint32_t key = id[u] >= 0 ? key_of(v) : 0u;
                        if (lp < a.keep_first || lp >= np - a.keep_last) key = 0xFFFFFFFFu;
                        if (gk) {   // (this lane wrote what it reads back)
                            if (g0 > 0) key = max(key, gk[lp]);
                            gk[lp] = key;
                        } else {
                            const uint32_t at = remote + (uint32_t)lp * 4;
                            if (g0 > 0) {
                                uint32_t old;
                                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(old) : "r"(at) : "memory");
                                key = max(key, old);
                            }
                            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(key) : "memory");
                        }
                    }
                }
            }
        }
        if (bad && p.status) atomicOr(p.status, bad);
    }
    if (gk) __threadfence();
    if (CS > 1) cluster_sync();
    else __syncthreads();
    if (rank != 0) return;

    // ---- the largest T with at least n_sel keys >= T, two bits a round; keys of warp w: [w0, w1)
    const uint32_t* src = gk ? gk : keys_sh;
    const int span = (np + kWarps - 1) / kWarps;
    const int w0 = min(np, warp * span), w1 = min(np, w0 + span);
    const uint32_t want = (uint32_t)a.n_sel;
    uint32_t T = 0;
    bool exact = false;                // exactly n_sel keys are >= T
    for (int bit = 30; bit >= 0 && !exact; bit -= 2) {
        const uint32_t c1 = T | (1u << bit), c2 = T | (2u << bit), c3 = T | (3u << bit);
        uint32_t n12 = 0, n3 = 0;      // counts of c1 and c2 in 16 bits each (a lane counts at most span / 32)
        for (int i = w0 + lane; i < w1; i += 32) {
            const uint32_t k = gk ? __ldcg(src + i) : src[i];
            n12 += (k >= c1 ? 1u : 0u) + (k >= c2 ? 0x10000u : 0u);
            n3 += k >= c3;
        }
        const int b = (bit >> 1) & 1;  // two buffers: one barrier a round is enough
        const uint32_t r1 = __reduce_add_sync(0xffffffffu, n12 & 0xffffu), r2 = __reduce_add_sync(0xffffffffu, n12 >> 16);
        const uint32_t r3 = __reduce_add_sync(0xffffffffu, n3);
        if (lane == 0) {
            cnt[b][warp][0] = r1;
            cnt[b][warp][1] = r2;
            cnt[b][warp][2] = r3;
        }
        __syncthreads();
        uint32_t s1 = 0, s2 = 0, s3 = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            s1 += cnt[b][w][0];
            s2 += cnt[b][w][1];
            s3 += cnt[b][w][2];
        }
        if (s3 >= want) {
            T = c3;
            exact = s3 == want;
        } else if (s2 >= want) {
            T = c2;
            exact = s2 == want;
        } else if (s1 >= want) {
            T = c1;
            exact = s1 == want;
        }
    }
    // ---- keys above T and the first of those equal to T (all of them if T is exact), in page order
    uint32_t gt = 0, eq = 0;
    for (int i = w0; i < w1; i += 32) {
        const uint32_t k = i + lane < w1 ? (gk ? __ldcg(src + i + lane) : src[i + lane]) : 0u;
        gt += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && k > T));
        eq += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && k == T));
    }
    if (lane == 0) {
        tot_gt[warp] = gt;
        tot_eq[warp] = eq;
    }
    __syncthreads();
    uint32_t bg = 0, be = 0, all_gt = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            bg += tot_gt[w];
            be += tot_eq[w];
        }
        all_gt += tot_gt[w];
    }
    const uint32_t need = want - all_gt;   // keys equal to T that are taken
    for (int i = w0; i < w1; i += 32) {
        const uint32_t k = i + lane < w1 ? (gk ? __ldcg(src + i + lane) : src[i + lane]) : 0u;
        const uint32_t mg = __ballot_sync(0xffffffffu, i + lane < w1 && k > T);
        const uint32_t me = __ballot_sync(0xffffffffu, i + lane < w1 && k == T);
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t eq_before = be + __popc(me & below);
        const bool take = (mg >> lane & 1u) || ((me >> lane & 1u) && eq_before < need);
        if (take) out[bg + __popc(mg & below) + min(eq_before, need)] = i + lane;
        bg += __popc(mg);
        be += __popc(me);
    }
}

template <int D, bool BF16>
polykv_status run(const PagesSelectArgs& a, uint32_t* gkeys, cudaStream_t st) {
    auto kern = pages_select_kernel<D, BF16>;
    const int64_t units = (int64_t)a.s.A * a.p.H * a.s.nl;
    const bool shared = a.s.max_pages <= kMaxShared;
    // CTAs per unit: two a SM where there are few units, but no share below kMinPages pages
    int CS = 1;
    while (CS < 8 && units * CS < 2 * (int64_t)device_sm_count() && a.s.max_pages >= 2 * CS * (int64_t)kMinPages) CS *= 2;
    if (units * CS > 0x7FFFFFFF) return set_error(POLYKV_E_UNSUPPORTED, "pages_select: %lld units", (long long)units);
    const size_t smem = shared ? (size_t)a.s.max_pages * sizeof(uint32_t) : 0;
    cudaError_t e = cudaSuccess;
    if (smem > 32 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_select: smem attribute: %s", cudaGetErrorString(e));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * CS));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)CS;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, a, CS, shared ? (uint32_t*)nullptr : gkeys);
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_select launch: %s", cudaGetErrorString(e));
    return POLYKV_OK;
}

}  // namespace

size_t pages_select_workspace(const PagesView& p, int A, int nl, int64_t max_pages) {
    return max_pages <= kMaxShared ? 0 : (size_t)nl * (size_t)A * (size_t)p.H * (size_t)max_pages * sizeof(uint32_t);
}

polykv_status launch_pages_select(const PagesSelectArgs& a, polykv_dtype dt, void* ws, cudaStream_t st) {
    uint32_t* keys = static_cast<uint32_t*>(ws);
    const bool bf = dt == POLYKV_BF16;
    if (a.p.d == 128) return bf ? run<128, true>(a, keys, st) : run<128, false>(a, keys, st);
    return bf ? run<64, true>(a, keys, st) : run<64, false>(a, keys, st);
}

}  // namespace polykv
