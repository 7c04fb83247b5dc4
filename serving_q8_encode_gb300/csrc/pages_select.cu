// Which pages a sparse attention reads: for each (layer, sequence, kv head) the n pages with the highest
// score, a page's score being an upper bound of its tokens' logits,
//
//   score = max over the group's query heads of sum_d max(q_d lo_d, q_d hi_d)
//
// with lo / hi the page's lowest and highest key per coordinate. The sum decides whole numbers, so it is
// defined in fp32 in a fixed order: eight neighbouring coordinates left to right, then halves onto halves
// over the D / 8 partial sums. Products of two 16-bit values are exact in fp32, so fused multiply-adds give
// the same sums. Ties go to the lowest page.
//
// The scores read two rows per page (HBM binds long contexts, latency short ones); D / 8 lanes share a page
// with one 16-byte load of each row. The choice is a search for the n-th largest key, bit by bit, in one
// block per (layer, sequence, kv head).
#include "pages_internal.cuh"

namespace polykv {
namespace {

constexpr int kScoreThreads = 128;
constexpr int kTile = 64;          // pages per block
constexpr int kPickThreads = 256;
constexpr int kPickCache = 8192;   // keys kept in shared memory

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

// grid: (sequences x kv heads, page tiles, layers)
template <int D, bool BF16>
__global__ void __launch_bounds__(kScoreThreads) pages_score_kernel(const PagesSelectArgs a, uint32_t* __restrict__ keys) {
    constexpr int LR = D / 8;          // lanes per page
    constexpr int PW = 32 / LR;        // pages a warp scores at once
    constexpr int GB = 4;              // query heads in registers
    const PagesView& p = a.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sq = blockIdx.x / p.H, h = blockIdx.x - sq * p.H, l = blockIdx.z;
    uint32_t bad = 0;
    const int64_t len = clamp_len(a.s.lens[sq], a.s.max_pages, p.page, &bad);
    if (bad && p.status && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(p.status, bad);
    const int np = (int)((len + p.page - 1) / p.page);
    const int p0 = blockIdx.y * kTile;
    if (p0 >= np || np <= a.n_sel) return;   // all pages are taken: nothing to score
    const int p1 = min(np, p0 + kTile);
    const int ch = lane % LR, sub = lane / LR;
    const uint16_t* qb = a.q + l * a.qs.layer + sq * a.qs.row + (int64_t)h * a.G * a.qs.head + 8 * ch;
    const int32_t* table = a.s.table + (int64_t)sq * a.s.max_pages;
    uint32_t* out = keys + (((int64_t)l * a.s.A + sq) * p.H + h) * a.s.max_pages;
    const int64_t lbase = (int64_t)(a.s.layer0 + l) * p.n_pages;
    for (int g0 = 0; g0 < a.G; g0 += GB) {
        float q[GB][8];
#pragma unroll
        for (int g = 0; g < GB; ++g) {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (g0 + g < a.G) w = __ldg(reinterpret_cast<const uint4*>(qb + (g0 + g) * a.qs.head));
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2<BF16>(ww[i]);
                q[g][2 * i] = f.x;
                q[g][2 * i + 1] = f.y;
            }
        }
        for (int pb = p0 + warp * PW; pb < p1; pb += (kScoreThreads / 32) * PW) {
            const int lp = pb + sub;
            int64_t id = -1;
            if (lp < p1) id = check_page(table[lp], p.n_pages, &bad);
            uint4 wl = make_uint4(0u, 0u, 0u, 0u), wh = wl;
            if (id >= 0) {
                const uint16_t* b = p.bounds + ((lbase + id) * p.H + h) * 2 * D + 8 * ch;
                wl = __ldg(reinterpret_cast<const uint4*>(b));
                wh = __ldg(reinterpret_cast<const uint4*>(b + D));
            }
            const uint32_t lw[4] = {wl.x, wl.y, wl.z, wl.w}, hw[4] = {wh.x, wh.y, wh.z, wh.w};
            float lo[8], hi[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 fl = unpack2<BF16>(lw[i]), fh = unpack2<BF16>(hw[i]);
                lo[2 * i] = fl.x;
                lo[2 * i + 1] = fl.y;
                hi[2 * i] = fh.x;
                hi[2 * i + 1] = fh.y;
            }
            float best = -INFINITY;
#pragma unroll
            for (int g = 0; g < GB; ++g) {
                float s = fmaxf(q[g][0] * lo[0], q[g][0] * hi[0]);
#pragma unroll
                for (int i = 1; i < 8; ++i) s += fmaxf(q[g][i] * lo[i], q[g][i] * hi[i]);
#pragma unroll
                for (int o = LR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (g0 + g < a.G) best = fmaxf(best, s);
            }
            if (lp < p1 && ch == 0) {
                uint32_t key = id >= 0 ? key_of(best) : 0u;
                if (lp < a.keep_first || lp >= np - a.keep_last) key = 0xFFFFFFFFu;
                if (g0 > 0) key = max(key, out[lp]);   // this lane wrote it
                out[lp] = key;
            }
        }
    }
    if (bad && p.status) atomicOr(p.status, bad);
}

__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t* red) {
    const uint32_t w = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = w;
    __syncthreads();
    uint32_t s = 0;
#pragma unroll
    for (int i = 0; i < kPickThreads / 32; ++i) s += red[i];
    return s;
}

// grid: (sequences x kv heads, layers)
__global__ void __launch_bounds__(kPickThreads) pages_pick_kernel(const PagesSelectArgs a, const uint32_t* __restrict__ keys) {
    __shared__ uint32_t cache[kPickCache];
    __shared__ uint32_t red[kPickThreads / 32], scan_gt[kPickThreads / 32], scan_eq[kPickThreads / 32];
    const PagesView& p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sq = blockIdx.x / p.H, h = blockIdx.x - sq * p.H, l = blockIdx.y;
    uint32_t dummy = 0;
    const int64_t len = clamp_len(a.s.lens[sq], a.s.max_pages, p.page, &dummy);
    const int np = (int)((len + p.page - 1) / p.page);
    const int64_t unit = ((int64_t)l * a.s.A + sq) * p.H + h;
    int32_t* out = a.out + unit * a.n_sel;
    if (np <= a.n_sel) {
        for (int i = tid; i < a.n_sel; i += kPickThreads) out[i] = i < np ? i : -1;
        return;
    }
    const uint32_t* src = keys + unit * a.s.max_pages;
    if (np <= kPickCache) {
        for (int i = tid; i < np; i += kPickThreads) cache[i] = src[i];
        __syncthreads();
        src = cache;
    }
    // the largest T with at least n_sel keys >= T
    uint32_t T = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t cand = T | (1u << bit);
        uint32_t n = 0;
        for (int i = tid; i < np; i += kPickThreads) n += src[i] >= cand;
        if (block_sum(n, red) >= (uint32_t)a.n_sel) T = cand;
    }
    // all keys above T, and the first keys equal to T, in page order
    const int per = (np + kPickThreads - 1) / kPickThreads;
    const int i0 = min(np, tid * per), i1 = min(np, i0 + per);
    uint32_t gt = 0, eq = 0;
    for (int i = i0; i < i1; ++i) {
        gt += src[i] > T;
        eq += src[i] == T;
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
        scan_gt[warp] = ig;
        scan_eq[warp] = ie;
    }
    __syncthreads();
    uint32_t bg = ig - gt, be = ie - eq, all_gt = 0;
    for (int w = 0; w < kPickThreads / 32; ++w) {
        if (w < warp) {
            bg += scan_gt[w];
            be += scan_eq[w];
        }
        all_gt += scan_gt[w];
    }
    const uint32_t need = (uint32_t)a.n_sel - all_gt;   // keys equal to T that are taken
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = src[i];
        if (k > T || (k == T && be < need)) out[bg + min(be, need)] = i;
        bg += k > T;
        be += k == T;
    }
}

template <int D, bool BF16>
polykv_status run(const PagesSelectArgs& a, uint32_t* keys, cudaStream_t st) {
    const unsigned units = (unsigned)(a.s.A * a.p.H);
    if (a.s.max_pages > a.n_sel) {
        const unsigned tiles = (unsigned)((a.s.max_pages + kTile - 1) / kTile);
        pages_score_kernel<D, BF16><<<dim3(units, tiles, (unsigned)a.s.nl), kScoreThreads, 0, st>>>(a, keys);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_select score launch: %s", cudaGetErrorString(e));
    }
    pages_pick_kernel<<<dim3(units, (unsigned)a.s.nl), kPickThreads, 0, st>>>(a, keys);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_select launch: %s", cudaGetErrorString(e));
    return POLYKV_OK;
}

}  // namespace

size_t pages_select_workspace(const PagesView& p, int A, int nl, int64_t max_pages) {
    return (size_t)nl * (size_t)A * (size_t)p.H * (size_t)max_pages * sizeof(uint32_t);
}

polykv_status launch_pages_select(const PagesSelectArgs& a, polykv_dtype dt, void* ws, cudaStream_t st) {
    uint32_t* keys = static_cast<uint32_t*>(ws);
    const bool bf = dt == POLYKV_BF16;
    if (a.p.d == 128) return bf ? run<128, true>(a, keys, st) : run<128, false>(a, keys, st);
    return bf ? run<64, true>(a, keys, st) : run<64, false>(a, keys, st);
}

}  // namespace polykv
