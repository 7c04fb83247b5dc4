// The frame of attention of one new token per sequence over a paged cache, for the 16-bit cache (pages_attend.cu) and the
// 8-bit one (pages_attend8.cu): the work list and its walk, the producer warp, the join of cut units, and the kernel around a
// format's step. A format F brings what depends on how keys and values are held: the shape of its tiles, the query's
// registers, and one 16-token step of scores, softmax and values.
#pragma once

#include <cmath>
#include <cstdlib>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "pages_rows.cuh"
#include "tc_ptx.cuh"

namespace polykv {
namespace attend {

constexpr int kWarps = 4;                    // consumer warps
constexpr int kConsumers = 32 * kWarps;
constexpr int kThreads = kConsumers + 32;    // and the producer
constexpr int kMaxPerSm = 3;                 // CTAs per SM that the workspace is sized for
constexpr int kMaxCtas = 1024;
constexpr int kMaxStages = 8;
constexpr int kPassRows = 4;                 // rows that the warps join at once
constexpr int kJoinPieces = 128;             // pieces whose weights stand in shared memory at once
constexpr uint64_t kWaitNs = 2000000000ull;
// How a format's work is cut: chunks of S 16-token steps (4 or 8; the producer's work is per chunk, which a chunk of 8-bit codes
// has to earn with twice the tokens).
template <int S>
struct Cut {
    static constexpr uint32_t kSteps = S;
    static constexpr int kTokens = S * kPageStep;
    // What starting a unit costs, in chunks: finding its pages and query, and joining the warps. It stands as
    // virtual items before the unit's chunks in the work list, so that ranges full of short units hold fewer.
    static constexpr uint32_t kUnitCost = 8 / S;
    // Units of at most this many chunks are not cut: leaving pieces and joining them costs about 3 us, a chunk half one
    // (15 pages of 16 tokens for each of 160 units: 12.5 us cut, 9.3 us whole).
    static constexpr uint32_t kWhole = S == 4 ? 5 : 2;
    // A whole unit of at most this many chunks is left to one consumer warp, so that four of them go at once.
    static constexpr uint32_t kShort = 8 / S;
};
constexpr int kBoxTokens = 64;               // of a tensor copy at most
constexpr uint32_t kMinItems = 1;            // a CTA's least share

// The cache as two tensors of rows (token slots) for the tensor copies: boxes of a page (at most 64 rows) and,
// for a page's filled part, of 16 rows; 64 columns (128 bytes) wide.
struct PageMaps {
    CUtensorMap k_box, v_box, k_step, v_step;
};

template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (BF16) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
}

// k8, both sides fp32 with a 10-bit fraction; the low 13 bits do not count.
__device__ __forceinline__ void mma_tf32(float (&d)[4], float a0, float a1, float a2, float a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t to_tf32(float x) {   // to the nearest
    uint32_t u;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(u) : "f"(x));
    return u;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
    return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
__device__ __forceinline__ float ex2a(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool BF16>
__device__ __forceinline__ void store_out(const PagesAttendArgs& a, int64_t row, int D, int col, const float4& v) {
    if (a.out_f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * D + col) = v;
    } else {
        uint2 w;
        w.x = pack_rn<BF16>(v.x, v.y);
        w.y = pack_rn<BF16>(v.z, v.w);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + col) = w;
    }
}
// One finished row's four columns: normalised, or unnormalised for a caller that joins them with another
// part (the sums then go to a.ml). A row without tokens has L = 0 and gives zeros.
template <bool BF16>
__device__ __forceinline__ void finish4(const PagesAttendArgs& a, int64_t row, int D, int col, float4 v, float M,
                                        float L) {
    if (!a.ml) {
        const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);   // a NaN stays one
        v.x *= inv;
        v.y *= inv;
        v.z *= inv;
        v.w *= inv;
    } else if (col == 0) {   // a NaN sum keeps a maximum, else it would count as a part without tokens
        *reinterpret_cast<float2*>(a.ml + 2 * row) = make_float2(L == L ? M : fmaxf(M, 0.0f), L);
    }
    store_out<BF16>(a, row, D, col, v);
}

// The sequences' items (chunks and unit cost) as a running sum in shared memory, pre[a] standing before sequence a,
// and their lengths. Up to kWarpSeqs sequences are one warp's work, in front of the one barrier that the CTA's set-up
// needs anyway.
constexpr int kWarpSeqs = 256;
template <class C, bool WIN>
__device__ __forceinline__ void scan_items(const PagesAttendArgs& a, uint32_t* pre, int32_t* lens, uint32_t* wsum, bool report) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool one_warp = a.s.A <= kWarpSeqs;
    if (!one_warp || warp == 0) {
        const int threads = one_warp ? 32 : kThreads;
        const int per = (a.s.A + threads - 1) / threads;
        const int i0 = tid * per, i1 = min(a.s.A, i0 + per);
        uint32_t sum = 0, bad = 0;
        for (int i = i0; i < i1; ++i) {
            const int64_t len = clamp_len(__ldg(a.s.lens + i), a.s.max_pages, a.p.page, &bad);
            const uint32_t n = WIN ? window_steps(len, a.p.page, window_of(len, a.p.page, a.window, a.sinks)) : seq_steps(len, a.p.page, a.n_sel);
            lens[i] = (int32_t)len;
            pre[i] = sum;
            sum += n ? (n + C::kSteps - 1) / C::kSteps + C::kUnitCost : 0;
        }
        if (bad && report && a.p.status) atomicOr(a.p.status, bad);
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        uint32_t base = inc - sum;
        if (!one_warp) {
            if (lane == 31) wsum[warp] = inc;
            __syncthreads();
            for (int w = 0; w < warp; ++w) base += wsum[w];
        }
        for (int i = i0; i < i1; ++i) pre[i] += base;
        if (i1 == a.s.A && i0 < i1) pre[a.s.A] = base + sum;
    }
    __syncthreads();
}

// One CTA's range of the work list, piece by piece. The producer and the consumers walk it alike.
struct Piece {
    int l, sq, h, rg;        // layer, sequence, kv head, row group
    uint32_t c0, c1, n;      // chunks [c0, c1) of the unit's n
    uint64_t u0;             // the unit's first chunk in the work list
    bool solo;               // a whole short unit
};
template <class C>
struct Walk {
    static constexpr uint32_t kUnitCost = C::kUnitCost;
    const uint32_t* pre;
    uint64_t x, xe;
    int A, HR, RG;
    int l, sq, hr;
    uint32_t i0;

    __device__ __forceinline__ Walk(const uint32_t* pre_, int A_, int H, int RG_, uint64_t x_, uint64_t xe_)
        : pre(pre_), x(x_), xe(xe_), A(A_), HR(H * RG_), RG(RG_) {
        const uint64_t per_layer = (uint64_t)HR * pre[A];
        l = per_layer ? (int)quotient(x, per_layer) : 0;
        const uint64_t rem = x - (uint64_t)l * per_layer;
        int lo = 0, hi = A - 1;
        while (lo < hi) {   // the last sequence with pre * HR <= rem (it has items)
            const int mid = (lo + hi + 1) >> 1;
            if ((uint64_t)pre[mid] * HR <= rem) lo = mid;
            else hi = mid - 1;
        }
        sq = lo;
        const uint64_t in_seq = rem - (uint64_t)pre[sq] * HR;
        const uint32_t items = max(1u, pre[sq + 1] - pre[sq]);
        hr = (int)quotient(in_seq, items);
        i0 = (uint32_t)(in_seq - (uint64_t)hr * items);
    }
    // The next piece with chunks; false when the range is done.
    __device__ __forceinline__ bool next(Piece* p) {
        while (x < xe) {
            const uint32_t items = pre[sq + 1] - pre[sq];
            const uint32_t i1 = xe - x < (uint64_t)(items - i0) ? i0 + (uint32_t)(xe - x) : items;
            p->l = l;
            p->sq = sq;
            p->h = RG == 1 ? hr : hr / RG;
            p->rg = RG == 1 ? 0 : hr - p->h * RG;
            p->n = items - kUnitCost;
            p->c0 = i0 > kUnitCost ? i0 - kUnitCost : 0;
            p->c1 = i1 > kUnitCost ? i1 - kUnitCost : 0;
            p->u0 = x - i0 + kUnitCost;
            if (p->n <= C::kWhole) {   // whole, in the range that holds its first item
                p->c0 = 0;
                p->c1 = i0 == 0 ? p->n : 0;
            }
            x += i1 - i0;
            i0 = 0;
            if (i1 == items && ++hr == HR) {
                hr = 0;
                do {
                    if (++sq == A) {
                        sq = 0;
                        ++l;
                    }
                } while (x < xe && pre[sq + 1] == pre[sq]);
            }
            if (p->c0 < p->c1) {
                p->solo = p->c0 == 0 && p->c1 == p->n && p->n <= C::kShort;
                return true;
            }
        }
        return false;
    }
};

// Partials in the workspace: CTA c leaves the piece of a unit that began before its range in slot c of the first
// array, that of a unit that goes on behind it in slot c of the second. R rows each.
struct Partials {
    float* acc;    // [2][ctas][R][D]
    float2* ml;    // [2][ctas][R]
    int ctas;
};

// Joins the pieces [0, np) of the unit that began in CTA c0. Four columns of a row per thread; a row's pieces are
// shared out over the consumers' thread groups. The pieces' loads go out before their weights are known.
template <int D, int R, bool BF16>
__device__ __forceinline__ void join_pieces(const PagesAttendArgs& a, const Partials& w, uint32_t c0, int np, int64_t out_row, int rows,
                            float* scratch) {
    constexpr int TPR = D / 4;                 // threads per row
    constexpr int NG = kConsumers / TPR;       // thread groups: rows, or shares of a row's pieces
    constexpr int kBatch = 16;                 // loads in flight per thread
    const int grp = threadIdx.x / TPR, ln = threadIdx.x - grp * TPR, col = 4 * ln;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* wt = scratch;                       // [kWarps][kJoinPieces]
    float* sum = scratch + kWarps * kJoinPieces;   // [NG][D]
    auto slot = [&](int i) { return ((i == 0 ? w.ctas : 0) + (int)c0 + i) * R; };
    int rp = 1;
    while (rp < rows && rp < kWarps) rp <<= 1;     // rows in flight (NG is a multiple)
    const int parts = NG / rp;
    for (int r0 = 0; r0 < rows; r0 += rp) {
        const int r = r0 + grp % rp, part = grp / rp;
        float M = -INFINITY, L = 0.0f;         // of row r0 + warp, in warps below rp
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = 0; p0 < np; p0 += kJoinPieces) {
            const int pn = min(kJoinPieces, np - p0);
            float4 y[kBatch];
            auto load = [&](int b) {
#pragma unroll
                for (int e = 0; e < kBatch; ++e) {
                    const int i = part + (b + e) * parts;
                    if (r < rows && i < pn) y[e] = __ldcg(reinterpret_cast<const float4*>(w.acc + (slot(p0 + i) + r) * D + col));
                }
            };
            load(0);
            // warp k: the pieces' weights of row r0 + k, relative to the row's maximum so far
            if (warp < rp && r0 + warp < rows) {
                float2 ml[kJoinPieces / 32];
                float mx = M;
#pragma unroll
                for (int e = 0; e < kJoinPieces / 32; ++e) {
                    const int i = lane + 32 * e;
                    ml[e] = i < pn ? __ldcg(w.ml + slot(p0 + i) + r0 + warp) : make_float2(-INFINITY, 0.0f);
                }
#pragma unroll
                for (int e = 0; e < kJoinPieces / 32; ++e) mx = fmaxf(mx, ml[e].x);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float ms = mx == -INFINITY ? 0.0f : mx;
                float l = 0.0f;
#pragma unroll
                for (int e = 0; e < kJoinPieces / 32; ++e) {
                    const float f = ex2a(ml[e].x - ms);
                    wt[warp * kJoinPieces + lane + 32 * e] = f;
                    l = fmaf(ml[e].y, f, l);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                const float f = ex2a(M - ms);
                L = fmaf(L, f, l);
                M = mx;
                if (lane == 0) {
                    sum[warp * 4] = f;
                    sum[warp * 4 + 1] = M;
                    sum[warp * 4 + 2] = L;
                }
            }
            tc::named_bar(1, kConsumers);
            if (r < rows) {
                const float f = sum[(grp % rp) * 4];
                v.x *= f;
                v.y *= f;
                v.z *= f;
                v.w *= f;
                const float* wr = wt + (grp % rp) * kJoinPieces;
                for (int b = 0; part + b * parts < pn; b += kBatch) {
                    if (b > 0) load(b);
#pragma unroll
                    for (int e = 0; e < kBatch; ++e) {
                        const int i = part + (b + e) * parts;
                        if (i < pn) {
                            const float g = wr[i];
                            v.x = fmaf(y[e].x, g, v.x);
                            v.y = fmaf(y[e].y, g, v.y);
                            v.z = fmaf(y[e].z, g, v.z);
                            v.w = fmaf(y[e].w, g, v.w);
                        }
                    }
                }
                if (p0 + kJoinPieces >= np) {
                    M = sum[(grp % rp) * 4 + 1];
                    L = sum[(grp % rp) * 4 + 2];
                }
            }
            tc::named_bar(1, kConsumers);
        }
        *reinterpret_cast<float4*>(sum + grp * D + col) = v;
        tc::named_bar(1, kConsumers);
        if (part == 0 && r < rows) {
            for (int k = 1; k < parts; ++k) {
                const float4 y = *reinterpret_cast<const float4*>(sum + (grp + k * rp) * D + col);
                v.x += y.x;
                v.y += y.y;
                v.z += y.z;
                v.w += y.w;
            }
            finish4<BF16>(a, out_row + r, D, col, v, M, L);
        }
        tc::named_bar(1, kConsumers);
    }
}

template <int D>
constexpr int scratch_bytes() {   // the warps' partials of one pass, or the join's weights and sums
    constexpr int part = kWarps * kPassRows * D * 4, join = (kWarps * kJoinPieces + kConsumers * 4) * 4;
    return part > join ? part : join;
}
struct Join {   // a unit to join
    int64_t row;
    uint32_t c0;
    int np, rows;
};
struct Shared {   // behind the ring and the scratch
    uint64_t full[kMaxStages], empty[kMaxStages];
    alignas(8) uint32_t info[kMaxStages][4];      // visible tokens of each of the chunk's steps, 16 bits each
    float2 scale[kMaxStages][8];       // a step's key and value scale (8-bit cache)
    float pm[kWarps][16], pl[kWarps][16];
    uint32_t wsum[kThreads / 32];
    Join join[2];
    int joins, abort;
};


// RT row tiles of 8 query heads: 1 for units of up to 8, 2 for up to 16.
// WIN: under a window (in a kernel of its own: its few more instructions before the first copy cost the others 0.3 us).
template <class F, int RT, bool WIN>
__global__ void __launch_bounds__(kThreads, F::per_sm(RT))
    pages_attend_kernel(const __grid_constant__ PagesAttendArgs a, const __grid_constant__ PageMaps maps, const int NS,
                        uint32_t* __restrict__ ws_count, const __grid_constant__ Partials parts, const bool stall) {
    using C = typename F::Chunk;
    constexpr int D = F::D, S = C::kSteps;
    constexpr bool BF16 = F::BF16;
    constexpr int MT = D / 16;      // value m-tiles
    constexpr int R = 8 * RT;
    constexpr int kStage = F::kStage;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* ring = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    float* scratch = reinterpret_cast<float*>(ring + NS * kStage);
    Shared& sh = *reinterpret_cast<Shared*>(ring + NS * kStage + scratch_bytes<D>());
    uint32_t* pre = reinterpret_cast<uint32_t*>(&sh + 1);
    int32_t* lens = reinterpret_cast<int32_t*>(pre + a.s.A + 1);
    const uint32_t ring_u = tc::smem_u32(ring);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagesView& p = a.p;
    const int RG = (a.G + R - 1) / R;   // row groups per kv head

    if (tid == 32) {
        for (int s = 0; s < NS; ++s) {
            tc::mbar_init(tc::smem_u32(&sh.full[s]), 1);
            tc::mbar_init(tc::smem_u32(&sh.empty[s]), kWarps);
        }
        tc::mbar_init_fence();
        sh.abort = sh.joins = 0;
    }
    if (tid == kConsumers) {   // the maps' descriptors on their way to the copy engine
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.k_box) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.v_box) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.k_step) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.v_step) : "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    scan_items<C, WIN>(a, pre, lens, sh.wsum, blockIdx.x == 0);
    const uint64_t total = (uint64_t)a.s.nl * p.H * RG * pre[a.s.A];
    const uint64_t most = total / kMinItems;
    const uint32_t nc = most < 1 ? 1u : (most < gridDim.x ? (uint32_t)most : gridDim.x);

    // sequences without tokens: zeros
    for (int i = blockIdx.x; i < a.s.A; i += gridDim.x)
        if (pre[i + 1] == pre[i])
            for (int idx = tid; idx < a.s.nl * a.Hq * (D / 4); idx += kThreads) {
                const int l = idx / (a.Hq * (D / 4)), rest = idx - l * (a.Hq * (D / 4));
                finish4<BF16>(a, ((int64_t)l * a.s.A + i) * a.Hq + rest / (D / 4), D, (rest % (D / 4)) * 4,
                              make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.0f);
            }
    if (blockIdx.x >= nc) return;
    const Shares shares(total, nc);
    Walk<C> walk(pre, a.s.A, p.H, RG, shares.first(blockIdx.x), shares.first(blockIdx.x + 1));
    Piece pc;
    volatile int* abort = &sh.abort;
    int s = 0;            // ring stage and the parity of its current round
    uint32_t round = 0;
    auto step_ring = [&]() {
        if (++s == NS) {
            s = 0;
            round ^= 1;
        }
    };

    if (warp == kWarps) {
        // ================================================================ producer
        uint32_t bad = 0;
        int issued = 0;
        const int sel_shift = page_shift(p.page) - 4;
        const int spb = p.page < kBoxTokens ? p.page / kPageStep : kBoxTokens / kPageStep;   // steps of a box
        while (walk.next(&pc)) {
            const int32_t* row_table = a.s.table + (int64_t)pc.sq * a.s.max_pages;
            const int32_t* row_sel =
                a.n_sel < 0 ? nullptr : a.sel + (((int64_t)pc.l * a.s.A + pc.sq) * p.H + pc.h) * a.n_sel;
            const int64_t len = lens[pc.sq];
            Window win;
            uint32_t steps;
            if constexpr (WIN) {
                win = window_of(len, p.page, a.window, a.sinks);
                steps = window_steps(len, p.page, win);
            } else {
                steps = seq_steps(len, p.page, a.n_sel);
            }
            const int64_t unit_page = (int64_t)(a.s.layer0 + pc.l) * p.n_pages;
            const int64_t head_row = (unit_page * p.H + pc.h) * p.page;
            // lane j looks up step j of the next 32 / S chunks, one batch ahead
            int row = 0, next_row = 0;
            uint32_t mask = 0, next_mask = 0;
            float2 scale = make_float2(0.f, 0.f), next_scale = scale;
            auto look_up = [&](uint32_t st, int* r, uint32_t* m, float2* sc) {
                *r = 0;
                *m = 0;
                if (st < steps && st < pc.c1 * S) {
                    int slot, n;
                    int64_t lp;
                    uint32_t seen;
                    if constexpr (WIN) {
                        lp = window_page(st, p.page, win, len, &slot, &seen);
                    } else {
                        const int64_t choice = row_sel ? (int64_t)row_sel[st >> sel_shift] : 0;
                        lp = step_page(st, p.page, a.n_sel, choice, len, &slot, &n, &bad);
                        seen = (1u << n) - 1u;
                    }
                    const int64_t id = lp >= 0 && seen ? check_page(row_table[lp], p.n_pages, &bad) : -1;
                    if (id >= 0) {
                        *r = (int)(head_row + id * p.H * p.page + slot);   // fits: checked with the maps
                        *m = seen;
                        if constexpr (F::kScales)
                            *sc = __ldg(reinterpret_cast<const float2*>(p.scales) + (unit_page + id) * p.H + pc.h);
                    }
                }
            };
            look_up(pc.c0 * S + lane, &next_row, &next_mask, &next_scale);
            for (uint32_t c = pc.c0; c < pc.c1; ++c) {
                const int at = (int)((c - pc.c0) & (32 / S - 1)) * S;
                if (at == 0) {
                    row = next_row;
                    mask = next_mask;
                    scale = next_scale;
                    look_up((c + 32 / S) * S + lane, &next_row, &next_mask, &next_scale);
                }
                // lane j < S: step j of this chunk
                const int my_row = __shfl_sync(0xffffffffu, row, at + (lane & (S - 1)));
                const uint32_t my_mask = __shfl_sync(0xffffffffu, mask, at + (lane & (S - 1)));
                float2 my_scale;
                if constexpr (F::kScales) {
                    my_scale.x = __shfl_sync(0xffffffffu, scale.x, at + (lane & (S - 1)));
                    my_scale.y = __shfl_sync(0xffffffffu, scale.y, at + (lane & (S - 1)));
                }
                const uint32_t live = __ballot_sync(0xffffffffu, lane < S && my_mask != 0);
                const uint32_t loads = __popc(live);
                uint32_t info = my_mask << (16 * (lane & 1));
                info |= __shfl_xor_sync(0xffffffffu, info, 1);
                uint32_t high = 0;
                if constexpr (S == 4) high = __shfl_xor_sync(0xffffffffu, info, 2);
                const uint32_t full = tc::smem_u32(&sh.full[s]);
                if (issued >= NS) tc::mbar_wait(tc::smem_u32(&sh.empty[s]), round ^ 1u, abort, kWaitNs);
                ++issued;
                if (__all_sync(0xffffffffu, *abort == 0) && !stall) {
                    if constexpr (S == 4) {
                        if (lane == 0) *reinterpret_cast<uint2*>(sh.info[s]) = make_uint2(info, high);
                    } else {
                        if (lane < S && !(lane & 1)) sh.info[s][lane >> 1] = info;
                    }
                    if constexpr (F::kScales) {
                        if (lane < S) sh.scale[s][lane] = my_scale;
                        __syncwarp();
                    }
                    if (lane == 0) tc::mbar_arrive_expect_tx(full, loads * F::kStepBytes);
                    __syncwarp();
                    // one copy per box when all of the box's steps have tokens to see, else one per step that has
                    const uint32_t box = ((1u << spb) - 1u) << ((lane & (S - 1)) & ~(spb - 1));
                    const bool boxed = (live & box) == box;
                    if (lane < S && (boxed ? (lane & (spb - 1)) == 0 : my_mask != 0))
                        F::copy(ring_u + s * kStage, lane, boxed ? &maps.k_box : &maps.k_step, boxed ? &maps.v_box : &maps.v_step,
                                my_row, full);
                }
                __syncwarp();
                step_ring();
            }
        }
        if (bad && p.status) atomicOr(p.status, bad);
        // the producer stays until its copies have landed (each stage's last round), or, after a wait has given up
        // anywhere in the CTA, for 50 ms more
        const uint64_t t0 = tc::globaltimer();
        uint64_t limit = kWaitNs;
        for (int k = 0; k < NS && k < issued; ++k) {
            s = s == 0 ? NS - 1 : s - 1;
            if (s == NS - 1) round ^= 1;
            while (!tc::mbar_try(tc::smem_u32(&sh.full[s]), round)) {
                const uint64_t t = tc::globaltimer() - t0;
                if (limit == kWaitNs && *abort) limit = t + 50000000ull;
                if (t > limit) {
                    *abort = 1;
                    break;
                }
            }
        }
        if (*abort && p.status && lane == 0) atomicOr(p.status, kPagesTimeout);
        return;
    }

    // ==================================================================== consumers
    const int g = lane >> 2, t = lane & 3;
    const F fmt(g, t);
    int turn = 0;   // whose the next short unit is
    while (walk.next(&pc)) {
        bool mine = true;
        if (pc.solo) {
            mine = turn == warp;
            turn = (turn + 1) & (kWarps - 1);
        }
        const int rows = min(R, a.G - pc.rg * R);
        typename F::template Query<RT> query;
        if (mine)
            fmt.load(query, a.q + pc.l * a.qs.layer + pc.sq * a.qs.row + (int64_t)(pc.h * a.G + pc.rg * R) * a.qs.head, a.qs.head, rows);
        float m[RT], lsum[RT], o[RT][MT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            m[r] = -INFINITY;
            lsum[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[r][i][0] = o[r][i][1] = o[r][i][2] = o[r][i][3] = 0.0f;
        }
        for (uint32_t ch = pc.c0; ch < pc.c1; ++ch) {
            const bool ok = tc::mbar_wait(tc::smem_u32(&sh.full[s]), round, abort, kWaitNs);
            const bool live = __all_sync(0xffffffffu, ok);   // the warp converges before its matrix instructions
            // a short unit's owner takes all of the chunk's steps, otherwise each warp its own
            const int st0 = pc.solo ? 0 : warp, by = pc.solo ? 1 : kWarps, st1 = !live || (pc.solo && !mine) ? 0 : S;
            for (int st = st0; st < st1; st += by) {
                const uint32_t seen = reinterpret_cast<const uint16_t*>(sh.info[s])[st];
                if (seen == 0) continue;
                fmt.template step<RT>(ring + s * kStage, st, seen, sh.scale[s][st], a.scale_log2, query, m, lsum, o);
            }
            tc::fence_proxy_async();   // this thread's reads of the stage, before the copies that refill it
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.empty[s]));
            step_ring();
        }
        const int64_t out_row = ((int64_t)pc.l * a.s.A + pc.sq) * a.Hq + pc.h * a.G + pc.rg * R;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            lsum[r] += __shfl_xor_sync(0xffffffffu, lsum[r], 1);
            lsum[r] += __shfl_xor_sync(0xffffffffu, lsum[r], 2);
        }
        if (pc.solo) {   // the warp has the whole unit: its rows are finished in registers
            if (mine) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float L0 = __shfl_sync(0xffffffffu, lsum[r], 8 * t), L1 = __shfl_sync(0xffffffffu, lsum[r], 8 * t + 4);
                    const float M0 = __shfl_sync(0xffffffffu, m[r], 8 * t), M1 = __shfl_sync(0xffffffffu, m[r], 8 * t + 4);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 8 * r + 2 * t + e;
                        if (row < rows) {
#pragma unroll
                            for (int i = 0; i < MT; i += 2)
                                finish4<BF16>(a, out_row + row, D, F::col(g, i),
                                              make_float4(o[r][i][e], o[r][i][2 + e], o[r][i + 1][e], o[r][i + 1][2 + e]),
                                              e ? M1 : M0, e ? L1 : L0);
                        }
                    }
                }
            }
            continue;
        }
        // ---- the warps' partials, combined in shared memory, four rows at a time
        const bool whole = pc.c0 == 0 && pc.c1 == pc.n;
        const int slot = (int)blockIdx.x + (pc.c0 == 0 ? parts.ctas : 0);
        if (t == 0) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                sh.pm[warp][8 * r + g] = m[r];
                sh.pl[warp][8 * r + g] = lsum[r];
            }
        }
#pragma unroll
        for (int ps = 0; ps < R / kPassRows; ++ps) {
            if (ps * kPassRows >= rows) break;
            // rows 4 ps .. + 3 stand in the lanes with t = 2 (ps & 1) + {0, 1} of tile ps >> 1
            if (t >> 1 == (ps & 1)) {
                float* part = scratch + (warp * kPassRows + 2 * (t & 1)) * D;
#pragma unroll
                for (int i = 0; i < MT; i += 2) {
                    const int col = F::col(g, i);
                    const float(&x)[4] = o[ps >> 1][i];
                    const float(&y)[4] = o[ps >> 1][i + 1];
                    *reinterpret_cast<float4*>(part + col) = make_float4(x[0], x[2], y[0], y[2]);
                    *reinterpret_cast<float4*>(part + D + col) = make_float4(x[1], x[3], y[1], y[3]);
                }
            }
            tc::named_bar(1, kConsumers);
            for (int idx = tid; idx < min(kPassRows, rows - ps * kPassRows) * (D / 4); idx += kConsumers) {
                const int rr = idx / (D / 4), r = ps * kPassRows + rr, col = (idx - rr * (D / 4)) * 4;
                float M = sh.pm[0][r];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sh.pm[w][r]);
                float L = 0.0f;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    if (sh.pm[w][r] != -INFINITY || sh.pl[w][r] != 0.0f) {   // the second: only NaN logits
                        const float f = ex2a(sh.pm[w][r] - M);
                        const float4 y = *reinterpret_cast<const float4*>(scratch + (w * kPassRows + rr) * D + col);
                        L = fmaf(sh.pl[w][r], f, L);
                        v.x = fmaf(y.x, f, v.x);
                        v.y = fmaf(y.y, f, v.y);
                        v.z = fmaf(y.z, f, v.z);
                        v.w = fmaf(y.w, f, v.w);
                    }
                if (whole) {
                    finish4<BF16>(a, out_row + r, D, col, v, M, L);
                } else {
                    *reinterpret_cast<float4*>(parts.acc + (slot * R + r) * D + col) = v;
                    if (col == 0) parts.ml[slot * R + r] = make_float2(M, L);
                }
            }
            tc::named_bar(1, kConsumers);   // scratch and sums are written again
        }
        if (!whole) {
            const uint32_t c0 = shares.of(pc.u0);
            const int np = (int)(shares.of(pc.u0 + pc.n - 1) - c0) + 1;
            // the whole piece is written (the barrier above): one thread releases it and acquires the others'
            if (tid == 0) {
                uint32_t before;
                asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
                             : "=r"(before)
                             : "l"(ws_count + c0), "r"((uint32_t)np - 1)
                             : "memory");
                if (before == (uint32_t)np - 1) {
                    Join& x = sh.join[sh.joins++];   // at most two: the range's first and last unit
                    x.row = out_row;
                    x.c0 = c0;
                    x.np = np;
                    x.rows = rows;
                }
            }
        }
    }
    // ---- the units whose last piece arrived here
    tc::named_bar(1, kConsumers);
    for (int k = 0; k < sh.joins; ++k) {
        const Join x = sh.join[k];
        join_pieces<D, R, BF16>(a, parts, x.c0, x.np, x.row, x.rows, scratch);
    }
}

// The arrival counts come first: they are the part of the workspace that is zero between calls.
inline int grid_ctas(int per_sm) {
    const int n = device_sm_count() * per_sm;
    return n < kMaxCtas ? n : kMaxCtas;
}
struct WsLayout {
    size_t acc, ml, total;
};
inline WsLayout ws_layout(int nc, int R, int D) {
    WsLayout w;
    w.acc = kMaxCtas * sizeof(uint32_t);
    w.ml = w.acc + (size_t)2 * nc * R * D * sizeof(float);
    w.total = w.ml + (size_t)2 * nc * R * 2 * sizeof(float);
    return w;
}

// cuTensorMapEncodeTiled from the driver, looked up once (no link-time dependency on libcuda)
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// The cache as rows of `row_tokens` token slots, `cols` elements of `type` wide.
inline polykv_status make_maps(const PagesView& p, CUtensorMapDataType type, int cols, int row_tokens, int box_cols, int elem_bytes, PageMaps* m) {
    // token slots of all layers, pages and heads: below 2^31 for any cache that fits the card's memory
    const unsigned __int128 all = (unsigned __int128)p.L * p.n_pages * p.H * p.page;
    if (all >= ((unsigned __int128)1 << 31)) return set_error(POLYKV_E_UNSUPPORTED, "pages_attend: 2^31 or more token slots");
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return set_error(POLYKV_E_CUDA, "pages_attend: cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)all / row_tokens};
    const cuuint64_t strides[1] = {(cuuint64_t)cols * elem_bytes};
    const cuuint32_t estr[2] = {1, 1};
    const int box_tokens = p.page < kBoxTokens ? p.page : kBoxTokens;
    struct { CUtensorMap* map; void* base; int rows; } want[4] = {
        {&m->k_box, p.k, box_tokens / row_tokens}, {&m->v_box, p.v, box_tokens / row_tokens},
        {&m->k_step, p.k, kPageStep / row_tokens}, {&m->v_step, p.v, kPageStep / row_tokens}};
    for (auto& w : want) {
        const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)w.rows};
        const CUresult r = enc(w.map, type, 2, w.base, dims, strides, box, estr,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) return set_error(POLYKV_E_CUDA, "pages_attend: tensor map encode failed (%d)", (int)r);
    }
    return POLYKV_OK;
}

template <class F, int RT>
polykv_status run(const PagesAttendArgs& a, const PageMaps& maps, void* ws, cudaStream_t st) {
    constexpr int R = 8 * RT;
    constexpr int D = F::D;
    auto kern = a.window > 0 ? pages_attend_kernel<F, RT, true> : pages_attend_kernel<F, RT, false>;
    const WsLayout w = ws_layout(grid_ctas(kMaxPerSm), R, D);
    char* base = static_cast<char*>(ws);
    // as many stages as let per_sm CTAs share an SM's 228 KB (1 KB of each is the system's)
    constexpr size_t most = 233472 / F::per_sm(RT) - 1024;
    const size_t extra = 1024 + scratch_bytes<D>() + sizeof(Shared) + (size_t)(2 * a.s.A + 1) * sizeof(uint32_t);
    const int fit = (int)((most - extra) / F::kStage);
    const int NS = fit < kMaxStages ? fit : kMaxStages;
    const size_t smem = extra + (size_t)NS * F::kStage;
    // the limit stands for the process: always the same, whatever this call needs, so that calls of other sizes from other
    // host threads do not lower it before the launch
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_attend: smem attribute: %s", cudaGetErrorString(e));
    // Test hook for the bounded waits: POLYKV_TEST_STALL=1 makes the producer copy nothing.
    const char* env = getenv("POLYKV_TEST_STALL");
    const bool stall = env && env[0] == '1';
    const Partials parts = {reinterpret_cast<float*>(base + w.acc), reinterpret_cast<float2*>(base + w.ml),
                            grid_ctas(F::per_sm(RT))};
    e = launch_after(kern, dim3((unsigned)parts.ctas), kThreads, smem, st, a, maps, NS, reinterpret_cast<uint32_t*>(base),
                     parts, stall);
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_attend launch: %s", cudaGetErrorString(e));
    return POLYKV_OK;
}

}  // namespace attend

struct PagesTma {   // made at the first attention call (it needs the driver)
    std::mutex mu;
    bool made = false;
    attend::PageMaps maps;
};

// The tensor maps of a 16-bit cache.
polykv_status pages_wide_maps(const PagesView& p, const attend::PageMaps** maps);

polykv_status launch_pages_attend8(const PagesAttendArgs& a, polykv_dtype dt, void* ws, cudaStream_t st);

}  // namespace polykv
