// Attention of one new token per sequence over a paged key-value cache.
//
//   out[l][a][hq] = sum_t softmax_t(scale q . k_t) v_t     over the sequence's tokens t < lens[a], or over
//                                                          those in its chosen pages; zeros if there are none
//
// Query head hq reads kv head hq / G. The keys and values of a sequence stand in pages of 16..128 tokens,
// each (layer, page, kv head) one contiguous [page][d] block, found through the sequence's block table.
//
// The work is one pass over K and V (one per 16 query heads of a kv head): 4 G d flop for 4 d bytes per token and
// kv head, so HBM binds it, and streaming at its rate takes about 190 KB in flight per SM: more than the registers
// hold. Each CTA is a producer warp that keeps a ring of 64-token chunks in shared memory filled by tensor copies
// (the 128-byte swizzle makes the consumers' fragment reads free of bank conflicts), and four consumer warps that
// take 16 tokens of a chunk each, on m16n8k16 matrix instructions (f16 values: m16n8k8 in tf32, for its exponents)
// with the softmax in registers. The producer runs ahead over the ends of units (one layer, sequence, head), so
// joining warps and starting units costs no bandwidth.
//
// The list of all (layer, sequence, head, chunk) items is cut into one contiguous range per CTA, from the
// lengths on the device: ragged batches and one long sequence spread alike, and a captured graph stays right
// when the lengths change. A range that starts or ends inside a unit leaves a softmax partial (running
// maximum, sum, unnormalised accumulator) in the workspace; the CTA that finishes a unit's last outstanding
// piece (an arrival count per unit, which wraps back to zero) joins its pieces in the order of the ranges,
// so results do not depend on timing and one launch does it all.
//
// Measured (bf16, 8 kv heads x 4 query heads, d = 128): one sequence of 131,071 tokens 86.3 us = 6.2 TB/s; 256 ragged
// sequences, 204 k tokens, 132 us = 6.3 TB/s; 15 x about 3,800 tokens 43.0 us = 5.4 TB/s; the chunks stream at 7 TB/s,
// and about 8 us go to finding the work (4 dependent loads), the last chunk, the release of the pieces and the join.
// f16 beside bf16, captured calls back to back: 93 and 92.5 us for the first, 111 and 108 us for 500 MB of 16 query heads a
// kv head (two row tiles, spilled registers); with f16's probabilities in f16, too short a range, 91 and 104 us.
// The same loop with K and V loaded into registers (12 warps an SM, 96 KB in flight) took 108 us for the first.
//
// Every wait is bounded (2 s): then the CTA's waits return at once, its loops run to their end so that
// barriers stay matched, the producer waits for its copies in flight, and the status word says so.
#include <cmath>
#include <cstdlib>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "pages_internal.cuh"
#include "tc_ptx.cuh"

namespace polykv {
namespace {

constexpr int kWarps = 4;                    // consumer warps
constexpr int kConsumers = 32 * kWarps;
constexpr int kThreads = kConsumers + 32;    // and the producer
constexpr int kChunkSteps = kWarps;          // 16-token steps of a chunk
constexpr int kChunkTokens = kChunkSteps * kPageStep;
constexpr int kMaxPerSm = 3;                 // CTAs per SM that the workspace is sized for
constexpr int kMaxCtas = 1024;
constexpr int kMaxStages = 8;
constexpr int kPassRows = 4;                 // rows that the warps join at once
constexpr int kJoinPieces = 128;             // pieces whose weights stand in shared memory at once
constexpr uint64_t kWaitNs = 2000000000ull;
// What starting a unit costs, in chunks: finding its pages and query, and joining the warps. It stands as
// virtual items before the unit's chunks in the work list, so that ranges full of short units hold fewer.
constexpr uint32_t kUnitCost = 2;
// Units of at most this many chunks are not cut: leaving pieces and joining them costs about 3 us, a chunk half one
// (15 pages of 16 tokens for each of 160 units: 12.5 us cut, 9.3 us whole).
constexpr uint32_t kWhole = 5;
// A whole unit of at most this many chunks is left to one consumer warp, so that four of them go at once.
constexpr uint32_t kShort = 2;
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

template <bool BF16>
__device__ __forceinline__ uint32_t pack_rn(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&w));
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
            const uint32_t n = seq_steps(len, a.p.page, a.n_sel);
            lens[i] = (int32_t)len;
            pre[i] = sum;
            sum += n ? (n + kChunkSteps - 1) / kChunkSteps + kUnitCost : 0;
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
struct Walk {
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
            if (p->n <= kWhole) {   // whole, in the range that holds its first item
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
                p->solo = p->c0 == 0 && p->c1 == p->n && p->n <= kShort;
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
constexpr int stage_bytes() { return 2 * kChunkTokens * D * 2; }   // a chunk's keys and values
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
    uint32_t info[kMaxStages];   // tokens of each of the chunk's steps, a byte each
    float pm[kWarps][16], pl[kWarps][16];
    uint32_t wsum[kThreads / 32];
    Join join[2];
    int joins, abort;
};

// Resident CTAs per SM: by the ring, about 190 KB an SM in stages of 32 KB (d = 128) or 16 KB.
template <int D>
constexpr int per_sm() { return D == 64 ? 3 : 2; }

// RT row tiles of 8 query heads: 1 for units of up to 8, 2 for up to 16.
template <int D, int RT, bool BF16>
__global__ void __launch_bounds__(kThreads, per_sm<D>())
    pages_attend_kernel(const __grid_constant__ PagesAttendArgs a, const __grid_constant__ PageMaps maps, const int NS,
                        uint32_t* __restrict__ ws_count, const __grid_constant__ Partials parts, const bool stall) {
    constexpr int KS = D / 16;      // score k-steps
    constexpr int MT = D / 16;      // value m-tiles
    constexpr int HV = D / 64;      // 64-column halves of a row
    constexpr int R = 8 * RT;
    constexpr int TERMS = BF16 ? 3 : 2;   // parts that a probability is split into (below)
    constexpr int PW = BF16 ? 2 : 4;      // words of a part of a lane's four probabilities
    constexpr int kHalf = kChunkTokens * 128;   // bytes of 64 columns of a chunk
    constexpr int kStage = stage_bytes<D>();
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
    scan_items(a, pre, lens, sh.wsum, blockIdx.x == 0);
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
    Walk walk(pre, a.s.A, p.H, RG, shares.first(blockIdx.x), shares.first(blockIdx.x + 1));
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
        const int spb = p.page < 64 ? p.page / kPageStep : kChunkSteps;   // steps of a box
        while (walk.next(&pc)) {
            const int32_t* row_table = a.s.table + (int64_t)pc.sq * a.s.max_pages;
            const int32_t* row_sel =
                a.n_sel < 0 ? nullptr : a.sel + (((int64_t)pc.l * a.s.A + pc.sq) * p.H + pc.h) * a.n_sel;
            const int64_t len = lens[pc.sq];
            const uint32_t steps = seq_steps(len, p.page, a.n_sel);
            const int64_t head_row = ((int64_t)(a.s.layer0 + pc.l) * p.n_pages * p.H + pc.h) * p.page;
            // lane j looks up step j of the next eight chunks, one batch ahead
            int row = 0, valid = 0, next_row = 0, next_valid = 0;
            auto look_up = [&](uint32_t st, int* r, int* v) {
                *v = *r = 0;
                if (st < steps && st < pc.c1 * kChunkSteps) {
                    const int64_t choice = row_sel ? (int64_t)row_sel[st >> sel_shift] : 0;
                    int slot, n;
                    const int64_t lp = step_page(st, p.page, a.n_sel, choice, len, &slot, &n, &bad);
                    const int64_t id = lp >= 0 ? check_page(row_table[lp], p.n_pages, &bad) : -1;
                    if (id >= 0) {
                        *r = (int)(head_row + id * p.H * p.page + slot);   // fits: checked with the maps
                        *v = n;
                    }
                }
            };
            look_up(pc.c0 * kChunkSteps + lane, &next_row, &next_valid);
            for (uint32_t c = pc.c0; c < pc.c1; ++c) {
                const int at = (int)((c - pc.c0) & 7) * kChunkSteps;
                if (at == 0) {
                    row = next_row;
                    valid = next_valid;
                    look_up((c + 8) * kChunkSteps + lane, &next_row, &next_valid);
                }
                // lane j < 4: step j of this chunk
                const int my_row = __shfl_sync(0xffffffffu, row, at + (lane & 3));
                const int my_valid = __shfl_sync(0xffffffffu, valid, at + (lane & 3));
                const int last_valid = __shfl_sync(0xffffffffu, my_valid, (lane & 3) | (spb - 1));
                const uint32_t loads = __popc(__ballot_sync(0xffffffffu, lane < kChunkSteps && my_valid > 0));
                uint32_t info = (uint32_t)my_valid << (8 * (lane & 3));
                info |= __shfl_xor_sync(0xffffffffu, info, 1);
                info |= __shfl_xor_sync(0xffffffffu, info, 2);
                const uint32_t full = tc::smem_u32(&sh.full[s]);
                if (issued >= NS) tc::mbar_wait(tc::smem_u32(&sh.empty[s]), round ^ 1u, abort, kWaitNs);
                ++issued;
                if (__all_sync(0xffffffffu, *abort == 0) && !stall) {
                    if (lane == 0) {
                        sh.info[s] = info;
                        tc::mbar_arrive_expect_tx(full, loads * (kPageStep * D * 4));
                    }
                    __syncwarp();
                    // one copy per box when all of the box's steps have tokens, else one per step that has
                    const bool boxed = last_valid > 0;
                    if (lane < kChunkSteps && (boxed ? (lane & (spb - 1)) == 0 : my_valid > 0)) {
                        const uint32_t dst = ring_u + s * kStage + lane * (kPageStep * 128);
                        const void* km = boxed ? &maps.k_box : &maps.k_step;
                        const void* vm = boxed ? &maps.v_box : &maps.v_step;
#pragma unroll
                        for (int hf = 0; hf < HV; ++hf) {
                            tc::tma_2d_g2s(dst + hf * kHalf, km, 64 * hf, my_row, full);
                            tc::tma_2d_g2s(dst + (HV + hf) * kHalf, vm, 64 * hf, my_row, full);
                        }
                    }
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
    // This lane's 16-byte chunks in the swizzled tiles (chunk j of row r stands at j ^ (r & 7)): keys of tokens
    // 8 jj + g, columns 64 hf + 16t + 8c .. + 8; values of tokens {2t, 2t+1, 2t+8, 2t+9}, columns 64 hf + 8g .. + 8
    const int k_at[2] = {g * 128 + ((2 * t) ^ g) * 16, g * 128 + ((2 * t + 1) ^ g) * 16};
    const int v_at[2] = {2 * t * 128 + (g ^ (2 * t)) * 16, (2 * t + 1) * 128 + (g ^ (2 * t + 1)) * 16};
    int turn = 0;   // whose the next short unit is
    while (walk.next(&pc)) {
        bool mine = true;
        if (pc.solo) {
            mine = turn == warp;
            turn = (turn + 1) & (kWarps - 1);
        }
        const int rows = min(R, a.G - pc.rg * R);
        // queries: the k-steps of chunk (hf, c) take its words {0, 1} and {2, 3}
        uint32_t qa[KS][2 * RT];
        if (mine) {
            const uint16_t* qb =
                a.q + pc.l * a.qs.layer + pc.sq * a.qs.row + (int64_t)(pc.h * a.G + pc.rg * R) * a.qs.head;
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < 2 * HV; ++c) {
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if (8 * r + g < rows)
                        w = __ldg(reinterpret_cast<const uint4*>(qb + (8 * r + g) * a.qs.head + 64 * (c >> 1) + 16 * t +
                                                                 8 * (c & 1)));
                    qa[2 * c][r] = w.x;
                    qa[2 * c][RT + r] = w.y;
                    qa[2 * c + 1][r] = w.z;
                    qa[2 * c + 1][RT + r] = w.w;
                }
        }
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
            const uint32_t info = live ? sh.info[s] : 0u;
            // a short unit's owner takes all of the chunk's steps, otherwise each warp its own
            const int st0 = pc.solo ? 0 : warp, st1 = pc.solo ? (mine ? kChunkSteps : 0) : warp + 1;
            for (int st = st0; st < st1; ++st) {
                const int now = (int)(info >> (8 * st)) & 0xff;
                if (now == 0) continue;
                const unsigned char* kt = ring + s * kStage + st * (kPageStep * 128);
                const unsigned char* vt = kt + HV * kHalf;
                // scores of rows g (and g + 8) for tokens 8 jj + 2t + {0, 1}, 64 columns at a time
                float sc[2][4];
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) sc[jj][0] = sc[jj][1] = sc[jj][2] = sc[jj][3] = 0.0f;
#pragma unroll
                for (int hf = 0; hf < HV; ++hf)
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        uint4 kw[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            kw[c] = *reinterpret_cast<const uint4*>(kt + hf * kHalf + jj * 1024 + k_at[c]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t b0 = word_of(kw[k >> 1], 2 * (k & 1)), b1 = word_of(kw[k >> 1], 2 * (k & 1) + 1);
                            const uint32_t(&qk)[2 * RT] = qa[4 * hf + k];
                            if constexpr (RT == 1) mma<BF16>(sc[jj], qk[0], 0u, qk[1], 0u, b0, b1);
                            else mma<BF16>(sc[jj], qk[0], qk[1], qk[2], qk[3], b0, b1);
                        }
                    }
                if (now < kPageStep) {   // slots behind the last token hold anything: keep them out of the softmax
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((e >> 1) * 8 + 2 * t + (e & 1) >= now) {
#pragma unroll
                            for (int r = 0; r < RT; ++r) sc[e >> 1][2 * r + (e & 1)] = -INFINITY;
                        }
                }
                uint32_t pf[RT][TERMS][PW];
                float a0[RT], a1[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    float xx[4], mx = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        xx[e] = sc[e >> 1][2 * r + (e & 1)] * a.scale_log2;
                        mx = fmaxf(mx, xx[e]);
                    }
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float mn = fmaxf(m[r], mx);
                    const float ms = mn == -INFINITY ? 0.0f : mn;
                    const float alpha = ex2a(m[r] - ms);
                    m[r] = mn;
                    float pr[4], ps = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        pr[e] = ex2a(xx[e] - ms);
                        ps += pr[e];
                    }
                    lsum[r] = fmaf(lsum[r], alpha, ps);
                    // accumulator rows 2t and 2t + 1 belong to lane quads 2t and 2t + 1
                    a0[r] = __shfl_sync(0xffffffffu, alpha, 8 * t);
                    a1[r] = __shfl_sync(0xffffffffu, alpha, 8 * t + 4);
                    // The probabilities enter the value product as a sum of parts, each the rounding of what the parts
                    // before left: 3 x 8 bits in bf16 beside bf16 values, 2 x 11 bits in tf32 beside f16 values (which
                    // tf32 holds as they are). Both have fp32's exponents, so that a probability keeps its accuracy
                    // however far it is below the largest; parts in f16 would end at 2^-25 of that, and a long
                    // context's many small ones would go missing from the values but not from the sum.
#pragma unroll
                    for (int k = 0; k < TERMS; ++k) {
                        if constexpr (BF16) {
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                pf[r][k][b] = pack_rn<BF16>(pr[2 * b], pr[2 * b + 1]);
                                const float2 f = unpack2<BF16>(pf[r][k][b]);
                                pr[2 * b] -= f.x;
                                pr[2 * b + 1] -= f.y;
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                pf[r][k][e] = to_tf32(pr[e]);
                                pr[e] -= __uint_as_float(pf[r][k][e]);
                            }
                        }
                    }
                }
                // m-tile i: A rows g and g + 8 are columns 64 (i >> 2) + 8g + 2 (i & 3) + {0, 1}. The matrix unit's
                // sums are cut off rather than rounded, so a step's product starts from zero (small parts first)
                // and joins the accumulator by a rounded fused multiply-add; a sum run through the unit over a
                // long context would lose about half a bit per step in one direction.
#pragma unroll
                for (int hf = 0; hf < HV; ++hf) {
                    uint4 vw[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        vw[e] = *reinterpret_cast<const uint4*>(vt + hf * kHalf + (e >> 1) * 1024 + v_at[e & 1]);
                    if (now < kPageStep) {   // nor may they meet a probability of zero
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if ((e >> 1) * 8 + 2 * t + (e & 1) >= now) vw[e] = make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t w0 = word_of(vw[0], k), w1 = word_of(vw[1], k);
                        const uint32_t w2 = word_of(vw[2], k), w3 = word_of(vw[3], k);
                        // tf32: tokens 2t and 2t + 1 are columns t and t + 4 of the first product, 2t + 8 and 2t + 9 of
                        // the second, as in this lane's probabilities
                        uint32_t f0, f1, f2, f3;
                        float2 x0, x1, x2, x3;
                        if constexpr (BF16) {
                            f0 = prmt(w0, w1, 0x5410u), f1 = prmt(w0, w1, 0x7632u);
                            f2 = prmt(w2, w3, 0x5410u), f3 = prmt(w2, w3, 0x7632u);
                        } else {
                            x0 = unpack2<BF16>(w0), x1 = unpack2<BF16>(w1);
                            x2 = unpack2<BF16>(w2), x3 = unpack2<BF16>(w3);
                        }
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                            for (int j = TERMS - 1; j >= 0; --j) {
                                if constexpr (BF16) {
                                    mma<BF16>(d, f0, f1, f2, f3, pf[r][j][0], pf[r][j][1]);
                                } else {
                                    mma_tf32(d, x0.x, x0.y, x1.x, x1.y, pf[r][j][0], pf[r][j][1]);
                                    mma_tf32(d, x2.x, x2.y, x3.x, x3.y, pf[r][j][2], pf[r][j][3]);
                                }
                            }
                            float(&acc)[4] = o[r][4 * hf + k];
                            acc[0] = fmaf(acc[0], a0[r], d[0]);
                            acc[1] = fmaf(acc[1], a1[r], d[1]);
                            acc[2] = fmaf(acc[2], a0[r], d[2]);
                            acc[3] = fmaf(acc[3], a1[r], d[3]);
                        }
                    }
                }
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
                                finish4<BF16>(a, out_row + row, D, 64 * (i >> 2) + 8 * g + 2 * (i & 3),
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
                float* part = scratch + (warp * kPassRows + 2 * (t & 1)) * D + 8 * g;
#pragma unroll
                for (int i = 0; i < MT; i += 2) {
                    const int col = 64 * (i >> 2) + 2 * (i & 3);
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
int grid_ctas(int per_sm) {
    const int n = device_sm_count() * per_sm;
    return n < kMaxCtas ? n : kMaxCtas;
}
struct WsLayout {
    size_t acc, ml, total;
};
WsLayout ws_layout(int nc, int R, int D) {
    WsLayout w;
    w.acc = kMaxCtas * sizeof(uint32_t);
    w.ml = w.acc + (size_t)2 * nc * R * D * sizeof(float);
    w.total = w.ml + (size_t)2 * nc * R * 2 * sizeof(float);
    return w;
}

// cuTensorMapEncodeTiled from the driver, looked up once (no link-time dependency on libcuda)
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
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

polykv_status make_maps(const PagesView& p, PageMaps* m) {
    // token slots of all layers, pages and heads: below 2^31 for any cache that fits the card's memory
    const unsigned __int128 all = (unsigned __int128)p.L * p.n_pages * p.H * p.page;
    if (all >= ((unsigned __int128)1 << 31)) return set_error(POLYKV_E_UNSUPPORTED, "pages_attend: 2^31 or more token slots");
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return set_error(POLYKV_E_CUDA, "pages_attend: cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[2] = {(cuuint64_t)p.d, (cuuint64_t)all};
    const cuuint64_t strides[1] = {(cuuint64_t)p.d * 2};
    const cuuint32_t estr[2] = {1, 1};
    struct { CUtensorMap* map; void* base; int rows; } want[4] = {
        {&m->k_box, p.k, p.page < kChunkTokens ? p.page : kChunkTokens}, {&m->v_box, p.v, p.page < kChunkTokens ? p.page : kChunkTokens},
        {&m->k_step, p.k, kPageStep}, {&m->v_step, p.v, kPageStep}};
    for (auto& w : want) {
        const cuuint32_t box[2] = {64, (cuuint32_t)w.rows};
        const CUresult r = enc(w.map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, w.base, dims, strides, box, estr,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) return set_error(POLYKV_E_CUDA, "pages_attend: tensor map encode failed (%d)", (int)r);
    }
    return POLYKV_OK;
}

template <int D, int RT, bool BF16>
polykv_status run(const PagesAttendArgs& a, const PageMaps& maps, void* ws, cudaStream_t st) {
    constexpr int R = 8 * RT;
    auto kern = pages_attend_kernel<D, RT, BF16>;
    const WsLayout w = ws_layout(grid_ctas(kMaxPerSm), R, D);
    char* base = static_cast<char*>(ws);
    // as many stages as let per_sm CTAs share an SM's 228 KB (1 KB of each is the system's)
    constexpr size_t most = 233472 / per_sm<D>() - 1024;
    const size_t extra = 1024 + scratch_bytes<D>() + sizeof(Shared) + (size_t)(2 * a.s.A + 1) * sizeof(uint32_t);
    const int fit = (int)((most - extra) / stage_bytes<D>());
    const int NS = fit < kMaxStages ? fit : kMaxStages;
    const size_t smem = extra + (size_t)NS * stage_bytes<D>();
    // the limit stands for the process: always the same, whatever this call needs, so that calls of other sizes from other
    // host threads do not lower it before the launch
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_attend: smem attribute: %s", cudaGetErrorString(e));
    // Test hook for the bounded waits: POLYKV_TEST_STALL=1 makes the producer copy nothing.
    const char* env = getenv("POLYKV_TEST_STALL");
    const bool stall = env && env[0] == '1';
    const Partials parts = {reinterpret_cast<float*>(base + w.acc), reinterpret_cast<float2*>(base + w.ml),
                            grid_ctas(per_sm<D>())};
    e = launch_after(kern, dim3((unsigned)parts.ctas), kThreads, smem, st, a, maps, NS, reinterpret_cast<uint32_t*>(base),
                     parts, stall);
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_attend launch: %s", cudaGetErrorString(e));
    return POLYKV_OK;
}

}  // namespace

struct PagesTma {   // made at the first attention call (it needs the driver)
    std::mutex mu;
    bool made = false;
    PageMaps maps;
};
PagesTma* pages_tma_new() { return new (std::nothrow) PagesTma; }
void pages_tma_free(PagesTma* t) { delete t; }

size_t pages_attend_workspace(const PagesView& p, int G) {
    return ws_layout(grid_ctas(kMaxPerSm), G <= 8 ? 8 : 16, p.d).total;
}

polykv_status launch_pages_attend(const PagesAttendArgs& a, polykv_dtype dt, void* ws, cudaStream_t st) {
    {
        std::lock_guard<std::mutex> lock(a.p.tma->mu);
        if (!a.p.tma->made) {
            const polykv_status s = make_maps(a.p, &a.p.tma->maps);
            if (s != POLYKV_OK) return s;
            a.p.tma->made = true;
        }
    }
    const PageMaps& m = a.p.tma->maps;
    const bool bf = dt == POLYKV_BF16;
    if (a.p.d == 128) {
        if (a.G <= 8) return bf ? run<128, 1, true>(a, m, ws, st) : run<128, 1, false>(a, m, ws, st);
        return bf ? run<128, 2, true>(a, m, ws, st) : run<128, 2, false>(a, m, ws, st);
    }
    if (a.G <= 8) return bf ? run<64, 1, true>(a, m, ws, st) : run<64, 1, false>(a, m, ws, st);
    return bf ? run<64, 2, true>(a, m, ws, st) : run<64, 2, false>(a, m, ws, st);
}

}  // namespace polykv
