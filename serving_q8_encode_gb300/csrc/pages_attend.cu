// Attention of one new token per sequence over a paged key-value cache.
//
//   out[l][a][hq] = sum_t softmax_t(scale q . k_t) v_t     over the sequence's tokens t < lens[a], or over
//                                                          those in its chosen pages; zeros if there are none
//
// Query head hq reads kv head hq / G. The keys and values of a sequence stand in pages of 16..128 tokens,
// each (layer, page, kv head) one contiguous [page][d] block, found through the sequence's block table.
//
// The work is one pass over K and V: 4 G d flop for 4 d bytes per token and kv head, so HBM binds it. The
// list of all (layer, sequence, head, 16-token step) items is cut into one contiguous range per CTA, from
// the lengths on the device: ragged batches and one long sequence spread alike, and a captured graph stays
// right when the lengths change. A range that starts or ends inside a unit (one layer, sequence, head)
// leaves a softmax partial (running maximum, sum, unnormalised accumulator) in the workspace; the CTA that
// finishes a unit's last outstanding piece (an arrival count per unit, which wraps back to zero) joins its
// pieces in the order of the ranges, so results do not depend on timing and one launch does it all.
#include <cmath>

#include "pages_internal.cuh"

namespace polykv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMinItems = 8;   // a CTA's least share

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
    } else if (col == 0) {
        *reinterpret_cast<float2*>(a.ml + 2 * row) = make_float2(M, L);
    }
    store_out<BF16>(a, row, D, col, v);
}

// What starting a unit costs, in steps: finding its pages and query, and joining the warps. It stands as
// virtual items before the unit's steps in the work list, so that ranges full of short units hold fewer.
constexpr uint32_t kUnitCost = 6;
// A whole unit of at most this many steps is left to one warp; its CTA takes as many of them at once.
constexpr uint32_t kShort = 8;

// The sequences' items (steps and unit cost) as a running sum in shared memory: pre[a] stand before sequence a.
__device__ __forceinline__ void scan_steps(const PagesAttendArgs& a, uint32_t* pre, uint32_t* wsum, bool report) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.s.A + kThreads - 1) / kThreads;
    const int i0 = tid * per, i1 = min(a.s.A, i0 + per);
    uint32_t sum = 0, bad = 0;
    for (int i = i0; i < i1; ++i) {
        const uint32_t n = seq_steps(clamp_len(a.s.lens[i], a.s.max_pages, a.p.page, &bad), a.p.page, a.n_sel);
        pre[i] = sum;
        sum += n ? n + kUnitCost : 0;
    }
    if (bad && report && a.p.status) atomicOr(a.p.status, bad);
    uint32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    uint32_t base = inc - sum;
    for (int w = 0; w < warp; ++w) base += wsum[w];
    for (int i = i0; i < i1; ++i) pre[i] += base;
    if (i1 == a.s.A && i0 < i1) pre[a.s.A] = base + sum;
    __syncthreads();
}

// Joins the pieces [0, np) of one cut unit: piece 0 in slot 2 c0 + 1, piece i in slot 2 (c0 + i). Four columns
// of a row per thread; a row's pieces are shared out over the CTA's thread groups. R * D floats of scratch.
template <int D, int R, bool BF16>
__device__ void join_pieces(const PagesAttendArgs& a, const float* ws_acc, const float* ws_ml, uint32_t c0, int np,
                            int64_t out_row, int rows, float* scratch, float2* scratch_ml) {
    constexpr int TPR = D / 4;              // threads per row
    constexpr int NG = kThreads / TPR;      // thread groups: 4 (D = 128) or 8
    const int grp = threadIdx.x / TPR, ln = threadIdx.x - grp * TPR, col = 4 * ln;
    int rp = 1;
    while (rp < rows && rp < NG) rp <<= 1;  // rows in flight
    const int parts = NG / rp;
    for (int r0 = 0; r0 < rows; r0 += rp) {
        const int r = r0 + grp % rp, part = grp / rp;
        float M = -INFINITY, L = 0.0f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
#pragma unroll 4
            for (int i = part; i < np; i += parts) {
                const int64_t at = (2 * ((int64_t)c0 + i) + (i == 0 ? 1 : 0)) * R + r;
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(ws_ml + 2 * at));
                const float4 y = __ldcg(reinterpret_cast<const float4*>(ws_acc + at * D + col));
                const float mn = fmaxf(M, ml.x), ms = mn == -INFINITY ? 0.0f : mn;
                const float f = ex2a(M - ms), w = ex2a(ml.x - ms);
                M = mn;
                L = fmaf(ml.y, w, L * f);
                v.x = fmaf(y.x, w, v.x * f);
                v.y = fmaf(y.y, w, v.y * f);
                v.z = fmaf(y.z, w, v.z * f);
                v.w = fmaf(y.w, w, v.w * f);
            }
        }
        *reinterpret_cast<float4*>(scratch + grp * D + col) = v;
        if (ln == 0) scratch_ml[grp] = make_float2(M, L);
        __syncthreads();
        if (part == 0 && r < rows) {
            for (int k = 1; k < parts; ++k) {
                const float2 ml = scratch_ml[grp + k * rp];
                const float4 y = *reinterpret_cast<const float4*>(scratch + (grp + k * rp) * D + col);
                const float mn = fmaxf(M, ml.x), ms = mn == -INFINITY ? 0.0f : mn;
                const float f = ex2a(M - ms), w = ex2a(ml.x - ms);
                M = mn;
                L = fmaf(ml.y, w, L * f);
                v.x = fmaf(y.x, w, v.x * f);
                v.y = fmaf(y.y, w, v.y * f);
                v.z = fmaf(y.z, w, v.z * f);
                v.w = fmaf(y.w, w, v.w * f);
            }
            finish4<BF16>(a, out_row + r, D, col, v, M, L);
        }
        __syncthreads();
    }
}

// RT row tiles of 8 query heads: 1 for units of up to 8, 2 for up to 16.
// Resident CTAs per SM, by registers: a step's keys and values and the accumulators are D (1 + RT) of them.
constexpr int kMaxPerSm = 4;
template <int D, int RT>
constexpr int per_sm() { return D == 64 ? (RT == 1 ? 4 : 3) : (RT == 1 ? 3 : 2); }

template <int D, int RT, bool BF16>
__global__ void __launch_bounds__(kThreads, per_sm<D, RT>())
    pages_attend_kernel(const PagesAttendArgs a, uint32_t* __restrict__ ws_count, float* __restrict__ ws_acc,
                        float* __restrict__ ws_ml) {
    constexpr int KS = D / 16;      // score k-steps
    constexpr int MT = D / 16;      // value m-tiles
    constexpr int KC = D / 32;      // 16-byte key chunks per lane and token
    constexpr int VC = D / 64;      // 16-byte value chunks per lane and token
    constexpr int R = 8 * RT;
    constexpr int TERMS = BF16 ? 3 : 2;   // parts that a probability is split into (below)
    extern __shared__ uint32_t pre[];
    __shared__ __align__(16) float pacc[kWarps][R][D];
    __shared__ float pm[kWarps][R], pl[kWarps][R];
    __shared__ float2 jml[kThreads / (D / 4)];
    __shared__ uint32_t wsum[kWarps];
    __shared__ int last_here;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const PagesView& p = a.p;
    const int RG = (a.G + R - 1) / R;   // row groups per kv head
    const uint32_t HR = (uint32_t)(p.H * RG);

    scan_steps(a, pre, wsum, blockIdx.x == 0);
    const uint32_t S = pre[a.s.A];
    const uint64_t total = (uint64_t)a.s.nl * HR * S;
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

    uint64_t x = share(total, blockIdx.x, nc);
    const uint64_t xe = share(total, blockIdx.x + 1, nc);
    uint32_t bad = 0;
    // the unit that holds item x: layer ul, sequence usq, head index uhr (kv head and row group)
    int ul, usq, uhr;
    uint32_t i0;                        // item within the unit
    {
        const uint64_t per_layer = (uint64_t)HR * S;
        ul = per_layer ? (int)(x / per_layer) : 0;
        const uint64_t rem = x - (uint64_t)ul * per_layer;
        int lo = 0, hi = a.s.A - 1;
        while (lo < hi) {   // the last sequence with pre * HR <= rem (it has steps)
            const int mid = (lo + hi + 1) >> 1;
            if ((uint64_t)pre[mid] * HR <= rem) lo = mid;
            else hi = mid - 1;
        }
        usq = lo;
        const uint64_t in_seq = rem - (uint64_t)pre[usq] * HR;
        const uint32_t items = max(1u, pre[usq + 1] - pre[usq]);
        uhr = (int)(in_seq / items);
        i0 = (uint32_t)(in_seq - (uint64_t)uhr * items);
    }
    auto advance = [&]() {   // to the next unit
        if (++uhr == (int)HR) {
            uhr = 0;
            do {
                if (++usq == a.s.A) {
                    usq = 0;
                    ++ul;
                }
            } while (pre[usq + 1] == pre[usq]);
        }
    };
    while (x < xe) {
        uint32_t items = pre[usq + 1] - pre[usq];
        uint32_t i1 = xe - x < (uint64_t)(items - i0) ? i0 + (uint32_t)(xe - x) : items;
        int l = ul, sq = usq, hr = uhr;
        const uint64_t u0 = x - i0 + kUnitCost;   // the unit's first step in the list
        bool solo = false, mine = true;           // solo: each warp has a whole short unit (or none) for itself
        if (i0 == 0 && i1 == items && items <= kShort + kUnitCost) {
            solo = true;
            mine = false;
            for (int w = 0; w < kWarps; ++w) {    // the next units, as long as they are short and whole
                if (w == warp) {
                    mine = true;
                    l = ul, sq = usq, hr = uhr, i1 = items;
                }
                x += items;
                advance();
                if (x >= xe) break;
                const uint32_t next = pre[usq + 1] - pre[usq];
                if (next > kShort + kUnitCost || xe - x < (uint64_t)next) break;
                items = next;
            }
            if (!mine) i1 = 0;
        } else {
            x += i1 - i0;
            if (i1 == items) advance();
        }
        const uint32_t n = mine ? pre[sq + 1] - pre[sq] - kUnitCost : 0;
        const uint32_t s0 = i0 > kUnitCost ? i0 - kUnitCost : 0, s1 = i1 > kUnitCost ? i1 - kUnitCost : 0;
        i0 = 0;
        if (!solo && s0 >= s1) continue;          // only virtual items: the unit's steps are another CTA's
        const int h = hr / RG, rg = hr - h * RG;
        const int rows = min(R, a.G - rg * R);
        const int first = solo ? 0 : warp, stride = solo ? 1 : kWarps;

        // ---- where the warp's steps s0 + first + stride i are: lane j looks up step i = 32 b + j of batch b
        const int cnt = ((int)(s1 - s0) - first + stride - 1) / stride;
        const int32_t* row_table = a.s.table + (int64_t)sq * a.s.max_pages;
        const int32_t* row_sel =
            a.n_sel < 0 ? nullptr : a.sel + (((int64_t)l * a.s.A + sq) * p.H + h) * a.n_sel;
        uint32_t dummy = 0;
        const int64_t len = clamp_len(a.s.lens[sq], a.s.max_pages, p.page, &dummy);
        int my_id = 0, my_slot = 0, my_valid = 0;
        auto look_up = [&](int i) {
            my_valid = my_id = my_slot = 0;
            if (i < cnt) {
                const uint32_t st = s0 + first + stride * i;
                const int64_t choice = row_sel ? (int64_t)row_sel[st / (uint32_t)(p.page / kPageStep)] : 0;
                int valid;
                const int64_t lp = step_page(st, p.page, a.n_sel, choice, len, &my_slot, &valid, &bad);
                const int64_t id = lp >= 0 ? check_page(row_table[lp], p.n_pages, &bad) : -1;
                if (id >= 0) {
                    my_id = (int)id;
                    my_valid = valid;
                }
            }
        };
        const int64_t head_base = ((int64_t)(a.s.layer0 + l) * p.n_pages * p.H + h) * p.page * D;
        const int64_t page_elems = (int64_t)p.H * p.page * D;
        int64_t off = 0;
        int valid = 0;
        auto locate = [&](int i) {   // step i < cnt
            if (i > 0 && (i & 31) == 0) look_up(i + lane);
            const int id = __shfl_sync(0xffffffffu, my_id, i & 31), slot = __shfl_sync(0xffffffffu, my_slot, i & 31);
            valid = __shfl_sync(0xffffffffu, my_valid, i & 31);
            off = head_base + id * page_elems + slot * D;
        };
        // keys of tokens 8 jj + g: chunk c holds dims 32c + 8t .. + 8; values of tokens {2t, 2t+1, 2t+8, 2t+9}:
        // chunk c holds dims 64c + 8g .. + 8. Tokens that do not exist are zeros, never read.
        uint4 kw[2][KC], vw[4][VC];
        auto load_k = [&]() {
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                for (int c = 0; c < KC; ++c)
                    kw[jj][c] = 8 * jj + g < valid
                                    ? __ldg(reinterpret_cast<const uint4*>(p.k + off + (8 * jj + g) * D + 32 * c + 8 * t))
                                    : make_uint4(0u, 0u, 0u, 0u);
        };
        auto load_v = [&]() {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int tok = (e >> 1) * 8 + 2 * t + (e & 1);
#pragma unroll
                for (int c = 0; c < VC; ++c)
                    vw[e][c] = tok < valid ? __ldg(reinterpret_cast<const uint4*>(p.v + off + tok * D + 64 * c + 8 * g))
                                           : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        look_up(lane);

        // queries: k-step 2c + {0, 1} takes words {0, 1} and {2, 3} of the lane's 16-byte chunk at dims 32c + 8t
        uint32_t qa[KS][2 * RT];
        {
            const uint16_t* qb = a.q + l * a.qs.layer + sq * a.qs.row + (int64_t)(h * a.G + rg * R) * a.qs.head;
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if (8 * r + g < rows)
                        w = __ldg(reinterpret_cast<const uint4*>(qb + (8 * r + g) * a.qs.head + 32 * c + 8 * t));
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
        // Registers carry one step: the next step's keys are loaded as soon as the scores have used these, the
        // next values as soon as the value product has, so loads are in flight all the time.
        if (cnt > 0) {
            locate(0);
            load_k();
            load_v();
        }
        for (int i = 0; i < cnt; ++i) {
            const int now = valid;
            // scores of rows g (and g + 8) for tokens 8 jj + 2t + {0, 1}
            float sc[2][4];
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                sc[jj][0] = sc[jj][1] = sc[jj][2] = sc[jj][3] = 0.0f;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const uint32_t b0 = word_of(kw[jj][s >> 1], 2 * (s & 1)), b1 = word_of(kw[jj][s >> 1], 2 * (s & 1) + 1);
                    if constexpr (RT == 1) mma<BF16>(sc[jj], qa[s][0], 0u, qa[s][1], 0u, b0, b1);
                    else mma<BF16>(sc[jj], qa[s][0], qa[s][1], qa[s][2], qa[s][3], b0, b1);
                }
            }
            if (i + 1 < cnt) {
                locate(i + 1);
                load_k();
            }
            uint32_t pf[RT][TERMS][2];
            float a0[RT], a1[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                float xx[4], mx = -INFINITY;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int tok = (e >> 1) * 8 + 2 * t + (e & 1);
                    xx[e] = tok < now ? sc[e >> 1][2 * r + (e & 1)] * a.scale_log2 : -INFINITY;
                    mx = fmaxf(mx, xx[e]);
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[r], mx);
                const float ms = mn == -INFINITY ? 0.0f : mn;   // a row that has seen no token yet adds p = 0
                const float alpha = ex2a(m[r] - ms);
                m[r] = mn;
                float pr[4], ps = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    pr[e] = ex2a(xx[e] - ms);
                    ps += pr[e];
                }
                lsum[r] = lsum[r] * alpha + ps;
                // accumulator rows 2t and 2t + 1 belong to lane quads 2t and 2t + 1
                a0[r] = __shfl_sync(0xffffffffu, alpha, 8 * t);
                a1[r] = __shfl_sync(0xffffffffu, alpha, 8 * t + 4);
                // The probabilities enter the value product in the inputs' type, as a sum of parts, each the
                // rounding of what the parts before left: 3 x 8 bits (bf16) or 2 x 11 bits (f16), so the
                // product keeps fp32's accuracy.
#pragma unroll
                for (int k = 0; k < TERMS; ++k)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        pf[r][k][b] = pack_rn<BF16>(pr[2 * b], pr[2 * b + 1]);
                        const float2 f = unpack2<BF16>(pf[r][k][b]);
                        pr[2 * b] -= f.x;
                        pr[2 * b + 1] -= f.y;
                    }
            }
            // m-tile i: A rows g and g + 8 are dims 64 (i >> 2) + 8g + 2 (i & 3) + {0, 1}. The matrix unit's sums
            // are cut off rather than rounded, so a step's product starts from zero (small parts first) and
            // joins the accumulator by a rounded fused multiply-add; a sum run through the unit over a long
            // context would lose about half a bit per step in one direction.
#pragma unroll
            for (int i2 = 0; i2 < MT; ++i2) {
                const uint32_t w0 = word_of(vw[0][i2 >> 2], i2 & 3), w1 = word_of(vw[1][i2 >> 2], i2 & 3);
                const uint32_t w2 = word_of(vw[2][i2 >> 2], i2 & 3), w3 = word_of(vw[3][i2 >> 2], i2 & 3);
                const uint32_t f0 = prmt(w0, w1, 0x5410u), f1 = prmt(w0, w1, 0x7632u);
                const uint32_t f2 = prmt(w2, w3, 0x5410u), f3 = prmt(w2, w3, 0x7632u);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = TERMS - 1; k >= 0; --k) mma<BF16>(d, f0, f1, f2, f3, pf[r][k][0], pf[r][k][1]);
                    o[r][i2][0] = fmaf(o[r][i2][0], a0[r], d[0]);
                    o[r][i2][1] = fmaf(o[r][i2][1], a1[r], d[1]);
                    o[r][i2][2] = fmaf(o[r][i2][2], a0[r], d[2]);
                    o[r][i2][3] = fmaf(o[r][i2][3], a1[r], d[3]);
                }
            }
            if (i + 1 < cnt) load_v();
        }
        const int64_t out_row = ((int64_t)l * a.s.A + sq) * a.Hq + h * a.G + rg * R;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            lsum[r] += __shfl_xor_sync(0xffffffffu, lsum[r], 1);
            lsum[r] += __shfl_xor_sync(0xffffffffu, lsum[r], 2);
        }
        if (solo) {   // the warp has the whole unit: its rows are finished in registers
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
        // ---- the warps' partials, combined in shared memory
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float ls = lsum[r];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int col = 64 * (i >> 2) + 8 * g + 2 * (i & 3);
                *reinterpret_cast<float2*>(&pacc[warp][8 * r + 2 * t][col]) = make_float2(o[r][i][0], o[r][i][2]);
                *reinterpret_cast<float2*>(&pacc[warp][8 * r + 2 * t + 1][col]) = make_float2(o[r][i][1], o[r][i][3]);
            }
            if (t == 0) {
                pm[warp][8 * r + g] = m[r];
                pl[warp][8 * r + g] = ls;
            }
        }
        __syncthreads();
        const bool whole = s0 == 0 && s1 == n;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (s0 == 0 ? 1 : 0);
        for (int idx = tid; idx < rows * (D / 4); idx += kThreads) {
            const int r = idx / (D / 4), col = (idx - r * (D / 4)) * 4;
            float M = pm[0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) M = fmaxf(M, pm[w][r]);
            float L = 0.0f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (pm[w][r] != -INFINITY) {
                    const float f = ex2a(pm[w][r] - M);
                    const float4 y = *reinterpret_cast<const float4*>(&pacc[w][r][col]);
                    L = fmaf(pl[w][r], f, L);
                    v.x = fmaf(y.x, f, v.x);
                    v.y = fmaf(y.y, f, v.y);
                    v.z = fmaf(y.z, f, v.z);
                    v.w = fmaf(y.w, f, v.w);
                }
            if (whole) {
                finish4<BF16>(a, out_row + r, D, col, v, M, L);
            } else {
                *reinterpret_cast<float4*>(ws_acc + (slot * R + r) * D + col) = v;
                if (col == 0) *reinterpret_cast<float2*>(ws_ml + (slot * R + r) * 2) = make_float2(M, L);
            }
        }
        if (!whole) {
            const uint32_t c0 = share_of(u0, total, nc);
            const int np = (int)(share_of(u0 + n - 1, total, nc) - c0) + 1;
            __threadfence();   // this thread's part of the piece, before the arrival below
            __syncthreads();
            if (tid == 0) last_here = atomicInc(ws_count + c0, (uint32_t)np - 1) == (uint32_t)np - 1;
            __syncthreads();
            if (last_here) {
                __threadfence();
                join_pieces<D, R, BF16>(a, ws_acc, ws_ml, c0, np, out_row, rows, &pacc[0][0][0], jml);
            }
        }
        __syncthreads();   // the partials' shared memory is reused by the next unit
    }
    if (bad && p.status) atomicOr(p.status, bad);
}

// The arrival counts come first: they are the part of the workspace that is zero between calls.
constexpr int kMaxCtas = 1024;
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

template <int D, int RT, bool BF16>
polykv_status run(const PagesAttendArgs& a, void* ws, cudaStream_t st) {
    constexpr int R = 8 * RT;
    auto kern = pages_attend_kernel<D, RT, BF16>;
    const WsLayout w = ws_layout(grid_ctas(kMaxPerSm), R, D);
    char* base = static_cast<char*>(ws);
    const size_t smem = (size_t)(a.s.A + 1) * sizeof(uint32_t);
    if (RT == 2) {   // static and dynamic shared memory pass 48 KB for many sequences
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)((kPagesMaxSeqs + 1) * sizeof(uint32_t)));
        if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_attend: smem attribute: %s", cudaGetErrorString(e));
    }
    kern<<<grid_ctas(per_sm<D, RT>()), kThreads, smem, st>>>(a, reinterpret_cast<uint32_t*>(base),
                                                          reinterpret_cast<float*>(base + w.acc),
                                                          reinterpret_cast<float*>(base + w.ml));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_attend launch: %s", cudaGetErrorString(e));
    return POLYKV_OK;
}

}  // namespace

size_t pages_attend_workspace(const PagesView& p, int G) {
    return ws_layout(grid_ctas(kMaxPerSm), G <= 8 ? 8 : 16, p.d).total;
}

polykv_status launch_pages_attend(const PagesAttendArgs& a, polykv_dtype dt, void* ws, cudaStream_t st) {
    const bool bf = dt == POLYKV_BF16;
    if (a.p.d == 128) {
        if (a.G <= 8) return bf ? run<128, 1, true>(a, ws, st) : run<128, 1, false>(a, ws, st);
        return bf ? run<128, 2, true>(a, ws, st) : run<128, 2, false>(a, ws, st);
    }
    if (a.G <= 8) return bf ? run<64, 1, true>(a, ws, st) : run<64, 1, false>(a, ws, st);
    return bf ? run<64, 2, true>(a, ws, st) : run<64, 2, false>(a, ws, st);
}

}  // namespace polykv
