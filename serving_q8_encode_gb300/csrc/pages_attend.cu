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
#include "pages_attend.cuh"

namespace polykv {
namespace attend {

// Keys and values in 16 bits: rows of 64 columns (128 bytes) in the swizzled tiles, the two halves of a 128-wide head in tiles
// of their own.
template <int D_, bool BF16_>
struct Wide {
    static constexpr int D = D_;
    static constexpr bool BF16 = BF16_, kScales = false;
    static constexpr int KS = D / 16;      // score k-steps
    static constexpr int MT = D / 16;      // value m-tiles
    static constexpr int HV = D / 64;      // 64-column halves of a row
    static constexpr int TERMS = BF16 ? 3 : 2;   // parts that a probability is split into (below)
    static constexpr int PW = BF16 ? 2 : 4;      // words of a part of a lane's four probabilities
    using Chunk = Cut<4>;
    static constexpr int kHalf = Chunk::kTokens * 128;         // bytes of 64 columns of a chunk
    static constexpr int kStage = 2 * Chunk::kTokens * D * 2;  // a chunk's keys and values
    static constexpr uint32_t kStepBytes = kPageStep * D * 4;
    // Resident CTAs per SM: by the ring, about 190 KB an SM in stages of 32 KB (d = 128) or 16 KB.
    static constexpr int per_sm(int) { return D == 64 ? 3 : 2; }

    template <int RT>
    struct Query {
        uint32_t a[KS][2 * RT];
    };

    // This lane's 16-byte chunks in the swizzled tiles (chunk j of row r stands at j ^ (r & 7)): keys of tokens
    // 8 jj + g, columns 64 hf + 16t + 8c .. + 8; values of tokens {2t, 2t+1, 2t+8, 2t+9}, columns 64 hf + 8g .. + 8
    const int g, t;
    const int k_at[2], v_at[2];
    __device__ __forceinline__ Wide(int g_, int t_)
        : g(g_), t(t_), k_at{g_ * 128 + ((2 * t_) ^ g_) * 16, g_ * 128 + ((2 * t_ + 1) ^ g_) * 16},
          v_at{2 * t_ * 128 + (g_ ^ (2 * t_)) * 16, (2 * t_ + 1) * 128 + (g_ ^ (2 * t_ + 1)) * 16} {}

    // The first of a lane's four accumulator columns of m-tiles i and i + 1 (i even).
    static __device__ __forceinline__ int col(int g, int i) { return 64 * (i >> 2) + 8 * g + 2 * (i & 3); }

    static __device__ __forceinline__ void copy(uint32_t stage, int st, const void* km, const void* vm, int row, uint32_t bar) {
        const uint32_t dst = stage + st * (kPageStep * 128);
#pragma unroll
        for (int hf = 0; hf < HV; ++hf) {
            tc::tma_2d_g2s(dst + hf * kHalf, km, 64 * hf, row, bar);
            tc::tma_2d_g2s(dst + (HV + hf) * kHalf, vm, 64 * hf, row, bar);
        }
    }

    // queries: the k-steps of chunk (hf, c) take its words {0, 1} and {2, 3}
    template <int RT>
    __device__ __forceinline__ void load(Query<RT>& query, const uint16_t* qb, int64_t head, int rows) const {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int c = 0; c < 2 * HV; ++c) {
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (8 * r + g < rows)
                    w = __ldg(reinterpret_cast<const uint4*>(qb + (8 * r + g) * head + 64 * (c >> 1) + 16 * t + 8 * (c & 1)));
                query.a[2 * c][r] = w.x;
                query.a[2 * c][RT + r] = w.y;
                query.a[2 * c + 1][r] = w.z;
                query.a[2 * c + 1][RT + r] = w.w;
            }
    }

    template <int RT>
    __device__ __forceinline__ void step(const unsigned char* stage, int st, uint32_t seen, const float2&, float scale_log2,
                                         const Query<RT>& query, float (&m)[RT], float (&lsum)[RT], float (&o)[RT][MT][4]) const {
        const unsigned char* kt = stage + st * (kPageStep * 128);
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
                    const uint32_t(&qk)[2 * RT] = query.a[4 * hf + k];
                    if constexpr (RT == 1) mma<BF16>(sc[jj], qk[0], 0u, qk[1], 0u, b0, b1);
                    else mma<BF16>(sc[jj], qk[0], qk[1], qk[2], qk[3], b0, b1);
                }
            }
        if (seen != 0xffffu) {   // what is not visible holds anything: keep it out of the softmax
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!(seen >> ((e >> 1) * 8 + 2 * t + (e & 1)) & 1u)) {
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
                xx[e] = sc[e >> 1][2 * r + (e & 1)] * scale_log2;
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
            if (seen != 0xffffu) {   // nor may it meet a probability of zero
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!(seen >> ((e >> 1) * 8 + 2 * t + (e & 1)) & 1u)) vw[e] = make_uint4(0u, 0u, 0u, 0u);
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
};

}  // namespace attend

PagesTma* pages_tma_new() { return new (std::nothrow) PagesTma; }
void pages_tma_free(PagesTma* t) { delete t; }

size_t pages_attend_workspace(const PagesView& p, int G) {
    return attend::ws_layout(attend::grid_ctas(attend::kMaxPerSm), G <= 8 ? 8 : 16, p.d).total;
}

polykv_status pages_wide_maps(const PagesView& p, const attend::PageMaps** maps) {
    std::lock_guard<std::mutex> lock(p.tma->mu);
    if (!p.tma->made) {
        const polykv_status s = attend::make_maps(p, CU_TENSOR_MAP_DATA_TYPE_UINT16, p.d, 1, 64, 2, &p.tma->maps);
        if (s != POLYKV_OK) return s;
        p.tma->made = true;
    }
    *maps = &p.tma->maps;
    return POLYKV_OK;
}

polykv_status launch_pages_attend(const PagesAttendArgs& a, polykv_dtype dt, void* ws, cudaStream_t st) {
    using namespace attend;
    if (a.p.code != kPagesWide) return launch_pages_attend8(a, dt, ws, st);
    const PageMaps* maps;
    const polykv_status s = pages_wide_maps(a.p, &maps);
    if (s != POLYKV_OK) return s;
    const PageMaps& m = *maps;
    const bool bf = dt == POLYKV_BF16;
    if (a.p.d == 128) {
        if (a.G <= 8) return bf ? run<Wide<128, true>, 1>(a, m, ws, st) : run<Wide<128, false>, 1>(a, m, ws, st);
        return bf ? run<Wide<128, true>, 2>(a, m, ws, st) : run<Wide<128, false>, 2>(a, m, ws, st);
    }
    if (a.G <= 8) return bf ? run<Wide<64, true>, 1>(a, m, ws, st) : run<Wide<64, false>, 1>(a, m, ws, st);
    return bf ? run<Wide<64, true>, 2>(a, m, ws, st) : run<Wide<64, false>, 2>(a, m, ws, st);
}

}  // namespace polykv
