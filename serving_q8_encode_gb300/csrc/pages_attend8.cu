// Attention of one new token per sequence over a paged cache held in 8 bits: codes (int8 or e4m3) with one fp32 scale per
// (page, kv head) for the keys and one for the values.
//
//   x_t = softmax_scale s_k(page of t) (q . kc_t),   out = sum_t softmax_t(x) s_v(page of t) vc_t
//
// The frame, the work list and the join are the 16-bit kernel's (pages_attend.cuh); half the bytes pass, so a step's
// instructions count for twice as much. Codes of either kind are exact in f16, so both products run on m16n8k16 in f16:
//   - a lane reads 16 neighbouring codes at a time and turns pairs of them into f16 in registers (int8: byte permutes into
//     1024 + 128 + code, less 1152; e4m3: the conversion instruction);
//   - bf16 queries enter multiplied by a power of two per row that brings their largest to [2^14, 2^15): exact down to
//     2^-31 of it, and 2^-39 of it at worst below that;
//   - probabilities are kept relative to 2^15 times the running maximum's and enter as two f16 parts, 22 bits for all down to
//     2^-18 of the largest, 2^-40 of the largest at worst: 2^20 of those together change an output by 2^-20 of itself;
//   - a step lies in one page, so its scales are two numbers: the keys' joins the logit's factor, the values' the
//     accumulator's rounded multiply-add.
//
// Measured (8 kv heads x 4 query heads, d = 128): one sequence of 131,071 tokens, int8, 58 us = 4.6 TB/s, 15 of about 3,800 tokens,
// e4m3, 31.5 us. The copies alone, without any arithmetic, take 51 and 28.7 us; the rest is instructions, about 430 for a step
// of 16 tokens. Chunks of 128 tokens, since the producer's work is per chunk (64: 60.5 and 32.6 us); three blocks an SM spill (60 us).
#include "pages_attend.cuh"

namespace polykv {
namespace attend {

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    mma<false>(d, a0, a1, a2, a3, b0, b1);
}

__device__ __forceinline__ uint64_t pair_of(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
// (x, y) = (x, y) a + (dx, dy) s, a rounded product and a fused one.
__device__ __forceinline__ void join2(float& x, float& y, float dx, float dy, uint64_t a, uint64_t s) {
    asm("{\n .reg .b64 v, d;\n mov.b64 v, {%0, %1};\n mov.b64 d, {%2, %3};\n mul.rn.f32x2 v, v, %4;\n fma.rn.f32x2 v, d, %5, v;\n"
        " mov.b64 {%0, %1}, v;\n}"
        : "+f"(x), "+f"(y)
        : "f"(dx), "f"(dy), "l"(a), "l"(s));
}

// Four codes in a word, as two pairs of f16.
template <int CODE>
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (CODE == kPagesInt8) {
        const uint32_t u = w ^ 0x80808080u;                      // code + 128
        const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));   // 1152
        const uint32_t a = prmt(u, 0x64646464u, 0x4140u), b = prmt(u, 0x64646464u, 0x4342u);       // 1024 + code + 128
        const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias), y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
        lo = *reinterpret_cast<const uint32_t*>(&x);
        hi = *reinterpret_cast<const uint32_t*>(&y);
    } else {
        asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
            : "=r"(lo), "=r"(hi) : "r"(w));
    }
}

template <int D_, int CODE, bool BF16_>
struct Narrow {
    static constexpr int D = D_;
    static constexpr bool BF16 = BF16_, kScales = true;   // BF16: the queries' and a 16-bit output's type
    static constexpr int KS = D / 16, MT = D / 16;
    using Chunk = Cut<8>;
    static constexpr int kTile = Chunk::kTokens * D;      // bytes of a chunk's keys, or values
    static constexpr int kStage = 2 * kTile;
    static constexpr uint32_t kStepBytes = 2 * kPageStep * D;
    static constexpr int per_sm(int rt) { return D == 64 ? 3 : 2; }
    static constexpr float kTop = 15.0f;                  // log2 of the largest probability as it is held

    template <int RT>
    struct Query {
        uint32_t a[KS][2 * RT];   // f16: k-step j has the lane's columns D/4 t + 4j + {0, 1} and {2, 3}
        float unit[RT];           // what a row's products are multiples of
    };

    const int g, t;
    __device__ __forceinline__ Narrow(int g_, int t_) : g(g_), t(t_) {}

    static __device__ __forceinline__ int col(int g, int i) { return (D / 8) * g + 2 * i; }

    // Byte `b` of token `tok` of a step in the swizzled tile: rows of 128 bytes, one token or (D = 64) two each.
    static __device__ __forceinline__ int at(int tok, int b) {
        const int row = D == 128 ? tok : tok >> 1, byte = D == 128 ? b : (tok & 1) * 64 + b;
        return row * 128 + (((byte >> 4) ^ (row & 7)) << 4 | (byte & 15));
    }

    static __device__ __forceinline__ void copy(uint32_t stage, int st, const void* km, const void* vm, int row, uint32_t bar) {
        const uint32_t dst = stage + st * (kPageStep * D);
        tc::tma_2d_g2s(dst, km, 0, D == 128 ? row : row >> 1, bar);
        tc::tma_2d_g2s(dst + kTile, vm, 0, D == 128 ? row : row >> 1, bar);
    }

    template <int RT>
    __device__ __forceinline__ void load(Query<RT>& query, const uint16_t* qb, int64_t head, int rows) const {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            uint4 w[KS / 2];
#pragma unroll
            for (int c = 0; c < KS / 2; ++c) {
                w[c] = make_uint4(0u, 0u, 0u, 0u);
                if (8 * r + g < rows) w[c] = __ldg(reinterpret_cast<const uint4*>(qb + (8 * r + g) * head + (D / 4) * t + 8 * c));
            }
            query.unit[r] = 1.0f;
            if constexpr (BF16) {
                float top = 0.0f;
#pragma unroll
                for (int c = 0; c < KS / 2; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = unpack2<true>(word_of(w[c], i));
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^(14 - exponent), from 2^-113 to 2^100; infinities stay what they are
                int e = 14 - ((int)(__float_as_uint(top) >> 23) - 127);
                e = e > 100 ? 100 : e;
                if (!(top < INFINITY)) e = 0;
                const float up = __uint_as_float((uint32_t)(e + 127) << 23);
                query.unit[r] = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                for (int c = 0; c < KS / 2; ++c) {
                    uint32_t* x = reinterpret_cast<uint32_t*>(&w[c]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = unpack2<true>(x[i]);
                        x[i] = pack_rn<false>(f.x * up, f.y * up);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < KS / 2; ++c) {
                query.a[2 * c][r] = w[c].x;
                query.a[2 * c][RT + r] = w[c].y;
                query.a[2 * c + 1][r] = w[c].z;
                query.a[2 * c + 1][RT + r] = w[c].w;
            }
        }
    }

    template <int RT>
    __device__ __forceinline__ void step(const unsigned char* stage, int st, uint32_t seen, const float2& scale, float scale_log2,
                                         const Query<RT>& query, float (&m)[RT], float (&lsum)[RT], float (&o)[RT][MT][4]) const {
        const unsigned char* kt = stage + st * (kPageStep * D);
        const unsigned char* vt = kt + kTile;
        const float2 sc2 = scale;
        // scores of rows g (and g + 8) for tokens 8 jj + 2t + {0, 1}
        float sc[2][4];
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            sc[jj][0] = sc[jj][1] = sc[jj][2] = sc[jj][3] = 0.0f;
            uint4 kw[D / 64];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) kw[c] = *reinterpret_cast<const uint4*>(kt + at(8 * jj + g, (D / 4) * t + 16 * c));
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                uint32_t b0, b1;
                widen<CODE>(word_of(kw[j >> 2], j & 3), b0, b1);
                const uint32_t(&qk)[2 * RT] = query.a[j];
                if constexpr (RT == 1) mma_f16(sc[jj], qk[0], 0u, qk[1], 0u, b0, b1);
                else mma_f16(sc[jj], qk[0], qk[1], qk[2], qk[3], b0, b1);
            }
        }
        uint32_t pf[RT][2][2];
        float a0[RT], a1[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float unit = scale_log2 * query.unit[r] * sc2.x;
            float xx[4], mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                xx[e] = sc[e >> 1][2 * r + (e & 1)] * unit;
                if (seen != 0xffffu && !(seen >> ((e >> 1) * 8 + 2 * t + (e & 1)) & 1u)) xx[e] = -INFINITY;   // holds anything
                mx = fmaxf(mx, xx[e]);
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[r], mx - kTop);
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
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                pf[r][0][b] = pack_rn<false>(pr[2 * b], pr[2 * b + 1]);
                const float2 f = unpack2<false>(pf[r][0][b]);
                pf[r][1][b] = pack_rn<false>(pr[2 * b] - f.x, pr[2 * b + 1] - f.y);
            }
        }
        // A rows g and g + 8 of m-tile i are columns D/8 g + 2i + {0, 1}; as in the 16-bit kernel a step's product starts from
        // zero (small parts first) and joins the accumulator by a rounded multiply-add
        constexpr int W = D / 32;   // words of a token's codes per lane
        uint32_t vw[4][W];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int tok = (e >> 1) * 8 + 2 * t + (e & 1);
            if constexpr (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4*>(vt + at(tok, 16 * g));
                vw[e][0] = x.x, vw[e][1] = x.y, vw[e][2] = x.z, vw[e][3] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(vt + at(tok, 8 * g));
                vw[e][0] = x.x, vw[e][1] = x.y;
            }
            if (seen != 0xffffu && !(seen >> tok & 1u)) {
#pragma unroll
                for (int w = 0; w < W; ++w) vw[e][w] = 0u;
            }
        }
        uint64_t aa[RT];
        const uint64_t sv = pair_of(sc2.y, sc2.y);
#pragma unroll
        for (int r = 0; r < RT; ++r) aa[r] = pair_of(a0[r], a1[r]);
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {   // two columns of the word's four, tokens side by side
                uint32_t f0, f1, f2, f3;
                widen<CODE>(prmt(vw[0][w], vw[1][w], hf ? 0x7362u : 0x5140u), f0, f1);
                widen<CODE>(prmt(vw[2][w], vw[3][w], hf ? 0x7362u : 0x5140u), f2, f3);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma_f16(d, f0, f1, f2, f3, pf[r][1][0], pf[r][1][1]);
                    mma_f16(d, f0, f1, f2, f3, pf[r][0][0], pf[r][0][1]);
                    float(&acc)[4] = o[r][2 * w + hf];   // two at a time
                    join2(acc[0], acc[1], d[0], d[1], aa[r], sv);
                    join2(acc[2], acc[3], d[2], d[3], aa[r], sv);
                }
            }
    }
};

namespace {

template <int D, int CODE>
polykv_status run8(const PagesAttendArgs& a, const PageMaps& m, bool bf, void* ws, cudaStream_t st) {
    if (a.G <= 8) return bf ? run<Narrow<D, CODE, true>, 1>(a, m, ws, st) : run<Narrow<D, CODE, false>, 1>(a, m, ws, st);
    return bf ? run<Narrow<D, CODE, true>, 2>(a, m, ws, st) : run<Narrow<D, CODE, false>, 2>(a, m, ws, st);
}

}  // namespace
}  // namespace attend

polykv_status launch_pages_attend8(const PagesAttendArgs& a, polykv_dtype dt, void* ws, cudaStream_t st) {
    using namespace attend;
    {
        std::lock_guard<std::mutex> lock(a.p.tma->mu);
        if (!a.p.tma->made) {
            const polykv_status s = make_maps(a.p, CU_TENSOR_MAP_DATA_TYPE_UINT8, 128, 128 / a.p.d, 128, 1, &a.p.tma->maps);
            if (s != POLYKV_OK) return s;
            a.p.tma->made = true;
        }
    }
    const PageMaps& m = a.p.tma->maps;
    const bool bf = dt == POLYKV_BF16;
    if (a.p.code == kPagesInt8)
        return a.p.d == 128 ? run8<128, kPagesInt8>(a, m, bf, ws, st) : run8<64, kPagesInt8>(a, m, bf, ws, st);
    return a.p.d == 128 ? run8<128, kPagesE4m3>(a, m, bf, ws, st) : run8<64, kPagesE4m3>(a, m, bf, ws, st);
}

}  // namespace polykv
