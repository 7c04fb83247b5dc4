// One row of attention at a time, in fp32, by one warp: the definition as a program, for what the tensor-core kernel of
// pages_prompt.cu leaves to it.
#pragma once

#include "pages_rows.cuh"
#include "tc_ptx.cuh"

namespace polykv {

// Where a row belongs: its sequence and its place there.
struct RowOf {
    int seq;
    int64_t place;
};
// Elements E lane .. + E of a token's keys (which = 0) or values, E = D / 32.
template <int D>
__device__ __forceinline__ const uint32_t* row_part(const PagesView& p, int64_t unit, int slot, int which, int lane) {
    return reinterpret_cast<const uint32_t*>((which ? p.v : p.k) + (unit * p.page + slot) * D + D / 32 * lane);
}

// Eight tokens at a time, so that their loads and sums are on their way together: 0.19 us a token, where one after the other took 1.
template <int D, bool BF16>
__device__ __noinline__ void attend_row(const PagesRowsArgs& a, int l, const RowOf& at, int64_t r, int h, int lane, uint32_t* bad, volatile uint64_t* moved) {
    constexpr int E = D / 32, B = 8;
    const PagesView& p = a.p;
    const int shift = page_shift(p.page);
    const uint32_t* qw = reinterpret_cast<const uint32_t*>(a.q + l * a.qs.layer + r * a.qs.row + h * a.qs.head + E * lane);
    float q[E], o[E], M = -INFINITY, L = 0.0f;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        const float2 x = unpack2<BF16>(qw[i]);
        q[2 * i] = x.x, q[2 * i + 1] = x.y;
        o[2 * i] = o[2 * i + 1] = 0.0f;
    }
    const Window win = window_of(at.place + 1, p.page, a.window, a.sinks);
    const int64_t end = at.place + 1, lead = win.begin < win.sinks ? win.begin : win.sinks;   // [0, lead) and [begin, end)
    int64_t unit = -1, looked = -1;
    for (int64_t t0 = lead > 0 ? 0 : win.begin & ~(int64_t)(B - 1); t0 < end; t0 += B) {
        if (t0 >= lead && t0 + B <= win.begin) t0 = win.begin & ~(int64_t)(B - 1);
        if ((t0 & 63) == 0) {   // a sign of life for the block's waits; what is not finite stays so
            if (lane == 0) *moved = tc::globaltimer();
            bool lost = true;
#pragma unroll
            for (int i = 0; i < E; ++i) lost = lost && !(fabsf(o[i]) < INFINITY);
            if (__all_sync(0xffffffffu, lost)) break;
        }
        if (t0 >> shift != looked) {
            looked = t0 >> shift;
            const int64_t id = check_page(a.s.table[(int64_t)at.seq * a.s.max_pages + looked], p.n_pages, bad);
            unit = id < 0 ? -1 : ((int64_t)(a.s.layer0 + l) * p.n_pages + id) * p.H + h / a.G;
        }
        if (unit < 0) continue;   // a page that does not exist
        const int slot = (int)(t0 & (p.page - 1));
        auto seen = [&](int j) { return t0 + j < end && (t0 + j >= win.begin || t0 + j < lead); };
        uint32_t w[B][E / 2];
        float x[B];
#pragma unroll
        for (int j = 0; j < B; ++j)
#pragma unroll
            for (int i = 0; i < E / 2; ++i) w[j][i] = row_part<D>(p, unit, slot + j, 0, lane)[i];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            x[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float2 k = unpack2<BF16>(w[j][i]);
                x[j] = fmaf(q[2 * i + 1], k.y, fmaf(q[2 * i], k.x, x[j]));
            }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
#pragma unroll
            for (int j = 0; j < B; ++j) x[j] += __shfl_xor_sync(0xffffffffu, x[j], d);
        float m = M;
#pragma unroll
        for (int j = 0; j < B; ++j) {
            x[j] = seen(j) ? x[j] * a.scale_log2 : -INFINITY;
            m = fmaxf(m, x[j]);
        }
        const float ms = m == -INFINITY ? 0.0f : m, alpha = exp2f(M - ms);
        M = m;
        L *= alpha;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] *= alpha;
#pragma unroll
        for (int j = 0; j < B; ++j)
#pragma unroll
            for (int i = 0; i < E / 2; ++i) w[j][i] = row_part<D>(p, unit, slot + j, 1, lane)[i];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if (x[j] == -INFINITY) continue;   // not seen, or a logit of -inf: the token is left out
            const float pr = exp2f(x[j] - ms);
            L += pr;
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float2 v = unpack2<BF16>(w[j][i]);
                o[2 * i] = fmaf(pr, v.x, o[2 * i]), o[2 * i + 1] = fmaf(pr, v.y, o[2 * i + 1]);
            }
        }
    }
    const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);   // a NaN stays one
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + (((int64_t)l * a.rows + r) * a.Hq + h) * D + E * lane);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) out[i] = pack_rn<BF16>(o[2 * i] * inv, o[2 * i + 1] * inv);
}

}  // namespace polykv
