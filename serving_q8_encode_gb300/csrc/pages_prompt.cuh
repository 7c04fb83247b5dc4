// One row of attention at a time, in fp32, by one warp: the definition as a program, for what the tensor-core kernel of
// pages_prompt.cu leaves to it.
#pragma once

#include "pages_rows.cuh"

namespace polykv {

// Where a row belongs: its sequence and its place there; place < 0 where nobody owns it.
struct RowOf {
    int seq;
    int64_t place, len;
};
// Elements col .. col + D/32 of a token's keys (which = 0) or values.
template <int D, bool BF16>
__device__ __forceinline__ void row_part(const PagesView& p, int64_t unit, int slot, int which, int lane, float (&f)[D / 32]) {
    constexpr int E = D / 32;
    const void* base = which ? p.v : p.k;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(base) + (unit * p.page + slot) * D + E * lane);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        const float2 x = unpack2<BF16>(w[i]);
        f[2 * i] = x.x, f[2 * i + 1] = x.y;
    }
}

template <int D, bool BF16>
__device__ __noinline__ void attend_row(const PagesRowsArgs& a, int l, const RowOf& at, int64_t r, int h, int lane, uint32_t* bad) {
    constexpr int E = D / 32;
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
    const int64_t end = at.place + 1, lead_end = win.begin < win.sinks ? win.begin : win.sinks;   // [0, lead_end) and [begin, end)
    int64_t unit = -1;
    for (int64_t t = lead_end > 0 ? 0 : win.begin; t < end; t = t + 1 == lead_end && win.begin > t ? win.begin : t + 1) {
        if (unit < 0 || (t & (p.page - 1)) == 0 || t == win.begin) {
            const int64_t id = check_page(a.s.table[(int64_t)at.seq * a.s.max_pages + (t >> shift)], p.n_pages, bad);
            unit = id < 0 ? -1 : ((int64_t)(a.s.layer0 + l) * p.n_pages + id) * p.H + h / a.G;
        }
        if (unit < 0) continue;   // a page that does not exist
        float k[E], x = 0.0f;
        row_part<D, BF16>(p, unit, (int)(t & (p.page - 1)), 0, lane, k);
#pragma unroll
        for (int i = 0; i < E; ++i) x = fmaf(q[i], k[i], x);
#pragma unroll
        for (int o2 = 16; o2 > 0; o2 >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o2);
        x *= a.scale_log2;
        const float m = fmaxf(M, x), ms = m == -INFINITY ? 0.0f : m;
        const float alpha = exp2f(M - ms), pr = exp2f(x - ms);
        M = m;
        L = fmaf(L, alpha, pr);
        if (x != -INFINITY) {   // a logit of -inf leaves its token out
            row_part<D, BF16>(p, unit, (int)(t & (p.page - 1)), 1, lane, k);
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = fmaf(pr, k[i], o[i] * alpha);
        }
    }
    const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);   // a NaN stays one
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + (((int64_t)l * a.rows + r) * a.Hq + h) * D + E * lane);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) out[i] = pack_rn<BF16>(o[2 * i] * inv, o[2 * i + 1] * inv);
}

}  // namespace polykv
