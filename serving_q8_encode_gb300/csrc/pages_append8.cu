// Appending keys and values to a paged cache held in 8 bits, with the position rotation applied on the way; and reading
// tokens back as 16-bit rows, from either kind of cache.
//
//   k' = R(pos f) k, q' = R(pos f) q, v' = v                                     as in the 16-bit append
//   per (page, kv head), keys and values apart:
//     s = max(s before, smallest 2^e with max |x| <= top 2^e)                    top = 127 (int8) or 448 (e4m3)
//     code = rn(x / s);   codes already there: rn(code (s before / s))           s before = 0 for a page's first token
//
// A power of two costs up to a bit of int8's fraction and none of e4m3's. For that, dividing is exact, so a code depends on
// nothing but its value and scale; a scale that rises at least doubles, so codes that are rewritten lose less than one step of
// the last scale in all (1/2 + 1/4 + ...), where a scale of max / 127 would rise with every new largest value; and e4m3 codes
// above the subnormals are moved without any loss.
//
// A block of values with an infinity or a NaN among it gets NaN for its scale: it reads as NaN, until its page is begun again.
//
// One block of threads takes one page's share of the new tokens and a group of heads, so that it alone sees what a scale
// depends on: it holds a head's new rows in registers (fp32, rotated), takes their largest over the threads, and writes codes.
// HBM binds long appends (2 bytes in, 1 out per element of k and v, 2 and 2 of q), latency the short ones. One token per
// sequence (a decode step): a row is 8 or 4 lanes' work, which agree on the scale by shuffles.
//
// Measured (d = 128, bf16): 7,194 tokens of 8 kv and 32 query heads, e4m3: 36.0 us = 4.5 TB/s of rows and codes; keys and values
// alone 14.7 us; half of the issue slots go to conversions and turns. 256 sequences of one token 3.0 us. Read back: 7.3 us =
// 6.0 TB/s, and 6.0 us (five dependent loads).
#include "pages_rows.cuh"

namespace polykv {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;   // query heads in flight per thread
constexpr uint32_t kNotFinite = 0x7F800000u;

// Cosine and sine of pos * turns, to their last place: a code next to a border depends on it. The angle's leading 25 bits go
// through the functions, exact in fp32 (rounding 32 bits to it would be off by up to 2^-23.3), the next 14 join by the first
// derivative (of what is left, 2^-25 turns, the square is 2^-45 of a radian).
__device__ __forceinline__ float2 turn_of(uint64_t pos, uint64_t turns, float mscale) {
    const uint64_t frac = pos * turns;                        // in units of 2^-64 turns
    const int32_t high = (int32_t)(uint32_t)(frac >> 32) & ~127;
    const float rest = (float)((uint32_t)(frac >> 25) & 0x3FFFu) * (6.283185307f / 549755813888.0f);   // 2 pi 2^-39
    float s, c;
    sincospif((float)high * (2.0f / 4294967296.0f), &s, &c);
    return make_float2(fmaf(-s, rest, c) * mscale, fmaf(c, rest, s) * mscale);
}

// The smallest power of two, 2^-100 at least, under which a value with these bits (sign off) is at most `top`; NaN for one that
// is not finite.
template <int CODE>
__device__ __forceinline__ float scale_for(uint32_t bits) {
    if (bits >= kNotFinite) return __uint_as_float(0x7FC00000u);
    // top = 1.984375 * 2^6 or 1.75 * 2^8
    const int e = (int)(bits >> 23) - 127 - (CODE == kPagesInt8 ? 6 : 8) + ((bits & 0x7FFFFFu) > (CODE == kPagesInt8 ? 0x7E0000u : 0x600000u));
    return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}
// The scale of a block with new values under `fresh` and earlier ones under `old` (0: none).
__device__ __forceinline__ float scale_with(float old, float fresh) { return old == old && fresh == fresh ? fmaxf(old, fresh) : old + fresh; }

template <int CODE>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
    if constexpr (CODE == kPagesInt8) {
        auto one = [](float x) { return (uint32_t)max(-127, min(127, __float2int_rn(x))) & 0xFFu; };
        return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
    } else {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return (uint32_t)lo | (uint32_t)hi << 16;
    }
}
template <int CODE>
__device__ __forceinline__ float4 value4(uint32_t w) {
    if constexpr (CODE == kPagesInt8) {
        return make_float4((float)(int8_t)(w & 0xFF), (float)(int8_t)(w >> 8 & 0xFF), (float)(int8_t)(w >> 16 & 0xFF), (float)(int8_t)(w >> 24));
    } else {
        uint32_t lo, hi;
        asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}" : "=r"(lo), "=r"(hi) : "r"(w));
        const float2 a = unpack2<false>(lo), b = unpack2<false>(hi);
        return make_float4(a.x, a.y, b.x, b.y);
    }
}
// Codes under one scale as codes under another.
template <int CODE>
__device__ __forceinline__ uint4 recode(uint4 w, float ratio) {
    uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = value4<CODE>(x[i]);
        x[i] = code4<CODE>(v.x * ratio, v.y * ratio, v.z * ratio, v.w * ratio);
    }
    return w;
}

// The 16 values of two chunks, rotated: f[0 .. 8) of the first, f[8 .. 16) of the second.
template <bool BF16>
__device__ __forceinline__ void spread(const uint4& x, const uint4& y, float (&f)[16]) {
    const uint32_t* xw = reinterpret_cast<const uint32_t*>(&x);
    const uint32_t* yw = reinterpret_cast<const uint32_t*>(&y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = unpack2<BF16>(xw[i]), b = unpack2<BF16>(yw[i]);
        f[2 * i] = a.x, f[2 * i + 1] = a.y, f[8 + 2 * i] = b.x, f[9 + 2 * i] = b.y;
    }
}
// cs[i] = (cosine, sine) of the lane's pair i: of elements i and 8 + i, or of neighbours (the first chunk's four, the second's).
__device__ __forceinline__ void rotate16(float (&f)[16], const float2 (&cs)[8], bool interleaved, bool second) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (interleaved) {
            if (i >= 4 && !second) continue;
            const float a = f[2 * i], b = f[2 * i + 1];
            f[2 * i] = a * cs[i].x - b * cs[i].y;
            f[2 * i + 1] = b * cs[i].x + a * cs[i].y;
        } else {
            const float a = f[i], b = f[8 + i];
            f[i] = a * cs[i].x - b * cs[i].y;
            f[8 + i] = b * cs[i].x + a * cs[i].y;
        }
    }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack_rn<BF16>(f[0], f[1]), pack_rn<BF16>(f[2], f[3]), pack_rn<BF16>(f[4], f[5]), pack_rn<BF16>(f[6], f[7]));
}
template <int CODE>
__device__ __forceinline__ uint2 codes8(const float* f, float inv) {
    return make_uint2(code4<CODE>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv), code4<CODE>(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}
__device__ __forceinline__ uint32_t largest(const float (&f)[16]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    return m;
}

// A thread's two 8-element chunks of a row of D, and whether they rotate.
struct Chunks {
    int a, b;
    bool rot_a, rot_b;
    __device__ __forceinline__ Chunks(const PagesAppendArgs& x, int c, int C) {
        const int rc = x.turns ? x.rot / 16 : 0;   // threads of a row that rotate
        a = x.interleaved || c < rc ? c : 2 * rc + 2 * (c - rc);
        b = x.interleaved ? c + C : (c < rc ? c + rc : a + 1);
        rot_a = a < (x.interleaved ? 2 * rc : rc);
        rot_b = x.interleaved ? b < 2 * rc : rot_a;
    }
    // Where the turn of the lane's pair i stands in shared memory: the pairs of neighbouring lanes side by side (in the order of
    // their frequencies all lanes of a warp would read four banks).
    __device__ __forceinline__ int pair(const PagesAppendArgs& x, int i) const {
        const int half = x.rot / 2;
        return x.interleaved ? (i & 3) * (half / 4) + (i < 4 || !rot_b ? a : b) : i * (half / 8) + a;
    }
    static __device__ __forceinline__ int place(const PagesAppendArgs& x, int f) {   // of frequency f
        const int half = x.rot / 2;
        return x.interleaved ? (f & 3) * (half / 4) + (f >> 2) : (f & 7) * (half / 8) + (f >> 3);
    }
};

__device__ __forceinline__ const uint16_t* source(const PagesAppendArgs& a, int l, int64_t r, int j) {
    return j < a.p.H       ? a.k + l * a.ks.layer + r * a.ks.row + j * a.ks.head
           : j < 2 * a.p.H ? a.v + l * a.vs.layer + r * a.vs.row + (j - a.p.H) * a.vs.head
                           : a.q + l * a.qs.layer + r * a.qs.row + (j - 2 * a.p.H) * a.qs.head;
}

// Runs of tokens. grid: (items, head groups, layers). Jobs are heads: kv heads' keys, kv heads' values, query heads. A thread
// owns two chunks of NI tokens of one job; PT = min(page, rows of a pass) tokens a pass, and where a page is shorter than a
// pass several jobs go side by side.
template <int D, int CODE, bool BF16, int NI>
__global__ void __launch_bounds__(kThreads, NI <= 2 ? 3 : 2) append8_kernel(const PagesAppendArgs a, int kv_groups, int kv_per, int q_per) {
    constexpr int C = D / 16, RP = kThreads / C;
    extern __shared__ float2 turn_sh[];   // [page][rot / 2 + 8]
    __shared__ AppendItem item;
    __shared__ int64_t page_id;
    __shared__ uint32_t red[2][kThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    const PagesView& p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == 0) {
        uint32_t bad = 0;
        const int s = find_seq(a.starts, a.s.A, blockIdx.x, p.page, lane);
        const int64_t start = a.starts[s];
        int64_t count = (int64_t)a.starts[s + 1] - start;
        const int64_t i = (int64_t)blockIdx.x - item_base(start, s, p.page);
        if (count < 0 || start < 0 || start + count > a.rows) {
            bad |= kPagesBadLength;
            count = 0;
        }
        AppendItem x;
        int64_t id = -1;
        if (append_item(start, count, a.s.lens[s], i, p.page, &x)) {
            if (x.lp < a.s.max_pages) id = check_page(a.s.table[(int64_t)s * a.s.max_pages + x.lp], p.n_pages, &bad);
            else bad |= kPagesBadLength;
        } else {
            x.n = 0;
        }
        if (lane == 0) {
            if (bad && p.status && blockIdx.y == 0 && blockIdx.z == 0) atomicOr(p.status, bad);
            item = x;
            page_id = id;
        }
    }
    __syncthreads();
    const int n = item.n;
    if (n == 0) return;
    const int64_t id = page_id;
    const int l = blockIdx.z, slot0 = item.slot0;
    // kv heads' keys and values first, then the query heads
    const bool queries = blockIdx.y >= kv_groups;
    const int j0 = queries ? 2 * p.H + (blockIdx.y - kv_groups) * q_per : blockIdx.y * kv_per;
    const int j1 = queries ? min(2 * p.H + a.Hq, j0 + q_per) : min(2 * p.H, j0 + kv_per);
    const int half = a.turns ? a.rot / 2 : 0, row_turns = half + 8;   // rows of turns half a line apart
    if (j0 < p.H || queries)
        for (int i = tid; i < n * half; i += kThreads) {
            const int tok = i / half, f = i - tok * half;
            const uint64_t pos = (uint64_t)(a.positions ? a.positions[item.row0 + tok] : item.lp * p.page + slot0 + tok + a.pos_offset);
            turn_sh[tok * row_turns + Chunks::place(a, f)] = turn_of(pos, __ldg(a.turns + f), a.mscale);
        }
    __syncthreads();
    const int pt = p.page < RP ? p.page : RP, side = RP / pt;   // tokens of a pass, jobs side by side
    const int c = tid % C, row = tid / C, tok0 = row % pt, js = row / pt;
    const int group_warps = pt * C / 32, w0 = js * group_warps;
    const Chunks ch(a, c, C);
    const int64_t unit0 = ((int64_t)(a.s.layer0 + l) * p.n_pages + (id < 0 ? 0 : id)) * p.H;
    if (queries) {   // nothing to agree on: several heads' rows in flight
        for (int tok = tok0; tok < n; tok += RP) {
            float2 cs[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) cs[e] = ch.rot_a ? turn_sh[tok * row_turns + ch.pair(a, e)] : make_float2(1.0f, 0.0f);
            for (int jb = j0 + js; jb < j1; jb += side * kBatch) {
                uint4 x[kBatch], y[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
                    if (jb + b * side < j1) {
                        const uint16_t* src = source(a, l, item.row0 + tok, jb + b * side);
                        x[b] = *reinterpret_cast<const uint4*>(src + 8 * ch.a);
                        y[b] = *reinterpret_cast<const uint4*>(src + 8 * ch.b);
                    }
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
                    if (jb + b * side < j1) {
                        float f[16];
                        spread<BF16>(x[b], y[b], f);
                        if (ch.rot_a) rotate16(f, cs, a.interleaved, ch.rot_b);
                        uint16_t* dst = a.q_out + l * a.qos.layer + (item.row0 + tok) * a.qos.row + (jb + b * side - 2 * p.H) * a.qos.head;
                        *reinterpret_cast<uint4*>(dst + 8 * ch.a) = pack8<BF16>(f);
                        *reinterpret_cast<uint4*>(dst + 8 * ch.b) = pack8<BF16>(f + 8);
                    }
            }
        }
        return;
    }
    uint4 x[NI], y[NI];
    auto load = [&](int j) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int tok = tok0 + i * RP;
            x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
            if (j < j1 && tok < n) {
                const uint16_t* src = source(a, l, item.row0 + tok, j);
                x[i] = *reinterpret_cast<const uint4*>(src + 8 * ch.a);
                y[i] = *reinterpret_cast<const uint4*>(src + 8 * ch.b);
            }
        }
    };
    load(j0 + js);
    int turn = 0;
    for (int jb = j0; jb < j1; jb += side, turn ^= 1) {
        const int j = jb + js;
        const bool here = j < j1;
        float f[NI][16];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            spread<BF16>(x[i], y[i], f[i]);
            if (ch.rot_a && j < p.H && tok0 + i * RP < n) {
                float2 cs[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) cs[e] = turn_sh[(tok0 + i * RP) * row_turns + ch.pair(a, e)];
                rotate16(f[i], cs, a.interleaved, ch.rot_b);
            }
            top = max(top, largest(f[i]));
        }
        load(j + side);   // the next job's rows are on their way over the reduction and the stores
        float old = 0.0f;
        float* sp = nullptr;
        uint8_t* codes = nullptr;
        if (here && id >= 0) {
            const int h = j < p.H ? j : j - p.H;
            sp = p.scales + 2 * (unit0 + h) + (j < p.H ? 0 : 1);
            codes = reinterpret_cast<uint8_t*>(j < p.H ? p.k : p.v) + (unit0 + h) * p.page * D;
            if (slot0 > 0) old = *sp;
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) red[turn][warp] = top;
        __syncthreads();
        if (!codes) continue;   // no job, or the page does not exist
        for (int w = 0; w < group_warps; ++w) top = max(top, red[turn][w0 + w]);
        const float s = scale_with(old, scale_for<CODE>(top));
        if (old != s && slot0 > 0) {   // codes that are there already
            const float ratio = s == s ? old / s : 0.0f;
            for (int i = tok0 * C + c; i < slot0 * (D / 16); i += pt * C) {
                uint4* w = reinterpret_cast<uint4*>(codes) + i;
                *w = recode<CODE>(*w, ratio);
            }
        }
        const float inv = s == s ? 1.0f / s : 0.0f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int tok = tok0 + i * RP;
            if (tok < n) {
                uint8_t* dst = codes + (int64_t)(slot0 + tok) * D;
                if (!(s == s)) {   // codes of a block that reads as NaN: zeros, so that they stay codes
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[i][e] = 0.0f;
                }
                *reinterpret_cast<uint2*>(dst + 8 * ch.a) = codes8<CODE>(f[i], inv);
                *reinterpret_cast<uint2*>(dst + 8 * ch.b) = codes8<CODE>(f[i] + 8, inv);
            }
        }
        if (tok0 == 0 && c == 0) *sp = s;
    }
}

// One token per sequence. grid: (sequences, groups of 256 threads' rows, layers); rows by job as above.
template <int D, int CODE, bool BF16>
__global__ void __launch_bounds__(kThreads) append8_one_kernel(const PagesAppendArgs a) {
    constexpr int C = D / 16;
    __shared__ float2 turn_sh[D / 2];
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    const PagesView& p = a.p;
    const int tid = threadIdx.x, lane = tid & 31;
    const int s = blockIdx.x, l = blockIdx.z;
    const int jobs = 2 * p.H + (a.q ? a.Hq : 0);
    const int j = blockIdx.y * (kThreads / C) + tid / C, c = tid % C;
    const Chunks ch(a, c, C);
    // the row, its sequence's length and its turns: nothing here waits for anything else
    const int64_t len = __ldg(a.s.lens + s);
    uint64_t turns = 0;
    if (a.turns && tid < a.rot / 2) turns = __ldg(a.turns + tid);
    uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
    if (j < jobs) {
        const uint16_t* src = source(a, l, s, j);
        x = *reinterpret_cast<const uint4*>(src + 8 * ch.a);
        y = *reinterpret_cast<const uint4*>(src + 8 * ch.b);
    }
    if (len < 0) return;                    // an idle slot
    uint32_t bad = 0;
    const int64_t lp = len >> page_shift(p.page);
    const int slot = (int)(len & (p.page - 1));
    int64_t id = -1;
    if (lp < a.s.max_pages) id = check_page(__ldg(a.s.table + (int64_t)s * a.s.max_pages + lp), p.n_pages, &bad);
    else bad |= kPagesBadLength;
    if (bad && p.status && tid == 0 && blockIdx.y == 0 && l == 0) atomicOr(p.status, bad);
    const bool kv = j < 2 * p.H && id >= 0;
    const int64_t unit = ((int64_t)(a.s.layer0 + l) * p.n_pages + (id < 0 ? 0 : id)) * p.H + (j < p.H ? j : j - p.H);
    float* sp = p.scales + 2 * unit + (j < p.H ? 0 : 1);
    const float old = kv && slot > 0 ? *sp : 0.0f;
    if (a.turns && tid < a.rot / 2)
        turn_sh[Chunks::place(a, tid)] = turn_of((uint64_t)(a.positions ? __ldg(a.positions + s) : len + a.pos_offset), turns, a.mscale);
    __syncthreads();
    float f[16];
    spread<BF16>(x, y, f);
    if (ch.rot_a && (j < p.H || j >= 2 * p.H)) {
        float2 cs[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) cs[e] = turn_sh[ch.pair(a, e)];
        rotate16(f, cs, a.interleaved, ch.rot_b);
    }
    if (j >= 2 * p.H && j < jobs) {
        uint16_t* dst = a.q_out + l * a.qos.layer + s * a.qos.row + (j - 2 * p.H) * a.qos.head;
        *reinterpret_cast<uint4*>(dst + 8 * ch.a) = pack8<BF16>(f);
        *reinterpret_cast<uint4*>(dst + 8 * ch.b) = pack8<BF16>(f + 8);
    }
    // from here the warp stays together: its rows' lanes agree on their scales, and it moves earlier codes as one
    uint32_t top = largest(f);
#pragma unroll
    for (int o = 1; o < C; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float sc = scale_with(old, scale_for<CODE>(top));
    uint8_t* codes = reinterpret_cast<uint8_t*>(j < p.H ? p.k : p.v) + unit * p.page * D;
    uint32_t moves = __ballot_sync(0xffffffffu, kv && slot > 0 && old != sc && c == 0);
    while (moves) {
        const int from = __ffs(moves) - 1;
        moves &= moves - 1;
        const float so = __shfl_sync(0xffffffffu, old, from), sn = __shfl_sync(0xffffffffu, sc, from);
        uint4* w = reinterpret_cast<uint4*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(codes), from));
        const float ratio = sn == sn ? so / sn : 0.0f;
#pragma unroll 4
        for (int i = lane; i < slot * (D / 16); i += 32) w[i] = recode<CODE>(w[i], ratio);
    }
    if (!kv) return;
    if (!(sc == sc)) {
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = 0.0f;
    }
    const float inv = sc == sc ? 1.0f / sc : 0.0f;
    uint8_t* dst = codes + (int64_t)slot * D;
    *reinterpret_cast<uint2*>(dst + 8 * ch.a) = codes8<CODE>(f, inv);
    *reinterpret_cast<uint2*>(dst + 8 * ch.b) = codes8<CODE>(f + 8, inv);
    if (c == 0) *sp = sc;
}

template <int D, int CODE, bool BF16>
polykv_status run(const PagesAppendArgs& a, cudaStream_t st) {
    constexpr int RP = kThreads / (D / 16);
    const int jobs = 2 * a.p.H + (a.q ? a.Hq : 0);
    cudaError_t e;
    if (!a.starts) {
        e = launch_after(append8_one_kernel<D, CODE, BF16>, dim3((unsigned)a.s.A, (unsigned)((jobs + RP - 1) / RP), (unsigned)a.s.nl),
                         kThreads, 0, st, a);
        return e == cudaSuccess ? POLYKV_OK : set_error(POLYKV_E_CUDA, "pages_append launch: %s", cudaGetErrorString(e));
    }
    const int64_t items = a.rows / a.p.page + 2 * (int64_t)a.s.A;
    // Heads per block: sixteen query heads (four turns of kBatch) and eight of keys or values, which share the cosines (their turns
    // in shared memory cost a block about what two heads cost); fewer where that leaves SMs without a block.
    const int side = a.p.page < RP ? RP / a.p.page : 1;
    const int64_t want = 3 * (int64_t)device_sm_count() / (a.q ? 2 : 1), per_layer = items * a.s.nl;
    auto per_group = [&](int heads, int most) {
        int64_t per = most;
        while (per > side && per_layer * ((heads + per - 1) / per) < want) per /= 2;
        return (int)((per + side - 1) / side * side);
    };
    const int kv_per = per_group(2 * a.p.H, 8 * side), q_per = per_group(a.Hq, 16 * side);
    const int kv_groups = (2 * a.p.H + kv_per - 1) / kv_per, groups = kv_groups + (a.q ? (a.Hq + q_per - 1) / q_per : 0);
    const size_t smem = a.turns ? (size_t)a.p.page * (a.rot / 2 + 8) * sizeof(float2) : 0;
    const dim3 grid((unsigned)items, (unsigned)groups, (unsigned)a.s.nl);
    auto go = [&](auto kern) {
        // the limit stands for the process: always the same, whatever this call needs
        cudaError_t x = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * (D / 2 + 8) * (int)sizeof(float2));
        return x == cudaSuccess ? launch_after(kern, grid, kThreads, smem, st, a, kv_groups, kv_per, q_per) : x;
    };
    switch (a.p.page / RP) {   // tokens of a page per thread
        case 0:
        case 1: e = go(append8_kernel<D, CODE, BF16, 1>); break;
        case 2: e = go(append8_kernel<D, CODE, BF16, 2>); break;
        default: e = go(append8_kernel<D, CODE, BF16, 128 / RP>); break;
    }
    return e == cudaSuccess ? POLYKV_OK : set_error(POLYKV_E_CUDA, "pages_append launch: %s", cudaGetErrorString(e));
}

template <int CODE>
polykv_status run_code(const PagesAppendArgs& a, bool bf, cudaStream_t st) {
    if (a.p.d == 128) return bf ? run<128, CODE, true>(a, st) : run<128, CODE, false>(a, st);
    return bf ? run<64, CODE, true>(a, st) : run<64, CODE, false>(a, st);
}

// A value in the row's type; one that is finite stays so (the largest e4m3 codes of an f16 block may pass f16's end by half a step).
template <bool BF16>
__device__ __forceinline__ float within(float x) {
    if constexpr (BF16) return x;
    else return fabsf(x) < INFINITY ? fminf(fmaxf(x, -65504.0f), 65504.0f) : x;
}

// Eight codes under a scale as values in the row's type.
template <int CODE, bool BF16>
__device__ __forceinline__ uint4 wide(const uint2& c, float s) {
    const float4 x = value4<CODE>(c.x), y = value4<CODE>(c.y);
    return make_uint4(pack_rn<BF16>(within<BF16>(x.x * s), within<BF16>(x.y * s)), pack_rn<BF16>(within<BF16>(x.z * s), within<BF16>(x.w * s)),
                      pack_rn<BF16>(within<BF16>(y.x * s), within<BF16>(y.y * s)), pack_rn<BF16>(within<BF16>(y.z * s), within<BF16>(y.w * s)));
}

// ------------------------------------------------------------------ tokens back as rows
// Eight elements of a row per thread and turn, rows of a token's heads next to each other on both sides. grid: (items, layers,
// shares of the tokens).
template <int CODE, bool BF16>
__global__ void __launch_bounds__(kThreads) gather_kernel(const PagesGatherArgs a) {
    __shared__ AppendItem item;
    __shared__ int64_t page_id;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    const PagesView& p = a.p;
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid < 32) {
        uint32_t bad = 0;
        const int s = find_seq(a.starts, a.s.A, blockIdx.x, p.page, lane);
        const int64_t start = a.starts[s];
        int64_t count = (int64_t)a.starts[s + 1] - start;
        const int64_t i = (int64_t)blockIdx.x - item_base(start, s, p.page);
        const int64_t len = a.s.lens[s];
        if (count < 0 || start < 0 || start + count > a.rows || (count > len && len >= 0)) {
            bad |= kPagesBadLength;
            count = 0;
        }
        AppendItem x;
        int64_t id = -1;
        if (len >= 0 && append_item(start, count, len - count, i, p.page, &x)) {
            if (x.lp < a.s.max_pages) id = check_page(a.s.table[(int64_t)s * a.s.max_pages + x.lp], p.n_pages, &bad);
            else bad |= kPagesBadLength;
        } else {
            x.n = 0;
        }
        if (lane == 0) {
            if (bad && p.status && blockIdx.y == 0 && blockIdx.z == 0) atomicOr(p.status, bad);
            item = x;
            page_id = id;
        }
    }
    __syncthreads();
    if (item.n == 0 || page_id < 0) return;
    const int l = blockIdx.y, per_row = p.d / 8, per_tok = p.H * per_row;
    const int64_t unit0 = ((int64_t)(a.s.layer0 + l) * p.n_pages + page_id) * p.H;
    const int total = item.n * per_tok;
#pragma unroll 4
    for (int i = blockIdx.z * kThreads + tid; i < total; i += gridDim.z * kThreads) {
        const int tok = i / per_tok, rest = i - tok * per_tok, h = rest / per_row, ch = rest - h * per_row;
        const int64_t at = ((unit0 + h) * p.page + item.slot0 + tok) * p.d + 8 * ch;
        const int64_t to = (((int64_t)l * a.rows + item.row0 + tok) * p.H + h) * p.d + 8 * ch;
        if constexpr (CODE == kPagesWide) {
            *reinterpret_cast<uint4*>(a.k + to) = *reinterpret_cast<const uint4*>(p.k + at);
            *reinterpret_cast<uint4*>(a.v + to) = *reinterpret_cast<const uint4*>(p.v + at);
        } else {
            const float2 s = __ldg(reinterpret_cast<const float2*>(p.scales) + unit0 + h);
            const uint2 kw = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(p.k) + at);
            const uint2 vw = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(p.v) + at);
            *reinterpret_cast<uint4*>(a.k + to) = wide<CODE, BF16>(kw, s.x);
            *reinterpret_cast<uint4*>(a.v + to) = wide<CODE, BF16>(vw, s.y);
        }
    }
}

// ------------------------------------------------------------------ pages of codes as 16-bit pages
// The pages that a sequence's rows see: each to the place [layer][page id] (sequences that share a page write the same bits), or,
// with a table to write, to [layer][sequence][logical page]. places: of a layer. grid: (shares of the pages, sequences, layers).
template <int CODE, bool BF16>
__global__ void __launch_bounds__(kThreads) expand_kernel(const PagesRowsArgs a, uint16_t* __restrict__ k, uint16_t* __restrict__ v,
                                                          const int64_t places, int32_t* __restrict__ table) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    const PagesView& p = a.p;
    const int s = blockIdx.y, l = blockIdx.z, tid = threadIdx.x, shift = page_shift(p.page);
    uint32_t bad = 0;   // the call's kernel says so
    const int64_t len = clamp_len(a.s.lens[s], a.s.max_pages, p.page, &bad), count = (int64_t)a.starts[s + 1] - a.starts[s];
    if (count <= 0) return;
    const int64_t first = len > count ? len - count : 0;   // the first row's place
    const Window w = window_of(first + 1, p.page, a.window, a.sinks);
    const int64_t lead = pages_of(w.sinks, p.page), from = w.begin >> shift, pages = pages_of(len, p.page);
    const int words = p.H * p.page * p.d / 8;              // of eight codes
    for (int64_t lp = blockIdx.x; lp < pages; lp += gridDim.x) {
        if (lp >= lead && lp < from) continue;
        const int64_t id = check_page(a.s.table[(int64_t)s * a.s.max_pages + lp], p.n_pages, &bad);
        const int64_t to = table ? (int64_t)s * a.s.max_pages + lp : id;
        if (table && l == 0 && tid == 0) table[to] = id < 0 ? -1 : (int32_t)to;
        if (id < 0) continue;
        const int64_t unit0 = ((int64_t)(a.s.layer0 + l) * p.n_pages + id) * p.H;
        const int64_t out0 = ((int64_t)l * places + to) * words;
        const uint2* kc = reinterpret_cast<const uint2*>(p.k) + unit0 * p.page * p.d / 8;
        const uint2* vc = reinterpret_cast<const uint2*>(p.v) + unit0 * p.page * p.d / 8;
#pragma unroll 4
        for (int i = tid; i < words; i += kThreads) {
            const float2 u = __ldg(reinterpret_cast<const float2*>(p.scales) + unit0 + i / (p.page * p.d / 8));
            reinterpret_cast<uint4*>(k)[out0 + i] = wide<CODE, BF16>(kc[i], u.x);
            reinterpret_cast<uint4*>(v)[out0 + i] = wide<CODE, BF16>(vc[i], u.y);
        }
    }
}

}  // namespace

polykv_status launch_pages_expand(const PagesRowsArgs& a, polykv_dtype dt, uint16_t* k, uint16_t* v, int64_t places, int32_t* table,
                                  cudaStream_t st) {
    const bool bf = dt == POLYKV_BF16;
    const int64_t want = 8 * (int64_t)device_sm_count() / ((int64_t)a.s.A * a.s.nl);
    const dim3 grid((unsigned)(want < 1 ? 1 : (want < a.s.max_pages ? want : a.s.max_pages)), (unsigned)a.s.A, (unsigned)a.s.nl);
    auto go = [&](auto kern) { return launch_after(kern, grid, kThreads, 0, st, a, k, v, places, table); };
    const cudaError_t e = a.p.code == kPagesInt8 ? (bf ? go(expand_kernel<kPagesInt8, true>) : go(expand_kernel<kPagesInt8, false>))
                                                 : (bf ? go(expand_kernel<kPagesE4m3, true>) : go(expand_kernel<kPagesE4m3, false>));
    return e == cudaSuccess ? POLYKV_OK : set_error(POLYKV_E_CUDA, "pages_attend_rows launch: %s", cudaGetErrorString(e));
}

polykv_status launch_pages_append8(const PagesAppendArgs& a, polykv_dtype dt, cudaStream_t st) {
    const bool bf = dt == POLYKV_BF16;
    return a.p.code == kPagesInt8 ? run_code<kPagesInt8>(a, bf, st) : run_code<kPagesE4m3>(a, bf, st);
}

polykv_status launch_pages_gather(const PagesGatherArgs& a, polykv_dtype dt, cudaStream_t st) {
    const bool bf = dt == POLYKV_BF16;
    const int64_t items = a.rows / a.p.page + 2 * (int64_t)a.s.A, want = 8 * (int64_t)device_sm_count();
    // as many blocks as are resident at once, while each thread has four chunks of a whole page
    int64_t shares = (want + items * a.s.nl - 1) / (items * a.s.nl);
    const int64_t most = (int64_t)a.p.page * a.p.H * (a.p.d / 8) / (4 * kThreads);
    shares = shares < most ? shares : most;
    const dim3 grid((unsigned)items, (unsigned)a.s.nl, (unsigned)(shares > 1 ? shares : 1));
    auto go = [&](auto kern) { return launch_after(kern, grid, kThreads, 0, st, a); };
    const cudaError_t e = a.p.code == kPagesWide   ? go(gather_kernel<kPagesWide, true>)
                          : a.p.code == kPagesInt8 ? (bf ? go(gather_kernel<kPagesInt8, true>) : go(gather_kernel<kPagesInt8, false>))
                                                   : (bf ? go(gather_kernel<kPagesE4m3, true>) : go(gather_kernel<kPagesE4m3, false>));
    return e == cudaSuccess ? POLYKV_OK : set_error(POLYKV_E_CUDA, "pages_gather launch: %s", cudaGetErrorString(e));
}

}  // namespace polykv
