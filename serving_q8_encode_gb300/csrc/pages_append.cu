// Appending keys and values to a paged cache, with the position rotation applied on the way.
//
//   k'[2 dims of pair j] = R(pos f_j) k[...]    R the rotation of a pair by an angle; f_j radians per position
//   q' likewise; v as it is; k' and v to the token's slot, q' to q_out
//   bounds[page][0 / 1] = lowest / highest k' over the page's tokens, per coordinate
//
// Every element is read once and written once: HBM binds long appends, latency the short ones. The angle
// would need 64 bits at far positions (pos f_j has to be known to about 1e-7 modulo 2 pi), so it is kept in
// turns as a 64-bit fixed-point fraction: pos * turns_j wraps modulo one turn by itself, exact to
// pos * 2^-65 turns, in integer arithmetic.
//
// Runs of tokens: one block takes one page's share of the new tokens (so that it alone folds the page's bounds)
// and a group of heads; a thread owns two 16-byte chunks of one token's rows that hold 8 pairs between them,
// computes the 8 cosines and sines once, and goes through the heads. One token per sequence (a decode step): a
// block takes a sequence and a group of heads, a thread one row's two chunks, and everything that does not
// depend on something else is on its way at once.
//
// Measured (bf16, 8 kv heads x 4 query heads, d = 128, with q): one token for each of 15 or 256 sequences 4.3 us,
// back to back (256 in the general kernel: 12.2 us); a prompt of 7,194 tokens 33.1 us = 5.3 TB/s, one wave of 456
// blocks; 24 layers of five ragged prompts at SmolLM2's shape (3.7 GB) 585 us = 6.3 TB/s. Two or four resident
// blocks instead of three: 743 and 622 us for the last; streaming store hints: 670 us; twice the rows a thread: 704 us.
#include "pages_internal.cuh"

namespace polykv {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;   // rows in flight per thread (2: 624 us, 8: 640 us against 588 us for the 3.7 GB above)
constexpr int kPerSm = 3;   // resident blocks of the kernel for runs of tokens
constexpr int kOld = 8;     // earlier keys in flight per lane

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&w));
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
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    if constexpr (BF16) {
        const __nv_bfloat162 r = __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    } else {
        const __half2 r = __hmin2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
}
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    if constexpr (BF16) {
        const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    } else {
        const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
}

// Rotates the 8 pairs that two chunks hold: (x[i], y[i]) when the halves are paired, neighbours otherwise.
// Products and sums in fp32, one rounding to the input type.
template <bool BF16>
__device__ __forceinline__ void rotate(uint4& x, uint4& y, const float (&cs)[8], const float (&sn)[8], bool interleaved) {
    uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
    uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = unpack2<BF16>(xw[i]), b = unpack2<BF16>(yw[i]);
        if (interleaved) {
            xw[i] = pack_rn<BF16>(a.x * cs[i] - a.y * sn[i], a.y * cs[i] + a.x * sn[i]);
            yw[i] = pack_rn<BF16>(b.x * cs[4 + i] - b.y * sn[4 + i], b.y * cs[4 + i] + b.x * sn[4 + i]);
        } else {
            xw[i] = pack_rn<BF16>(a.x * cs[2 * i] - b.x * sn[2 * i], a.y * cs[2 * i + 1] - b.y * sn[2 * i + 1]);
            yw[i] = pack_rn<BF16>(b.x * cs[2 * i] + a.x * sn[2 * i], b.y * cs[2 * i + 1] + a.y * sn[2 * i + 1]);
        }
    }
}

// Cosine and sine of pos * turns, from the fraction of a turn in [-1/2, 1/2): the special function unit's, whose
// documented error in [-pi, pi] is below 2^-21.1 absolute, 2^9 (bf16) or 2^6 (f16) times finer than the
// outputs' half step.
__device__ __forceinline__ void cos_sin(uint64_t pos, uint64_t turns, float mscale, float* c, float* s) {
    const int32_t frac = (int32_t)((pos * turns) >> 32);                  // in units of 2^-32 turns
    const float x = (float)frac * (6.283185307179586f / 4294967296.0f);   // radians
    *c = __cosf(x) * mscale;
    *s = __sinf(x) * mscale;
}

// The sequence that owns an append item (all lanes of the warp get it).
__device__ __forceinline__ int find_seq(const int32_t* starts, int A, int64_t item, int page, int lane) {
    int lo = 0, n = A;
    while (n > 1) {
        const int stride = (n + 31) / 32;
        const int i = lane * stride;
        const bool le = i < n && item_base(starts[lo + i], lo + i, page) <= item;
        const int cnt = max(1, __popc(__ballot_sync(0xffffffffu, le)));
        lo += (cnt - 1) * stride;
        n = min(stride, n - (cnt - 1) * stride);
    }
    return lo;
}

// grid: (items, head groups, layers). Jobs are rows by head: kv heads' keys, kv heads' values, query heads.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, kPerSm) pages_append_kernel(const PagesAppendArgs a, int jobs_per_group, int tb) {
    constexpr int C = D / 16;      // threads per token row
    __shared__ AppendItem item;
    __shared__ int64_t page_id;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    const PagesView& p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == 0) {
        const int64_t it = blockIdx.x;
        uint32_t bad = 0;
        const int s = find_seq(a.starts, a.s.A, it, p.page, lane);
        const int64_t start = a.starts[s];
        int64_t count = (int64_t)a.starts[s + 1] - start;
        const int64_t i = it - item_base(start, s, p.page);
        if (count < 0 || start < 0 || start + count > a.rows) {
            bad |= kPagesBadLength;
            count = 0;
        }
        AppendItem x;
        x.n = 0;
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
    const int l = blockIdx.z;
    const int jobs = 2 * p.H + (a.q ? a.Hq : 0);
    const int j0 = blockIdx.y * jobs_per_group, j1 = min(jobs, j0 + jobs_per_group);
    const int c = tid % C, rest = tid / C;
    const int tok0 = rest % tb, slot_j = rest / tb, nslots = kThreads / C / tb;
    const int64_t page_elems = (int64_t)p.H * p.page * D;
    const int64_t block0 = ((int64_t)(a.s.layer0 + l) * p.n_pages + (id < 0 ? 0 : id)) * page_elems;
    const int rc = a.turns ? a.rot / 16 : 0;   // threads of a row that rotate
    // this thread's two chunks, and whether they rotate
    const int ca = a.interleaved || c < rc ? c : 2 * rc + 2 * (c - rc);
    const int cb = a.interleaved ? c + C : (c < rc ? c + rc : ca + 1);
    const bool rot_a = ca < (a.interleaved ? 2 * rc : rc), rot_b = a.interleaved ? cb < 2 * rc : rot_a;

    for (int tok = tok0; tok < n; tok += tb) {
        const int64_t r = item.row0 + tok;
        float cs[8], sn[8];
        if (rot_a && (j0 < p.H || j1 > 2 * p.H)) {
            const int64_t place = item.lp * p.page + item.slot0 + tok;
            const uint64_t pos = (uint64_t)(a.positions ? a.positions[r] : place + a.pos_offset);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int f = a.interleaved ? (i < 4 ? 4 * ca + i : 4 * (rot_b ? cb : ca) + i - 4) : 8 * c + i;
                cos_sin(pos, __ldg(a.turns + f), a.mscale, &cs[i], &sn[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                cs[i] = 1.0f;
                sn[i] = 0.0f;
            }
        }
        for (int jb = j0 + slot_j; jb < j1; jb += nslots * kBatch) {
            uint4 x[kBatch], y[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int j = jb + b * nslots;
                if (j < j1) {
                    const uint16_t* src = j < p.H ? a.k + l * a.ks.layer + r * a.ks.row + j * a.ks.head
                                          : j < 2 * p.H ? a.v + l * a.vs.layer + r * a.vs.row + (j - p.H) * a.vs.head
                                                        : a.q + l * a.qs.layer + r * a.qs.row + (j - 2 * p.H) * a.qs.head;
                    x[b] = *reinterpret_cast<const uint4*>(src + 8 * ca);
                    y[b] = *reinterpret_cast<const uint4*>(src + 8 * cb);
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int j = jb + b * nslots;
                if (j < j1) {
                    uint16_t* dst;
                    if (j < 2 * p.H) {
                        if (id < 0) continue;   // the page does not exist: nothing to write to
                        const int h = j < p.H ? j : j - p.H;
                        dst = (j < p.H ? p.k : p.v) + block0 + ((int64_t)h * p.page + item.slot0 + tok) * D;
                    } else {
                        dst = a.q_out + l * a.qos.layer + r * a.qos.row + (j - 2 * p.H) * a.qos.head;
                    }
                    if (rot_a && (j < p.H || j >= 2 * p.H)) {
                        const uint4 y0 = y[b];
                        rotate<BF16>(x[b], y[b], cs, sn, a.interleaved);
                        if (!rot_b) y[b] = y0;
                    }
                    *reinterpret_cast<uint4*>(dst + 8 * ca) = x[b];
                    *reinterpret_cast<uint4*>(dst + 8 * cb) = y[b];
                }
            }
        }
    }
    if (!p.bounds || id < 0 || j0 >= p.H) return;
    // ---- the page's bounds over its tokens [0, slot0 + n): one warp per kv head of the group, D/8 lanes a row
    __syncthreads();   // the block's own key stores
    constexpr int LR = D / 8;      // lanes per row
    constexpr int TS = 32 / LR;    // rows a warp reads at once
    const int ch = lane % LR, ts = lane / LR;
    const int end = item.slot0 + n;
    for (int h = j0 + warp; h < min(j1, p.H); h += kThreads / 32) {
        const uint16_t* rows = p.k + block0 + (int64_t)h * p.page * D + 8 * ch;
        uint32_t lo[4], hi[4];
        const uint4 f = *reinterpret_cast<const uint4*>(rows + (int64_t)min(ts, end - 1) * D);
        lo[0] = hi[0] = f.x;
        lo[1] = hi[1] = f.y;
        lo[2] = hi[2] = f.z;
        lo[3] = hi[3] = f.w;
#pragma unroll 4
        for (int tt = ts + TS; tt < end; tt += TS) {
            const uint4 w = *reinterpret_cast<const uint4*>(rows + (int64_t)tt * D);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] = min2<BF16>(lo[i], ww[i]);
                hi[i] = max2<BF16>(hi[i], ww[i]);
            }
        }
#pragma unroll
        for (int o = LR; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] = min2<BF16>(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
                hi[i] = max2<BF16>(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
            }
        uint16_t* b = p.bounds + (((int64_t)(a.s.layer0 + l) * p.n_pages + id) * p.H + h) * 2 * D + 8 * ch;
        if (ts == 0) *reinterpret_cast<uint4*>(b) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (ts == 1) *reinterpret_cast<uint4*>(b + D) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
}

// One token per sequence. grid: (sequences, groups of 256 threads' rows, layers); rows by head as above.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) pages_append_one_kernel(const PagesAppendArgs a) {
    constexpr int C = D / 16;               // threads per row
    constexpr int kRows = kThreads / C;     // rows of a block
    __shared__ float cs_sh[D / 2], sn_sh[D / 2];
    __shared__ __align__(16) uint4 new_key[kRows][D / 8];
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    const PagesView& p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = blockIdx.x, l = blockIdx.z;
    const int jobs = 2 * p.H + (a.q ? a.Hq : 0);
    const int j0 = blockIdx.y * kRows, j = j0 + tid / C, c = tid % C;
    const int rc = a.turns ? a.rot / 16 : 0;
    const int ca = a.interleaved || c < rc ? c : 2 * rc + 2 * (c - rc);
    const int cb = a.interleaved ? c + C : (c < rc ? c + rc : ca + 1);
    const bool rot_a = ca < (a.interleaved ? 2 * rc : rc), rot_b = a.interleaved ? cb < 2 * rc : rot_a;
    // the row, its sequence's length and its turns: nothing here waits for anything else
    const int64_t len = __ldg(a.s.lens + s);
    uint64_t turns = 0;
    if (a.turns && tid < a.rot / 2) turns = __ldg(a.turns + tid);
    uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
    if (j < jobs) {
        const uint16_t* src = j < p.H       ? a.k + l * a.ks.layer + s * a.ks.row + j * a.ks.head
                              : j < 2 * p.H ? a.v + l * a.vs.layer + s * a.vs.row + (j - p.H) * a.vs.head
                                            : a.q + l * a.qs.layer + s * a.qs.row + (j - 2 * p.H) * a.qs.head;
        x = *reinterpret_cast<const uint4*>(src + 8 * ca);
        y = *reinterpret_cast<const uint4*>(src + 8 * cb);
    }
    if (len < 0) return;                    // an idle slot
    uint32_t bad = 0;
    const int shift = page_shift(p.page);
    const int64_t lp = len >> shift;
    const int slot = (int)(len & (p.page - 1));
    int64_t id = -1;
    if (lp < a.s.max_pages) id = check_page(__ldg(a.s.table + (int64_t)s * a.s.max_pages + lp), p.n_pages, &bad);
    else bad |= kPagesBadLength;
    if (bad && p.status && tid == 0 && blockIdx.y == 0 && l == 0) atomicOr(p.status, bad);
    if (a.turns && tid < a.rot / 2)
        cos_sin((uint64_t)(a.positions ? __ldg(a.positions + s) : len + a.pos_offset), turns, a.mscale, &cs_sh[tid], &sn_sh[tid]);
    const int64_t block0 = ((int64_t)(a.s.layer0 + l) * p.n_pages + (id < 0 ? 0 : id)) * p.H * p.page * D;
    // a warp per kv head of the group folds the bounds; its first head's earlier keys are on their way before the
    // barrier. Lane: chunk ch of rows ts, ts + TS, ...
    constexpr int LR = D / 8, TS = 32 / LR;
    const int ch = lane % LR, ts = lane / LR;
    const int h_end = min(j0 + kRows, p.H);
    const bool folds = p.bounds && id >= 0;
    uint4 old[kOld];
    auto load_old = [&](int h, int t0) {
        const uint16_t* rows = p.k + block0 + (int64_t)h * p.page * D + 8 * ch;
#pragma unroll
        for (int e = 0; e < kOld; ++e) {
            const int t = t0 + e * TS + ts;
            if (t < slot) old[e] = *reinterpret_cast<const uint4*>(rows + (int64_t)t * D);
        }
    };
    if (folds && j0 + warp < h_end) load_old(j0 + warp, 0);
    __syncthreads();
    if (j < jobs) {
        if (rot_a && (j < p.H || j >= 2 * p.H)) {
            float cs[8], sn[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int f = a.interleaved ? (i < 4 ? 4 * ca + i : 4 * (rot_b ? cb : ca) + i - 4) : 8 * c + i;
                cs[i] = cs_sh[f];
                sn[i] = sn_sh[f];
            }
            const uint4 y0 = y;
            rotate<BF16>(x, y, cs, sn, a.interleaved);
            if (!rot_b) y = y0;
        }
        uint16_t* dst = nullptr;
        if (j >= 2 * p.H) {
            dst = a.q_out + l * a.qos.layer + s * a.qos.row + (j - 2 * p.H) * a.qos.head;
        } else if (id >= 0) {               // a page that does not exist is not written
            const int h = j < p.H ? j : j - p.H;
            dst = (j < p.H ? p.k : p.v) + block0 + ((int64_t)h * p.page + slot) * D;
        }
        if (dst) {
            *reinterpret_cast<uint4*>(dst + 8 * ca) = x;
            *reinterpret_cast<uint4*>(dst + 8 * cb) = y;
        }
        if (j < p.H) {
            new_key[j - j0][ca] = x;
            new_key[j - j0][cb] = y;
        }
    }
    if (!folds || j0 >= p.H) return;
    __syncthreads();
    for (int h = j0 + warp; h < h_end; h += kThreads / 32) {
        const uint4 f = new_key[h - j0][ch];
        uint32_t lo[4] = {f.x, f.y, f.z, f.w}, hi[4] = {f.x, f.y, f.z, f.w};
        for (int t0 = 0; t0 < slot; t0 += kOld * TS) {
            if (t0 > 0 || h >= j0 + kThreads / 32) load_old(h, t0);
#pragma unroll
            for (int e = 0; e < kOld; ++e)
                if (t0 + e * TS + ts < slot) {
                    const uint32_t w[4] = {old[e].x, old[e].y, old[e].z, old[e].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        lo[i] = min2<BF16>(lo[i], w[i]);
                        hi[i] = max2<BF16>(hi[i], w[i]);
                    }
                }
        }
#pragma unroll
        for (int o = LR; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] = min2<BF16>(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
                hi[i] = max2<BF16>(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
            }
        uint16_t* b = p.bounds + (((int64_t)(a.s.layer0 + l) * p.n_pages + id) * p.H + h) * 2 * D + 8 * ch;
        if (ts == 0) *reinterpret_cast<uint4*>(b) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (ts == 1) *reinterpret_cast<uint4*>(b + D) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
}

template <int D, bool BF16>
polykv_status run(const PagesAppendArgs& a, cudaStream_t st) {
    const int jobs = 2 * a.p.H + (a.q ? a.Hq : 0);
    cudaError_t e;
    if (!a.starts) {
        constexpr int rows = kThreads / (D / 16);
        e = launch_after(pages_append_one_kernel<D, BF16>,
                         dim3((unsigned)a.s.A, (unsigned)((jobs + rows - 1) / rows), (unsigned)a.s.nl), kThreads, 0, st, a);
        if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_append launch: %s", cudaGetErrorString(e));
        return POLYKV_OK;
    }
    const int64_t items = a.rows / a.p.page + 2 * (int64_t)a.s.A;
    const int tb = a.p.page < 32 ? a.p.page : 32;   // tokens a block works on at once
    // Heads per block: as many blocks as are resident at once where the call is small, else 16 rows a thread, which
    // share the cosines.
    const int64_t per_layer = items * a.s.nl;
    const int64_t want = kPerSm * (int64_t)device_sm_count();
    int groups = (int)((want + per_layer - 1) / per_layer);
    const int slots = kThreads / (D / 16) / tb;
    const int floor_groups = (jobs + 16 * slots - 1) / (16 * slots);
    if (groups < floor_groups) groups = floor_groups;
    if (groups > jobs) groups = jobs;
    const int per = (jobs + groups - 1) / groups;
    groups = (jobs + per - 1) / per;
    e = launch_after(pages_append_kernel<D, BF16>, dim3((unsigned)items, (unsigned)groups, (unsigned)a.s.nl), kThreads, 0, st,
                     a, per, tb);
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages_append launch: %s", cudaGetErrorString(e));
    return POLYKV_OK;
}

}  // namespace

polykv_status launch_pages_append(const PagesAppendArgs& a, polykv_dtype dt, cudaStream_t st) {
    const bool bf = dt == POLYKV_BF16;
    if (a.p.d == 128) return bf ? run<128, true>(a, st) : run<128, false>(a, st);
    return bf ? run<64, true>(a, st) : run<64, false>(a, st);
}

}  // namespace polykv
