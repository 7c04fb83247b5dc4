// Block tables and slot maps from request lengths, on the GPU: which pages a step's new tokens take, where each row goes, and
// which pages come back.
//
// State: table [A][max_pages], lens [A] (negative: idle), first [A] (the first page behind the sinks that is still held), and
// the free pages as a ring with two running counters, head (pages taken so far) and tail (pages given so far): pages
// ring[head .. tail) modulo n_pages are free. Pages that come back go to the tail, so that a call that takes and gives at the
// same time never writes a place that it reads: the two ranges would meet only if more than n_pages were free.
//
//   plan:  need_s = ceil((len_s + new_s) / page) - ceil(len_s / page), from the ring in slot order while sum need <= free;
//          starts = exclusive sum of new; row r of slot s: place len_s + r - starts_s, slot id * page + place mod page;
//          with a window, pages wholly before place len_s + 1 - window and behind the sinks come back.
//   cut:   pages behind the first keep_s tokens come back.
//
// A few bytes per slot and 16 per row: latency binds all but the largest. Every CTA makes the sums over the slots for itself
// (at most 4,096, from three arrays that L2 holds; up to 256 in one warp, without a barrier) instead of waiting for one that does; the
// work that is long, rows and pages, is shared out flat. The last CTA to have read the state writes the new one (an arrival
// count; nobody waits).
//
// Measured, a cut and a plan: 15 slots of four tokens 6.5 us (sums by all warps: 8.2 us), 512 slots with 64 prompts 10.3 us (12.9).
#include "pages_internal.cuh"

namespace polykv {
namespace {

constexpr int kThreads = 512;
constexpr int kPer = kPagesMaxSeqs / kThreads;   // slots per thread at most

constexpr int kWarpSlots = 32 * kPer;            // slots that one warp sums up without a barrier

struct Sums {   // in shared memory, [A + 1] each, exclusive with the total behind the last
    int32_t *rows, *take, *give, *old;   // old: the slots' tokens
    __device__ __forceinline__ Sums(void* smem, int A) {
        rows = static_cast<int32_t*>(smem);
        take = rows + A + 1;
        give = take + A + 1;
        old = give + A + 1;
    }
};
size_t sums_bytes(int A) { return 4 * (size_t)(A + 1) * sizeof(int32_t); }
struct Scratch {
    int64_t warps[kThreads / 32];
    int32_t most;
    int last;
};

// Exclusive sum over the block's threads, or (alone) over one warp's.
__device__ __forceinline__ int64_t scan(int64_t x, bool alone, int64_t* warps, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (alone) {
        *total = __shfl_sync(0xffffffffu, inc, 31);
        return inc - x;
    }
    if (lane == 31) warps[warp] = inc;
    __syncthreads();
    int64_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) base = all;
        all += warps[w];
    }
    __syncthreads();
    *total = all;
    return base + inc - x;
}

// The last slot whose sum is at most i (it has items).
template <class T>
__device__ __forceinline__ int slot_of(const T* sums, int A, T i) {
    int lo = 0, hi = A - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sums[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// One block more has read the state; true in all threads of the one that came last (which leaves the count at zero).
__device__ __forceinline__ bool arrived_last(const PageTablesArgs& t, Scratch& sc) {
    if (gridDim.x == 1) {   // nobody else reads it
        __syncthreads();
        return true;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t before;
        asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(before) : "l"(t.arrivals), "r"(gridDim.x - 1) : "memory");
        sc.last = before == gridDim.x - 1;
    }
    __syncthreads();
    return sc.last != 0;
}

// A counter's place in the ring.
__device__ __forceinline__ int64_t ring_place(int64_t count, int64_t n) {
    const int64_t c = count < 0 ? 0 : count;   // none of these calls' is negative
    return c - (int64_t)quotient((uint64_t)c, (uint64_t)n) * n;
}
__device__ __forceinline__ int64_t ring_at(int64_t from, int64_t i, int64_t n) {   // from in [0, n), i in [0, n]
    const int64_t x = from + i;
    return x >= n ? x - n : x;
}

__global__ void __launch_bounds__(kThreads) tables_plan_kernel(const PageTablesArgs t, const int32_t* __restrict__ fresh, const int64_t n_rows,
                                                               int32_t* __restrict__ starts, int32_t* __restrict__ before,
                                                               int32_t* __restrict__ after, int64_t* __restrict__ slots,
                                                               int64_t* __restrict__ positions) {
    extern __shared__ int32_t smem[];
    const Sums sum(smem, t.A);
    __shared__ Scratch sc;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    const int tid = threadIdx.x, A = t.A, shift = page_shift(t.page);
    const bool alone = A <= kWarpSlots;
    const int per = alone ? (A + 31) / 32 : (A + kThreads - 1) / kThreads, i0 = tid * per, i1 = min(A, i0 + per);
    const int64_t head0 = t.counts[0], tail0 = t.counts[1];
    const int64_t free = max((int64_t)0, min(t.n_pages, tail0 - head0));
    uint32_t bad = 0;
    int32_t old[kPer], more[kPer], lens[kPer], first[kPer], need[kPer], give[kPer];   // this thread's slots
    bool granted[kPer];
    if (!alone || tid < 32) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (i0 + k >= i1) break;
            lens[k] = t.lens[i0 + k];
            first[k] = t.first[i0 + k];
            more[k] = max(0, fresh[i0 + k]);
        }
        int64_t sum_rows = 0, all_rows;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (i0 + k >= i1) break;
            old[k] = (int32_t)clamp_len(lens[k], t.max_pages, t.page, &bad);
            sum_rows += more[k];
        }
        int64_t row0 = scan(sum_rows, alone, sc.warps, &all_rows);
        // pages that each needs, 0 where its tokens or rows do not fit, and (in the upper half) pages that it gives back
        int64_t both = 0, all;
        bool fits[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (i0 + k >= i1) break;
            sum.rows[i0 + k] = (int32_t)min(row0, (int64_t)0x7FFFFFFF);   // beyond n_rows no row looks for its slot
            sum.old[i0 + k] = old[k];
            row0 += more[k];
            const int64_t had = pages_of(old[k], t.page), want = pages_of((int64_t)old[k] + more[k], t.page);
            fits[k] = want <= t.max_pages && row0 <= n_rows;
            if (!fits[k] && more[k] > 0) bad |= kPagesBadLength;
            need[k] = fits[k] ? (int32_t)(want - had) : 0;
            int64_t behind = 0;
            if (t.window > 0 && lens[k] >= 0) {
                const int64_t b = (int64_t)old[k] + 1 > t.window ? ((int64_t)old[k] + 1 - t.window) >> shift : 0;
                behind = b < had ? b : had;
            }
            const int64_t from = max(first[k], t.lead);
            give[k] = behind > from ? (int32_t)(behind - from) : 0;
            both += need[k] + ((int64_t)give[k] << 32);   // each below 2^31 in all
        }
        int64_t at = scan(both, alone, sc.warps, &all);
        if (tid == 0) {
            sum.rows[A] = (int32_t)min(all_rows, (int64_t)0x7FFFFFFF);
            sum.take[A] = (int32_t)all;
            sum.give[A] = (int32_t)(all >> 32);
            sc.most = 0;
        }
        if (alone) __syncwarp();
        else __syncthreads();
        int32_t most = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (i0 + k >= i1) break;
            sum.take[i0 + k] = (int32_t)at;
            sum.give[i0 + k] = (int32_t)(at >> 32);
            at += need[k] + ((int64_t)give[k] << 32);
            granted[k] = more[k] > 0 && fits[k] && (need[k] == 0 || (int32_t)at <= free);
            if (granted[k] && need[k] > 0) most = (int32_t)at;
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if ((tid & 31) == 0 && most > 0) atomicMax(&sc.most, most);
    }
    __syncthreads();
    const int32_t all_give = sum.give[A], all_rows = sum.rows[A];
    // more pages than the ring has places: the state is not one of these calls'
    const int64_t fit = all_give <= t.n_pages ? all_give : t.n_pages;
    if (fit < all_give) bad |= kPagesBadLength;
    const int32_t taken = sc.most;   // slots that need pages and get them are the first of those that need any
    const int64_t head = ring_place(head0, t.n_pages), tail = ring_place(tail0, t.n_pages);
    const bool summed = !alone || tid < 32;
    if (blockIdx.x == 0 && summed) {
        if (bad && t.status) atomicOr(t.status, bad);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (i0 + k >= i1) break;
            starts[i0 + k] = (int32_t)min((int64_t)sum.rows[i0 + k], n_rows);
            before[i0 + k] = granted[k] ? old[k] : -1;
            after[i0 + k] = granted[k] ? old[k] + more[k] : -1;
        }
        if (tid == 0) starts[A] = (int32_t)min((int64_t)all_rows, n_rows);
    }
    const int64_t at = (int64_t)blockIdx.x * kThreads + tid, stride = (int64_t)gridDim.x * kThreads;
    bad = 0;
    // pages into the table
    for (int64_t i = at; i < taken; i += stride) {
        const int s = slot_of(sum.take, A, (int32_t)i);
        const int64_t lp = pages_of(sum.old[s], t.page) + i - sum.take[s];
        t.table[(int64_t)s * t.max_pages + lp] = (int32_t)check_page(t.ring[ring_at(head, i, t.n_pages)], t.n_pages, &bad);
    }
    // pages behind the window into the ring
    for (int64_t i = at; i < fit; i += stride) {
        const int s = slot_of(sum.give, A, (int32_t)i);
        const int64_t lp = max(t.first[s], t.lead) + i - sum.give[s];
        int32_t* e = t.table + (int64_t)s * t.max_pages + lp;
        t.ring[ring_at(tail, i, t.n_pages)] = (int32_t)check_page(*e, t.n_pages, &bad);
        *e = -1;
    }
    // rows
    if (slots || positions)
        for (int64_t i = at; i < n_rows; i += stride) {
            int64_t place = -1, slot = -1;
            if (i < all_rows) {
                const int s = slot_of(sum.rows, A, (int32_t)i);
                const int64_t had = sum.old[s];
                const int64_t end = sum.rows[s + 1];
                const int32_t want = sum.take[s + 1] - sum.take[s];
                if (end <= n_rows && pages_of(had + end - sum.rows[s], t.page) <= t.max_pages && (want == 0 || sum.take[s + 1] <= free)) {
                    place = had + i - sum.rows[s];
                    const int64_t lp = place >> shift, held = pages_of(had, t.page);
                    const int32_t raw = lp < held ? t.table[(int64_t)s * t.max_pages + lp]
                                                  : t.ring[ring_at(head, sum.take[s] + lp - held, t.n_pages)];
                    const int64_t id = check_page(raw, t.n_pages, &bad);
                    slot = id < 0 ? -1 : id * t.page + (place & (t.page - 1));
                }
            }
            if (slots) slots[i] = slot;
            if (positions) positions[i] = place;
        }
    if (bad && t.status) atomicOr(t.status, bad);
    if (!arrived_last(t, sc) || !summed) return;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (i0 + k >= i1) break;
        if (granted[k]) t.lens[i0 + k] = old[k] + more[k];
        if (give[k] > 0) t.first[i0 + k] = max(first[k], t.lead) + give[k];
    }
    if (tid == 0) {
        t.counts[0] = head0 + taken;
        t.counts[1] = tail0 + fit;
    }
}

__global__ void __launch_bounds__(kThreads) tables_cut_kernel(const PageTablesArgs t, const int32_t* __restrict__ keep) {
    extern __shared__ int32_t sums[];   // [A + 1]
    __shared__ Scratch sc;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    const int tid = threadIdx.x, A = t.A;
    const bool alone = A <= kWarpSlots, summed = !alone || tid < 32;
    const int per = alone ? (A + 31) / 32 : (A + kThreads - 1) / kThreads, i0 = tid * per, i1 = min(A, i0 + per);
    const int64_t tail0 = t.counts[1];
    uint32_t bad = 0;
    int32_t stay[kPer], first[kPer], give[kPer];
    // a slot's pages [left, had) without those that a window has taken before, [lead, first)
    auto range = [&](int32_t len, int32_t stay_, int32_t first_, int64_t* left, int64_t* hole, int64_t* gone) {
        uint32_t ignore = 0;
        const int64_t had = pages_of(clamp_len(len, t.max_pages, t.page, &ignore), t.page);
        *left = pages_of(stay_ > 0 ? stay_ : 0, t.page);
        *hole = *left > t.lead ? *left : (int64_t)t.lead;
        const int64_t end = first_ < had ? first_ : had;
        *gone = end > *hole ? end - *hole : 0;
        return (int32_t)(had > *left ? had - *left - *gone : 0);
    };
    auto kept = [&](int32_t len, int32_t k) {
        uint32_t ignore = 0;
        const int32_t n = len < 0 ? -1 : (int32_t)clamp_len(len, t.max_pages, t.page, &ignore);
        return k < 0 ? -1 : (k < n ? k : n);
    };
    if (summed) {
        int64_t sum = 0, all;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (i0 + k >= i1) break;
            const int32_t len = t.lens[i0 + k];
            clamp_len(len, t.max_pages, t.page, &bad);
            first[k] = t.first[i0 + k];
            stay[k] = kept(len, keep[i0 + k]);
            int64_t left, hole, gone;
            give[k] = range(len, stay[k], first[k], &left, &hole, &gone);
            first[k] = stay[k] < 0 ? t.lead : min((int64_t)first[k], hole);
            sum += give[k];
        }
        int64_t at = scan(sum, alone, sc.warps, &all);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (i0 + k >= i1) break;
            sums[i0 + k] = (int32_t)at;
            at += give[k];
        }
        if (tid == 0) sums[A] = (int32_t)all;
    }
    __syncthreads();
    const int32_t all = sums[A];
    const int64_t tail = ring_place(tail0, t.n_pages);
    // more pages than the ring has places: the state is not one of these calls'
    const int64_t fit = all <= t.n_pages ? all : t.n_pages;
    if (fit < all) bad |= kPagesBadLength;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < fit; i += (int64_t)gridDim.x * kThreads) {
        const int s = slot_of(sums, A, (int32_t)i);
        const int32_t len = t.lens[s];
        int64_t left, hole, gone;
        range(len, kept(len, keep[s]), t.first[s], &left, &hole, &gone);
        int64_t lp = left + i - sums[s];
        if (lp >= hole) lp += gone;
        int32_t* e = t.table + (int64_t)s * t.max_pages + lp;
        t.ring[ring_at(tail, i, t.n_pages)] = (int32_t)check_page(*e, t.n_pages, &bad);
        *e = -1;
    }
    if (bad && t.status) atomicOr(t.status, bad);
    if (!arrived_last(t, sc) || !summed) return;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (i0 + k >= i1) break;
        t.lens[i0 + k] = stay[k];
        t.first[i0 + k] = first[k];
    }
    if (tid == 0) t.counts[1] = tail0 + fit;
}

}  // namespace

polykv_status launch_tables_plan(const PageTablesArgs& t, const int32_t* fresh, int64_t n_rows, int32_t* starts, int32_t* before,
                                 int32_t* after, int64_t* slots, int64_t* positions, cudaStream_t st) {
    // beyond 48 KB, the kernel's own Scratch among them, it needs leave, which stands for the process: always the same
    cudaError_t e = cudaSuccess;
    if (sums_bytes(t.A) > 40 * 1024) e = cudaFuncSetAttribute(tables_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sums_bytes(kPagesMaxSeqs));
    // a row a thread, on no more blocks than the card runs at once: each makes the sums over the slots first
    const int64_t most = device_sm_count(), want = (n_rows + kThreads - 1) / kThreads;
    const unsigned blocks = (unsigned)(want < 1 ? 1 : (want < most ? want : most));
    if (e == cudaSuccess)
        e = launch_after(tables_plan_kernel, dim3(blocks), kThreads, sums_bytes(t.A), st, t, fresh, n_rows, starts, before, after, slots, positions);
    return e == cudaSuccess ? POLYKV_OK : set_error(POLYKV_E_CUDA, "tables_plan launch: %s", cudaGetErrorString(e));
}

polykv_status launch_tables_cut(const PageTablesArgs& t, const int32_t* keep, cudaStream_t st) {
    // how many pages come back is on the device: a block for each 64 slots
    const cudaError_t e = launch_after(tables_cut_kernel, dim3((unsigned)((t.A + 63) / 64)), kThreads, (size_t)(t.A + 1) * sizeof(int32_t), st, t, keep);
    return e == cudaSuccess ? POLYKV_OK : set_error(POLYKV_E_CUDA, "tables_cut launch: %s", cudaGetErrorString(e));
}

}  // namespace polykv
