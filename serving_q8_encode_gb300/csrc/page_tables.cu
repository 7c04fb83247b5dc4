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
// (at most 4,096, from three arrays that L2 holds) instead of waiting for one that does; the work that is long, rows and
// pages, is shared out flat. The last CTA to have read the state writes the new one (an arrival count; nobody waits).
#include "pages_internal.cuh"

namespace polykv {
namespace {

constexpr int kThreads = 512;
constexpr int kPer = kPagesMaxSeqs / kThreads;   // slots per thread at most

struct Sums {   // in shared memory, all over the slots, exclusive with the total behind the last
    int64_t rows[kPagesMaxSeqs + 1];
    int32_t take[kPagesMaxSeqs + 1], give[kPagesMaxSeqs + 1];
};
struct Scratch {
    int64_t wide[kThreads / 32];
    int32_t narrow[kThreads / 32];
    int32_t most;
    int last;
};

// Exclusive sum over the block's threads; the scratch may be used again after the next barrier of the caller.
template <class T>
__device__ __forceinline__ T block_scan(T x, T* warps, T* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warps[warp] = inc;
    __syncthreads();
    T base = 0, all = 0;
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
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t before;
        asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(before) : "l"(t.arrivals), "r"(gridDim.x - 1) : "memory");
        sc.last = before == gridDim.x - 1;
    }
    __syncthreads();
    return sc.last != 0;
}

__device__ __forceinline__ int64_t ring_at(int64_t from, int64_t i, int64_t n) {   // from in [0, n), i in [0, n]
    const int64_t x = from + i;
    return x >= n ? x - n : x;
}

__global__ void __launch_bounds__(kThreads) tables_plan_kernel(const PageTablesArgs t, const int32_t* __restrict__ fresh, const int64_t n_rows,
                                                               int32_t* __restrict__ starts, int32_t* __restrict__ before,
                                                               int32_t* __restrict__ after, int64_t* __restrict__ slots,
                                                               int64_t* __restrict__ positions) {
    extern __shared__ __align__(16) unsigned char smem[];
    Sums& sum = *reinterpret_cast<Sums*>(smem);
    __shared__ Scratch sc;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    const int tid = threadIdx.x, A = t.A, shift = page_shift(t.page);
    const int per = (A + kThreads - 1) / kThreads, i0 = tid * per, i1 = min(A, i0 + per);
    const int64_t head0 = t.counts[0], tail0 = t.counts[1];
    const int64_t free = max((int64_t)0, min(t.n_pages, tail0 - head0));
    uint32_t bad = 0;
    int64_t old[kPer], more[kPer];   // this thread's slots: tokens, and how many it asks for
    int32_t lens[kPer], first[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (i0 + k >= i1) break;
        lens[k] = t.lens[i0 + k];
        first[k] = t.first[i0 + k];
        old[k] = clamp_len(lens[k], t.max_pages, t.page, &bad);
        more[k] = max(0, fresh[i0 + k]);
    }
    // rows
    int64_t sum_rows = 0, all_rows;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (i0 + k < i1) sum_rows += more[k];
    int64_t row0 = block_scan(sum_rows, sc.wide, &all_rows);
    // pages that each needs, 0 where its tokens or rows do not fit; pages that it gives back
    int32_t need[kPer], give[kPer], sum_need = 0, sum_give = 0, all_need, all_give;
    bool fits[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (i0 + k >= i1) break;
        sum.rows[i0 + k] = row0;
        row0 += more[k];
        const int64_t had = pages_of(old[k], t.page), want = pages_of(old[k] + more[k], t.page);
        fits[k] = want <= t.max_pages && row0 <= n_rows;
        if (!fits[k] && more[k] > 0) bad |= kPagesBadLength;
        need[k] = fits[k] ? (int32_t)(want - had) : 0;
        sum_need += need[k];
        int64_t behind = 0;
        if (t.window > 0 && lens[k] >= 0) {
            const int64_t b = old[k] + 1 > t.window ? (old[k] + 1 - t.window) >> shift : 0;
            behind = b < had ? b : had;
        }
        const int64_t from = first[k] > t.lead ? first[k] : t.lead;
        give[k] = behind > from ? (int32_t)(behind - from) : 0;
        sum_give += give[k];
    }
    int32_t take0 = block_scan(sum_need, sc.narrow, &all_need);
    int32_t give0 = block_scan(sum_give, sc.narrow, &all_give);
    if (tid == 0) {
        sum.rows[A] = all_rows;
        sum.take[A] = all_need;
        sum.give[A] = all_give;
        sc.most = 0;
    }
    __syncthreads();
    bool granted[kPer];
    int32_t most = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (i0 + k >= i1) break;
        sum.take[i0 + k] = take0;
        sum.give[i0 + k] = give0;
        take0 += need[k];
        give0 += give[k];
        granted[k] = more[k] > 0 && fits[k] && (need[k] == 0 || take0 <= free);
        if (granted[k] && need[k] > 0) most = max(most, take0);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if ((tid & 31) == 0 && most > 0) atomicMax(&sc.most, most);
    __syncthreads();
    // more pages than the ring has places: the state is not one of these calls'
    const int64_t fit = all_give <= t.n_pages ? all_give : t.n_pages;
    if (fit < all_give) bad |= kPagesBadLength;
    const int32_t taken = sc.most;   // slots that need pages and get them are the first of those that need any
    const int64_t head = ((head0 % t.n_pages) + t.n_pages) % t.n_pages, tail = ((tail0 % t.n_pages) + t.n_pages) % t.n_pages;
    if (blockIdx.x == 0) {
        if (bad && t.status) atomicOr(t.status, bad);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (i0 + k >= i1) break;
            const int64_t r = sum.rows[i0 + k];
            starts[i0 + k] = (int32_t)(r < n_rows ? r : n_rows);
            before[i0 + k] = granted[k] ? (int32_t)old[k] : -1;
            after[i0 + k] = granted[k] ? (int32_t)(old[k] + more[k]) : -1;
        }
        if (tid == 0) starts[A] = (int32_t)(all_rows < n_rows ? all_rows : n_rows);
    }
    // Rows and pages need what this block has read for its own slots only; of the others the sums, and their lengths, which
    // stand in L2 until the last block has read them: that one writes them.
    const int64_t at = (int64_t)blockIdx.x * kThreads + tid, stride = (int64_t)gridDim.x * kThreads;
    bad = 0;
    // pages into the table
    for (int64_t i = at; i < taken; i += stride) {
        const int s = slot_of(sum.take, A, (int32_t)i);
        const int64_t lp = pages_of(clamp_len(t.lens[s], t.max_pages, t.page, &bad), t.page) + i - sum.take[s];
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
                const int s = slot_of(sum.rows, A, i);
                const int64_t had = clamp_len(t.lens[s], t.max_pages, t.page, &bad);
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
    if (!arrived_last(t, sc)) return;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (i0 + k >= i1) break;
        if (granted[k]) t.lens[i0 + k] = (int32_t)(old[k] + more[k]);
        if (give[k] > 0) t.first[i0 + k] = max(first[k], t.lead) + give[k];
    }
    if (tid == 0) {
        t.counts[0] = head0 + taken;
        t.counts[1] = tail0 + fit;
    }
}

__global__ void __launch_bounds__(kThreads) tables_cut_kernel(const PageTablesArgs t, const int32_t* __restrict__ keep) {
    extern __shared__ __align__(16) unsigned char smem[];
    int32_t* sums = reinterpret_cast<int32_t*>(smem);   // [A + 1]
    __shared__ Scratch sc;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    const int tid = threadIdx.x, A = t.A;
    const int per = (A + kThreads - 1) / kThreads, i0 = tid * per, i1 = min(A, i0 + per);
    const int64_t tail0 = t.counts[1];
    uint32_t bad = 0;
    int32_t stay[kPer], first[kPer], give[kPer], sum = 0, all;
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
    int32_t at0 = block_scan(sum, sc.narrow, &all);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (i0 + k >= i1) break;
        sums[i0 + k] = at0;
        at0 += give[k];
    }
    if (tid == 0) sums[A] = all;
    __syncthreads();
    const int64_t tail = ((tail0 % t.n_pages) + t.n_pages) % t.n_pages;
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
    if (!arrived_last(t, sc)) return;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (i0 + k >= i1) break;
        t.lens[i0 + k] = stay[k];
        t.first[i0 + k] = first[k];
    }
    if (tid == 0) t.counts[1] = tail0 + fit;
}

}  // namespace

// Blocks for `work` items at four a thread, no more than the card runs at once.
static unsigned blocks_for(int64_t work) {
    const int64_t most = device_sm_count(), want = (work + 4 * kThreads - 1) / (4 * kThreads);
    return (unsigned)(want < 1 ? 1 : (want < most ? want : most));
}

polykv_status launch_tables_plan(const PageTablesArgs& t, const int32_t* fresh, int64_t n_rows, int32_t* starts, int32_t* before,
                                 int32_t* after, int64_t* slots, int64_t* positions, cudaStream_t st) {
    // the limit stands for the process: always the same
    cudaError_t e = cudaFuncSetAttribute(tables_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Sums));
    if (e == cudaSuccess)
        e = launch_after(tables_plan_kernel, dim3(blocks_for(n_rows + t.A)), kThreads, sizeof(Sums), st, t, fresh, n_rows, starts, before, after, slots, positions);
    return e == cudaSuccess ? POLYKV_OK : set_error(POLYKV_E_CUDA, "tables_plan launch: %s", cudaGetErrorString(e));
}

polykv_status launch_tables_cut(const PageTablesArgs& t, const int32_t* keep, cudaStream_t st) {
    // how many pages come back is on the device: a block for each 64 slots
    const cudaError_t e = launch_after(tables_cut_kernel, dim3((unsigned)((t.A + 63) / 64)), kThreads, (size_t)(t.A + 1) * sizeof(int32_t), st, t, keep);
    return e == cudaSuccess ? POLYKV_OK : set_error(POLYKV_E_CUDA, "tables_cut launch: %s", cudaGetErrorString(e));
}

}  // namespace polykv
