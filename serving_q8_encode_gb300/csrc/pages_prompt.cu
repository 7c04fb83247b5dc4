// Attention of runs of rows (prompts, chunks, drafted tokens) over a paged cache, causal, with a sliding window and sinks.
//
//   row i of a sequence stands at place p = len - count + i and sees tokens t <= p with t > p - window or t < sinks
//   out[row][hq] = sum_t softmax_t(scale q . k_t) v_t over what it sees; zeros if that is nothing
#include "pages_prompt.cuh"

namespace polykv {
namespace {

constexpr int kThreads = 256;

template <int D, int CODE, bool BF16>
__global__ void __launch_bounds__(kThreads) rows_exact_kernel(const PagesRowsArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what the kernels before wrote, from here on
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32), jobs = (int64_t)a.s.nl * a.rows * a.Hq;
    for (int64_t job = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); job < jobs; job += warps) {
        const int h = (int)(job % a.Hq);
        const int64_t r = job / a.Hq % a.rows;
        const int l = (int)(job / a.Hq / a.rows);
        uint32_t bad = 0;
        const RowOf at = row_of(a, r, lane, &bad);
        if (at.place >= 0) attend_row<D, CODE, BF16>(a, l, at, r, h, lane, &bad);
        if (bad && a.p.status && lane == 0) atomicOr(a.p.status, bad);
    }
}

template <int D, int CODE>
polykv_status run(const PagesRowsArgs& a, bool bf, cudaStream_t st) {
    const int64_t jobs = (int64_t)a.s.nl * a.rows * a.Hq, want = (jobs + kThreads / 32 - 1) / (kThreads / 32);
    const unsigned grid = (unsigned)(want < 0x7FFFFFFF ? want : 0x7FFFFFFF);
    const cudaError_t e = bf ? launch_after(rows_exact_kernel<D, CODE, true>, dim3(grid), kThreads, 0, st, a)
                             : launch_after(rows_exact_kernel<D, CODE, false>, dim3(grid), kThreads, 0, st, a);
    return e == cudaSuccess ? POLYKV_OK : set_error(POLYKV_E_CUDA, "pages_attend_rows launch: %s", cudaGetErrorString(e));
}

}  // namespace

size_t pages_rows_workspace(const PagesRowsArgs&) { return 0; }

polykv_status launch_pages_rows(const PagesRowsArgs& a, polykv_dtype dt, void*, cudaStream_t st) {
    const bool bf = dt == POLYKV_BF16;
    if (a.p.code == kPagesWide) return a.p.d == 128 ? run<128, kPagesWide>(a, bf, st) : run<64, kPagesWide>(a, bf, st);
    if (a.p.code == kPagesInt8) return a.p.d == 128 ? run<128, kPagesInt8>(a, bf, st) : run<64, kPagesInt8>(a, bf, st);
    return a.p.d == 128 ? run<128, kPagesE4m3>(a, bf, st) : run<64, kPagesE4m3>(a, bf, st);
}

}  // namespace polykv
