// Definitions shared by the paged cache's translation units.
#pragma once

#include "pages_index.cuh"
#include "polykv_internal.cuh"

namespace polykv {

struct PagesTma;   // attention's tensor maps of a cache (host)
PagesTma* pages_tma_new();
void pages_tma_free(PagesTma* t);

// Device view of a paged cache in caller memory.
struct PagesView {
    uint16_t* k;        // [L][n_pages][H][page][d]
    uint16_t* v;        // [L][n_pages][H][page][d]
    uint16_t* bounds;   // [L][n_pages][H][2][d]: lowest and highest key per coordinate, or NULL
    uint32_t* status;   // status word, or NULL
    int L, H, d, page;
    int64_t n_pages;
    PagesTma* tma;      // host only
};

// What every kernel needs to find a sequence's tokens.
struct SeqsArgs {
    const int32_t* table;   // [A][max_pages]
    const int32_t* lens;    // [A]
    int64_t max_pages;
    int A;
    int layer0, nl;
};

struct RowStrides {
    int64_t layer, row, head;   // in elements; the head dimension is contiguous
};

struct PagesAttendArgs {
    PagesView p;
    SeqsArgs s;
    const uint16_t* q;
    RowStrides qs;
    int G, Hq;
    const int32_t* sel;   // [nl][A][H][n_sel], or NULL
    int n_sel;            // -1: all pages
    float scale_log2;
    void* out;            // fp32 or input type [nl][A][Hq][d]; partials: fp32, unnormalised
    float* ml;            // partials: running maximum (log2 units) and sum per row; else NULL
    int out_f32;
};
size_t pages_attend_workspace(const PagesView& p, int G);
polykv_status launch_pages_attend(const PagesAttendArgs& a, polykv_dtype dt, void* ws, cudaStream_t st);

struct PagesAppendArgs {
    PagesView p;
    SeqsArgs s;
    const uint16_t *k, *v, *q;
    uint16_t* q_out;
    RowStrides ks, vs, qs, qos;
    int Hq;
    int64_t rows;
    const int32_t* starts;      // [A + 1], or NULL: row a belongs to sequence a
    const int64_t* positions;   // [rows], or NULL: the token's place in its sequence + pos_offset
    int64_t pos_offset;
    const uint64_t* turns;      // [rot / 2] turns per position in units of 2^-64, or NULL: no rotation
    int rot;                    // rotated leading dimensions
    int interleaved;
    float mscale;               // factor of the cosines and sines
};
polykv_status launch_pages_append(const PagesAppendArgs& a, polykv_dtype dt, cudaStream_t st);

struct PagesSelectArgs {
    PagesView p;
    SeqsArgs s;
    const uint16_t* q;
    RowStrides qs;
    int G, Hq;
    int32_t* out;   // [nl][A][H][n_sel]
    int n_sel, keep_first, keep_last;
};
size_t pages_select_workspace(const PagesView& p, int A, int nl, int64_t max_pages);
polykv_status launch_pages_select(const PagesSelectArgs& a, polykv_dtype dt, void* ws, cudaStream_t st);

// Launches a kernel that begins with griddepcontrol.wait as a programmatic dependent of what precedes it on the
// stream: its CTAs are placed while that finishes, which hides 1.5 to 4 us of a call.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace polykv
