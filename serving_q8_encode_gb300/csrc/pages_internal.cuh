// Definitions shared by the paged cache's translation units.
#pragma once

#include "pages_index.cuh"
#include "polykv_internal.cuh"

namespace polykv {

struct PagesTma;   // attention's tensor maps of a cache (host)
PagesTma* pages_tma_new();
void pages_tma_free(PagesTma* t);

// How a paged cache holds keys and values.
constexpr int kPagesWide = 0;   // 16 bits, the input type
constexpr int kPagesInt8 = 1;   // int8 codes, a scale per (page, kv head) for the keys and one for the values
constexpr int kPagesE4m3 = 2;   // e4m3 codes, likewise

// Device view of a paged cache in caller memory.
struct PagesView {
    uint16_t* k;        // [L][n_pages][H][page][d]; 8-bit codes where code says so
    uint16_t* v;        // [L][n_pages][H][page][d]
    uint16_t* bounds;   // [L][n_pages][H][2][d]: lowest and highest key per coordinate, or NULL
    uint32_t* status;   // status word, or NULL
    int L, H, d, page;
    int64_t n_pages;
    PagesTma* tma;      // host only
    int code;           // kPagesWide, ...
    float* scales;      // 8-bit codes: [L][n_pages][H][2], the keys' and the values'
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
    int window, sinks;    // window > 0 (all pages only): the last `window` tokens and the first `sinks`
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
polykv_status launch_pages_append8(const PagesAppendArgs& a, polykv_dtype dt, cudaStream_t st);

struct PagesGatherArgs {
    PagesView p;
    SeqsArgs s;
    const int32_t* starts;   // [A + 1]: sequence s's last starts[s + 1] - starts[s] tokens become rows from starts[s] on
    int64_t rows;
    uint16_t *k, *v;         // [nl][rows][H][d]
};
polykv_status launch_pages_gather(const PagesGatherArgs& a, polykv_dtype dt, cudaStream_t st);

struct PagesRowsArgs {
    PagesView p;
    SeqsArgs s;
    const uint16_t* q;       // [nl][rows][Hq][d] with strides
    RowStrides qs;
    int G, Hq;
    const int32_t* starts;   // [A + 1]: the rows of sequence s, the last of them its token lens[s] - 1
    int64_t rows;
    int window, sinks;       // window 0: everything before
    float scale_log2;
    uint16_t* out;           // [nl][rows][Hq][d], the input type
};
size_t pages_rows_workspace(const PagesRowsArgs& a);
// Pages of codes that the rows see, as 16-bit pages [nl][places][H][page][d]: by page id, or where there is a table to write,
// by place in the tables.
polykv_status launch_pages_expand(const PagesRowsArgs& a, polykv_dtype dt, uint16_t* k, uint16_t* v, int64_t places, int32_t* table,
                                  cudaStream_t st);
polykv_status launch_pages_rows(const PagesRowsArgs& a, polykv_dtype dt, void* ws, cudaStream_t st);

// Block tables and free pages of the slots that a caller serves.
struct PageTablesArgs {
    int32_t* table;     // [A][max_pages]
    int32_t* lens;      // [A], negative: idle
    int32_t* first;     // [A]: the first page behind the sinks that is still held
    int32_t* ring;      // [n_pages]
    int64_t* counts;    // pages taken from the ring so far, and given to it
    uint32_t* arrivals; // zero between calls
    uint32_t* status;
    int64_t max_pages, n_pages;
    int A, page, window, lead;   // lead: pages that hold the sinks
};
polykv_status launch_tables_plan(const PageTablesArgs& t, const int32_t* fresh, int64_t n_rows, int32_t* starts, int32_t* before,
                                 int32_t* after, int64_t* slots, int64_t* positions, cudaStream_t st);
polykv_status launch_tables_cut(const PageTablesArgs& t, const int32_t* keep, cudaStream_t st);

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
