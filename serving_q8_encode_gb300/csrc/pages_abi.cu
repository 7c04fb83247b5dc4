// C ABI of the paged cache: argument validation, dispatch, and the status word.
#include <cmath>
#include <new>

#include "pages_abi.cuh"

struct polykv_pages {
    polykv::PagesView view;
    polykv_dtype dtype;
};

namespace polykv {

const PagesView& pages_view(const polykv_pages* pages) { return pages->view; }
polykv_dtype pages_dtype(const polykv_pages* pages) { return pages->dtype; }

SeqsArgs pages_seqs(const polykv_pages_seqs* s) {
    SeqsArgs a;
    a.table = s->block_table;
    a.lens = s->lens;
    a.max_pages = s->max_pages;
    a.A = s->n_seqs;
    a.layer0 = s->layer0;
    a.nl = s->n_layers;
    return a;
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

polykv_status check_seqs(const polykv_pages* pages, const polykv_pages_seqs* s, int32_t n_q_heads) {
    if (!pages) return set_error(POLYKV_E_INVAL, "pages is NULL");
    if (!s) return set_error(POLYKV_E_INVAL, "seqs is NULL");
    const PagesView& v = pages->view;
    if (!s->block_table || !s->lens) return set_error(POLYKV_E_INVAL, "block_table and lens must be non-NULL");
    if ((reinterpret_cast<uintptr_t>(s->block_table) & 3u) || (reinterpret_cast<uintptr_t>(s->lens) & 3u))
        return set_error(POLYKV_E_INVAL, "block_table and lens must be 4-byte aligned");
    if (s->n_seqs < 1 || s->max_pages < 1) return set_error(POLYKV_E_INVAL, "n_seqs and max_pages must be >= 1");
    if (s->n_seqs > kPagesMaxSeqs)
        return set_error(POLYKV_E_UNSUPPORTED, "%d sequences in one call (at most %d)", s->n_seqs, kPagesMaxSeqs);
    if (s->n_layers < 1 || s->layer0 < 0 || s->layer0 > v.L - s->n_layers)
        return set_error(POLYKV_E_INVAL, "layers [%d, %d + %d) of %d", s->layer0, s->layer0, s->n_layers, v.L);
    if (s->max_pages > (int64_t)0x7FFFFFFF / v.page || s->max_pages > 65535 * (int64_t)64 ||
        (int64_t)s->n_seqs * s->max_pages * (v.page / kPageStep) > 0x7FFFFFFF)
        return set_error(POLYKV_E_UNSUPPORTED, "block table of %d x %lld pages is too large", s->n_seqs,
                         (long long)s->max_pages);
    if (n_q_heads < 1 || n_q_heads % v.H != 0)
        return set_error(POLYKV_E_INVAL, "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)", n_q_heads, v.H);
    if (n_q_heads > 4096 || (int64_t)n_q_heads * s->n_layers > (1 << 22))
        return set_error(POLYKV_E_UNSUPPORTED, "%d query heads x %d layers (at most 4096, and 2^22 in one call)", n_q_heads,
                         s->n_layers);
    return POLYKV_OK;
}

polykv_status check_rows(const char* name, const void* p, const polykv_row_strides& s) {
    if (!p) return set_error(POLYKV_E_INVAL, "%s is NULL", name);
    if (!aligned16(p) || s.layer % 8 != 0 || s.row % 8 != 0 || s.head % 8 != 0)
        return set_error(POLYKV_E_INVAL, "%s must be 16-byte aligned, its strides multiples of 8 elements", name);
    return POLYKV_OK;
}

RowStrides strides_of(const polykv_row_strides& s) { return RowStrides{s.layer, s.row, s.head}; }

// Clears the bits that were read, and no others: a kernel on another stream may have set one since.
__global__ void clear_bits_kernel(uint32_t* status, uint32_t read) { atomicAnd(status, ~read); }

}  // namespace

polykv_status check_pages_attend(const polykv_pages* pages, const polykv_pages_seqs* seqs, int32_t n_q_heads,
                                 const int32_t* selected, int64_t n_selected) {
    const polykv_status st = check_seqs(pages, seqs, n_q_heads);
    if (st != POLYKV_OK) return st;
    if (selected ? n_selected < 1 || n_selected > (1 << 20) : n_selected >= 0)
        return set_error(POLYKV_E_INVAL, "n_selected = %lld (1 .. 2^20, or negative with a NULL selected: all pages)",
                         (long long)n_selected);
    if (reinterpret_cast<uintptr_t>(selected) & 3u)
        return set_error(POLYKV_E_INVAL, "selected must be 4-byte aligned");
    return POLYKV_OK;
}

}  // namespace polykv

using namespace polykv;

extern "C" {

polykv_status polykv_pages_create(const polykv_pages_desc* d, polykv_pages** out) {
    if (!d || !out) return set_error(POLYKV_E_INVAL, "desc and out must be non-NULL");
    if (d->n_layers <= 0 || d->n_kv_heads <= 0 || d->n_pages <= 0)
        return set_error(POLYKV_E_INVAL, "n_layers, n_kv_heads and n_pages must be positive");
    if (d->n_layers > 65535 || d->n_kv_heads > 4096 || d->n_pages > 0x7FFFFFFF)
        return set_error(POLYKV_E_UNSUPPORTED, "at most 65535 layers, 4096 kv heads and 2^31 - 1 pages");
    if (d->in_dtype != POLYKV_F16 && d->in_dtype != POLYKV_BF16)
        return set_error(POLYKV_E_INVAL, "in_dtype must be POLYKV_F16 or POLYKV_BF16");
    if (d->head_dim != 64 && d->head_dim != 128)
        return set_error(POLYKV_E_UNSUPPORTED, "head_dim %d (supported: 64, 128)", d->head_dim);
    if (d->page_tokens != 16 && d->page_tokens != 32 && d->page_tokens != 64 && d->page_tokens != 128)
        return set_error(POLYKV_E_UNSUPPORTED, "page_tokens %d (supported: 16, 32, 64, 128)", d->page_tokens);
    if (!d->k_pages || !d->v_pages) return set_error(POLYKV_E_INVAL, "k_pages and v_pages must be non-NULL");
    if (!aligned16(d->k_pages) || !aligned16(d->v_pages) || !aligned16(d->key_bounds))
        return set_error(POLYKV_E_INVAL, "k_pages, v_pages and key_bounds must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(d->status) & 3u) return set_error(POLYKV_E_INVAL, "status must be 4-byte aligned");
    polykv_pages* p = new (std::nothrow) polykv_pages;
    if (!p) return set_error(POLYKV_E_INVAL, "host allocation failed");
    p->view.k = static_cast<uint16_t*>(d->k_pages);
    p->view.v = static_cast<uint16_t*>(d->v_pages);
    p->view.bounds = static_cast<uint16_t*>(d->key_bounds);
    p->view.status = d->status;
    p->view.L = d->n_layers;
    p->view.H = d->n_kv_heads;
    p->view.d = d->head_dim;
    p->view.page = d->page_tokens;
    p->view.n_pages = d->n_pages;
    p->dtype = d->in_dtype;
    p->view.tma = pages_tma_new();
    if (!p->view.tma) {
        delete p;
        return set_error(POLYKV_E_INVAL, "host allocation failed");
    }
    *out = p;
    return POLYKV_OK;
}

polykv_status polykv_pages_append(polykv_pages* pages, const polykv_pages_seqs* seqs, const polykv_pages_append_args* x,
                                  void* stream) {
    if (!x) return set_error(POLYKV_E_INVAL, "args is NULL");
    polykv_status st = check_seqs(pages, seqs, x->q ? x->n_q_heads : (pages ? pages->view.H : 1));
    if (st != POLYKV_OK) return st;
    if (x->n_rows < 0 || x->n_rows > 0x7FFFFFFF) return set_error(POLYKV_E_INVAL, "n_rows = %lld", (long long)x->n_rows);
    if (!x->starts && x->n_rows != seqs->n_seqs)
        return set_error(POLYKV_E_INVAL, "without starts every sequence appends one row: %lld rows, %d sequences",
                         (long long)x->n_rows, seqs->n_seqs);
    if (reinterpret_cast<uintptr_t>(x->starts) & 3u) return set_error(POLYKV_E_INVAL, "starts must be 4-byte aligned");
    if (reinterpret_cast<uintptr_t>(x->positions) & 7u)
        return set_error(POLYKV_E_INVAL, "positions must be 8-byte aligned");
    if (reinterpret_cast<uintptr_t>(x->turns) & 7u) return set_error(POLYKV_E_INVAL, "turns must be 8-byte aligned");
    if (x->n_rows == 0) return POLYKV_OK;
    if ((st = check_rows("k", x->k, x->k_strides)) != POLYKV_OK) return st;
    if ((st = check_rows("v", x->v, x->v_strides)) != POLYKV_OK) return st;
    if (x->turns) {
        if (x->rotary_dim < 16 || x->rotary_dim % 16 != 0 || x->rotary_dim > pages->view.d)
            return set_error(POLYKV_E_UNSUPPORTED, "rotary_dim %d (a multiple of 16, at most head_dim)", x->rotary_dim);
    }
    if (x->q) {
        if (!x->turns) return set_error(POLYKV_E_INVAL, "q is given but there is no rotation");
        if ((st = check_rows("q", x->q, x->q_strides)) != POLYKV_OK) return st;
        if ((st = check_rows("q_out", x->q_out, x->q_out_strides)) != POLYKV_OK) return st;
    }
    PagesAppendArgs a = {};
    a.p = pages->view;
    a.s = pages_seqs(seqs);
    a.k = static_cast<const uint16_t*>(x->k);
    a.v = static_cast<const uint16_t*>(x->v);
    a.q = static_cast<const uint16_t*>(x->q);
    a.q_out = static_cast<uint16_t*>(x->q_out);
    a.ks = strides_of(x->k_strides);
    a.vs = strides_of(x->v_strides);
    a.qs = strides_of(x->q_strides);
    a.qos = strides_of(x->q_out_strides);
    a.Hq = x->n_q_heads;
    a.rows = x->n_rows;
    a.starts = x->starts;
    a.positions = x->positions;
    a.pos_offset = x->pos_offset;
    a.turns = x->turns;
    a.rot = x->rotary_dim;
    a.interleaved = x->interleaved != 0;
    a.mscale = x->mscale;
    return launch_pages_append(a, pages->dtype, static_cast<cudaStream_t>(stream));
}

polykv_status polykv_pages_attend_workspace_size(const polykv_pages* pages, int32_t n_q_heads, size_t* bytes) {
    if (!pages || !bytes) return set_error(POLYKV_E_INVAL, "pages and bytes must be non-NULL");
    if (n_q_heads < 1 || n_q_heads % pages->view.H != 0)
        return set_error(POLYKV_E_INVAL, "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)", n_q_heads,
                         pages->view.H);
    *bytes = pages_attend_workspace(pages->view, n_q_heads / pages->view.H);
    return POLYKV_OK;
}

polykv_status polykv_pages_attend(const polykv_pages* pages, const polykv_pages_seqs* seqs, const void* q,
                                  const polykv_row_strides* q_strides, int32_t n_q_heads, const int32_t* selected,
                                  int64_t n_selected, float softmax_scale, void* out, int32_t out_f32, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    polykv_status st = check_pages_attend(pages, seqs, n_q_heads, selected, n_selected);
    if (st != POLYKV_OK) return st;
    if (!q_strides) return set_error(POLYKV_E_INVAL, "q_strides is NULL");
    if ((st = check_rows("q", q, *q_strides)) != POLYKV_OK) return st;
    if (!out || !aligned16(out)) return set_error(POLYKV_E_INVAL, "out must be non-NULL and 16-byte aligned");
    const PagesView& v = pages->view;
    const size_t need = pages_attend_workspace(v, n_q_heads / v.H);
    if (!workspace || !aligned16(workspace))
        return set_error(POLYKV_E_INVAL, "workspace must be non-NULL and 16-byte aligned");
    if (workspace_bytes < need)
        return set_error(POLYKV_E_BUFFER_TOO_SMALL, "pages_attend: workspace %zu < %zu bytes", workspace_bytes, need);
    PagesAttendArgs a = {};
    a.p = v;
    a.s = pages_seqs(seqs);
    a.q = static_cast<const uint16_t*>(q);
    a.qs = strides_of(*q_strides);
    a.Hq = n_q_heads;
    a.G = n_q_heads / v.H;
    a.sel = selected;
    a.n_sel = selected ? (int)n_selected : -1;
    a.scale_log2 = (softmax_scale > 0.0f ? softmax_scale : 1.0f / sqrtf((float)v.d)) * 1.4426950408889634f;
    a.out = out;
    a.out_f32 = out_f32 != 0;
    return launch_pages_attend(a, pages->dtype, workspace, static_cast<cudaStream_t>(stream));
}

polykv_status polykv_pages_select_workspace_size(const polykv_pages* pages, const polykv_pages_seqs* seqs, size_t* bytes) {
    if (!bytes) return set_error(POLYKV_E_INVAL, "bytes is NULL");
    const polykv_status st = check_seqs(pages, seqs, pages ? pages->view.H : 1);
    if (st != POLYKV_OK) return st;
    *bytes = pages_select_workspace(pages->view, seqs->n_seqs, seqs->n_layers, seqs->max_pages);
    return POLYKV_OK;
}

polykv_status polykv_pages_select(const polykv_pages* pages, const polykv_pages_seqs* seqs, const void* q,
                                  const polykv_row_strides* q_strides, int32_t n_q_heads, int64_t n_selected,
                                  int64_t keep_first, int64_t keep_last, int32_t* selected, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    polykv_status st = check_seqs(pages, seqs, n_q_heads);
    if (st != POLYKV_OK) return st;
    if (n_selected < 1 || n_selected > (1 << 20))
        return set_error(POLYKV_E_INVAL, "n_selected = %lld (1 .. 2^20)", (long long)n_selected);
    if (keep_first < 0 || keep_last < 0 || keep_first > n_selected || keep_last > n_selected - keep_first)   // a sum could wrap
        return set_error(POLYKV_E_INVAL, "keep_first (%lld) and keep_last (%lld) must be >= 0 and fit into n_selected (%lld)",
                         (long long)keep_first, (long long)keep_last, (long long)n_selected);
    if (!pages->view.bounds) return set_error(POLYKV_E_STATE, "select: the cache was created without key_bounds");
    if (!q_strides) return set_error(POLYKV_E_INVAL, "q_strides is NULL");
    if ((st = check_rows("q", q, *q_strides)) != POLYKV_OK) return st;
    if (!selected || (reinterpret_cast<uintptr_t>(selected) & 3u))
        return set_error(POLYKV_E_INVAL, "selected must be non-NULL and 4-byte aligned");
    const size_t need = pages_select_workspace(pages->view, seqs->n_seqs, seqs->n_layers, seqs->max_pages);
    if (need > 0 && (!workspace || !aligned16(workspace)))
        return set_error(POLYKV_E_INVAL, "workspace must be non-NULL and 16-byte aligned");
    if (workspace_bytes < need)
        return set_error(POLYKV_E_BUFFER_TOO_SMALL, "pages_select: workspace %zu < %zu bytes", workspace_bytes, need);
    PagesSelectArgs a = {};
    a.p = pages->view;
    a.s = pages_seqs(seqs);
    a.q = static_cast<const uint16_t*>(q);
    a.qs = strides_of(*q_strides);
    a.Hq = n_q_heads;
    a.G = n_q_heads / pages->view.H;
    a.out = selected;
    a.n_sel = (int)n_selected;
    a.keep_first = (int)keep_first;
    a.keep_last = (int)keep_last;
    return launch_pages_select(a, pages->dtype, workspace, static_cast<cudaStream_t>(stream));
}

polykv_status polykv_pages_status(const polykv_pages* pages, void* stream, uint32_t* flags) {
    if (!pages || !flags) return set_error(POLYKV_E_INVAL, "pages and flags must be non-NULL");
    *flags = 0;
    if (!pages->view.status) return set_error(POLYKV_E_STATE, "the cache was created without a status word");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t h = 0;
    cudaError_t e = cudaMemcpyAsync(&h, pages->view.status, sizeof(h), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess && h) {
        clear_bits_kernel<<<1, 1, 0, st>>>(pages->view.status, h);
        e = cudaGetLastError();
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    }
    if (e != cudaSuccess) return set_error(POLYKV_E_CUDA, "pages status read: %s", cudaGetErrorString(e));
    *flags = h;
    if (h & kPagesTimeout) return set_error(POLYKV_E_TIMEOUT, "pages: a kernel gave up waiting on a bounded device-side wait");
    if (h)
        return set_error(POLYKV_E_STATE, "pages:%s%s%s", (h & kPagesBadPage) ? " a page id outside the cache;" : "",
                         (h & kPagesBadLength) ? " a length beyond the block table, or starts out of order;" : "",
                         (h & kPagesBadChoice) ? " a chosen page beyond its sequence;" : "");
    return POLYKV_OK;
}

polykv_status polykv_pages_free(polykv_pages* pages) {
    if (pages) pages_tma_free(pages->view.tma);
    delete pages;
    return POLYKV_OK;
}

}  // extern "C"
