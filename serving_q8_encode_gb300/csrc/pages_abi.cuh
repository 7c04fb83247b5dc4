// The paged cache's handle, for the calls that take it together with a pool.
#pragma once

#include "pages_internal.cuh"

struct polykv_pages;

namespace polykv {

const PagesView& pages_view(const polykv_pages* pages);
polykv_dtype pages_dtype(const polykv_pages* pages);
SeqsArgs pages_seqs(const polykv_pages_seqs* s);
// selected NULL and n_selected < 0: attention over all pages
polykv_status check_pages_attend(const polykv_pages* pages, const polykv_pages_seqs* seqs, int32_t n_q_heads,
                                 const int32_t* selected, int64_t n_selected);

}  // namespace polykv
