// Index arithmetic of the paged cache, shared by its kernels and compiled for the host as well, so that
// the cases that could reach outside a buffer (pages that do not exist, lengths beyond the block table,
// starts that are out of order) are checked on the CPU.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define POLYKV_HD __host__ __device__ __forceinline__
#else
#define POLYKV_HD inline
#endif

namespace polykv {

constexpr int kPageStep = 16;           // tokens of one attention step; pages are a multiple of it
constexpr int kPagesMaxSeqs = 4096;     // sequences of one call (their step counts stand in shared memory)

// Status bits of a page cache (polykv_pages_status).
constexpr uint32_t kPagesBadPage = 1u;     // a page id outside [0, n_pages) where a token lives
constexpr uint32_t kPagesBadLength = 2u;   // a length beyond the block table, or starts out of order
constexpr uint32_t kPagesBadChoice = 4u;   // a chosen page beyond the sequence's last
constexpr uint32_t kPagesTimeout = 8u;     // a bounded wait gave up

// log2 of a page's tokens: 4 .. 7.
POLYKV_HD int page_shift(int page) { return page >= 128 ? 7 : (page >= 64 ? 6 : (page >= 32 ? 5 : 4)); }

// Pages that hold len tokens.
POLYKV_HD int64_t pages_of(int64_t len, int page) { return (len + page - 1) >> page_shift(page); }

// A length as the kernels use it: negative (an idle slot) counts as 0, one beyond the table is cut.
POLYKV_HD int64_t clamp_len(int64_t len, int64_t max_pages, int page, uint32_t* bad) {
    if (len <= 0) return 0;
    const int64_t room = max_pages * page;
    if (len > room) {
        *bad |= kPagesBadLength;
        return room;
    }
    return len;
}

// 16-token steps that attention takes for a sequence of (clamped) length len: over all of its tokens, or
// over n_sel chosen pages (n_sel < 0: all).
POLYKV_HD uint32_t seq_steps(int64_t len, int page, int n_sel) {
    if (n_sel < 0) return (uint32_t)((len + kPageStep - 1) / kPageStep);
    const int64_t pages = pages_of(len, page);
    return (uint32_t)((pages < n_sel ? pages : n_sel) * (page / kPageStep));
}

// Where a step's tokens are. valid = 0: nothing to read (a padded choice, or a page that does not exist).
struct StepAt {
    int64_t row;   // physical page * page + first slot: token row inside one (layer, kv head)'s pages
    int valid;     // tokens of the step that exist, 0..16
};

// Logical page and slot of a step; `chosen` is the entry of the choice list (ignored when n_sel < 0).
// Returns the logical page, or -1 where there is none to look up in the table.
POLYKV_HD int64_t step_page(uint32_t step, int page, int n_sel, int64_t chosen, int64_t len, int* slot, int* valid,
                            uint32_t* bad) {
    const int shift = page_shift(page) - 4;   // log2 of a page's steps
    const uint32_t at = step >> shift;
    *slot = (int)(step - (at << shift)) * kPageStep;
    *valid = 0;
    const int64_t lp = n_sel < 0 ? (int64_t)at : chosen;
    if (lp < 0) return -1;
    const int64_t left = len - (lp * page + *slot);
    if (lp * page >= len) {   // the lists of select() never name such a page
        *bad |= kPagesBadChoice;
        return -1;
    }
    if (left <= 0) return -1;
    *valid = left < kPageStep ? (int)left : kPageStep;
    return lp;
}

// What a window leaves of a sequence of (clamped) length len: the tokens [0, sinks) and [begin, len). Its pages are taken in
// order: the first `lead`, then those from page `from` on. Without a window (window = 0) that is all of them.
struct Window {
    int64_t begin, from;
    int32_t sinks, lead;
};
POLYKV_HD Window window_of(int64_t len, int page, int window, int sinks) {
    Window w;
    w.begin = window > 0 && len > window ? len - window : 0;
    w.sinks = window > 0 ? sinks : 0;
    const int64_t pages = pages_of(len, page), lead = pages_of(w.sinks, page);
    w.lead = (int32_t)(lead < pages ? lead : pages);
    const int64_t first = w.begin >> page_shift(page);
    w.from = first > w.lead ? first : w.lead;
    return w;
}
// Their 16-token steps: all but those of the pages between.
POLYKV_HD uint32_t window_steps(int64_t len, int page, const Window& w) {
    return (uint32_t)((len + kPageStep - 1) / kPageStep - ((w.from - w.lead) << (page_shift(page) - 4)));
}
// The page and slot of a step, and which of its 16 tokens are visible, a bit each (0: nothing to read).
POLYKV_HD int64_t window_page(uint32_t step, int page, const Window& w, int64_t len, int* slot, uint32_t* mask) {
    const int shift = page_shift(page) - 4;
    const uint32_t at = step >> shift;
    *slot = (int)(step - (at << shift)) * kPageStep;
    const int64_t lp = at < (uint32_t)w.lead ? (int64_t)at : w.from + (at - (uint32_t)w.lead);
    const int64_t t = lp * page + *slot;
    auto below = [&](int64_t end) {   // the step's tokens before `end`
        const int64_t n = end - t;
        return n >= kPageStep ? 0xffffu : (n <= 0 ? 0u : (1u << (int)n) - 1u);
    };
    *mask = below(len) & (~below(w.begin) | below(w.sinks));
    return lp;
}

// A page id from the table: in range, or -1 with the status bit.
POLYKV_HD int64_t check_page(int64_t id, int64_t n_pages, uint32_t* bad) {
    if (id >= 0 && id < n_pages) return id;
    *bad |= kPagesBadPage;
    return -1;
}

// The work items of an append are pages: item i of sequence s covers the tokens that fall into its
// (first + i)-th page. Sequence s owns the items [item_base(s), item_base(s + 1)): starts[s] / page + 2 s
// rises by at least n / page + 2 >= ceil((n - 1) / page) + 1, the most pages n tokens can touch, and the
// host needs no device value for the total, rows / page + 2 * seqs.
POLYKV_HD int64_t item_base(int64_t start, int64_t s, int page) { return (start >> page_shift(page)) + 2 * s; }

// One item's tokens. rows [row0, row0 + n) of k, v and q go to logical page lp, slots [slot0, slot0 + n).
struct AppendItem {
    int64_t lp, row0;
    int slot0, n;
};
// start/count: the sequence's rows (count <= 0: none); len: its tokens before; i: item within the sequence.
POLYKV_HD bool append_item(int64_t start, int64_t count, int64_t len, int64_t i, int page, AppendItem* it) {
    if (count <= 0 || len < 0 || i < 0) return false;
    const int64_t first = len >> page_shift(page);
    it->lp = first + i;
    const int64_t begin = it->lp * page > len ? it->lp * page : len;     // token range in the sequence
    const int64_t stop = (it->lp + 1) * page < len + count ? (it->lp + 1) * page : len + count;
    if (begin >= stop) return false;
    it->row0 = start + (begin - len);
    it->slot0 = (int)(begin - it->lp * page);
    it->n = (int)(stop - begin);
    return true;
}

// a / b, by the short division where both fit into 32 bits.
POLYKV_HD uint64_t quotient(uint64_t a, uint64_t b) {
    return ((a | b) >> 32) == 0 ? (uint64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// A list of `total` items cut into n contiguous shares whose sizes differ by at most one.
struct Shares {
    uint64_t q, big;   // share size, and items in the shares that have one more
    uint32_t r;        // how many those are
    POLYKV_HD Shares(uint64_t total, uint32_t n) {
        q = quotient(total, n);
        r = (uint32_t)(total - q * n);
        big = r * (q + 1);
    }
    POLYKV_HD uint64_t first(uint32_t c) const { return q * c + (c < r ? c : r); }   // of share c
    POLYKV_HD uint32_t of(uint64_t x) const {                                        // the share that holds item x
        return (uint32_t)(x < big ? quotient(x, q + 1) : r + quotient(x - big, q));
    }
};

}  // namespace polykv
