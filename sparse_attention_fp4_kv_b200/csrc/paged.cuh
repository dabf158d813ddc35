// Page tables of the paged FP4 cache.
#pragma once

#include "common.cuh"

namespace csa2 {

// The pool and its tables, as every paged call takes them.
struct PagedKv {
    const int32_t *table;  // [S][max_pages]
    int max_pages, page_size, n_pages;
};

// Host-side checks shared by the paged calls. MAX_PAGES keeps an index and a grid's
// stride on top of it within 32 bits.
constexpr int MAX_PAGES = 1 << 30;
inline bool paged_shape_ok(int max_pages, int page_size, int n_pages) {
    return max_pages >= 1 && max_pages <= MAX_PAGES && page_size >= 1 && n_pages >= 1 && n_pages <= MAX_PAGES &&
           (int64_t)max_pages * page_size < (1ll << 40) && (int64_t)n_pages * page_size < (1ll << 40);
}

// pos = entry * page_size + slot. A 64-bit division costs tens of instructions
// more than a 32-bit one, and positions are rarely that far.
__device__ __forceinline__ void page_of(int64_t pos, int page_size, int64_t &entry, int &slot) {
    if ((uint64_t)pos >> 32) {
        entry = pos / page_size;
        slot = (int)(pos - entry * page_size);
    } else {
        const uint32_t e = (uint32_t)pos / (uint32_t)page_size;
        entry = e;
        slot = (int)((uint32_t)pos - e * (uint32_t)page_size);
    }
}

// Row of the pool (page * page_size + slot) that holds position pos of sequence
// b; -1 if it has no page.
__device__ __forceinline__ int64_t paged_row(const PagedKv &k, int64_t b, int64_t pos) {
    if (pos < 0) return -1;
    int64_t e;
    int slot;
    page_of(pos, k.page_size, e, slot);
    if (e >= k.max_pages) return -1;
    const int32_t page = __ldg(k.table + b * k.max_pages + e);
    if (page < 0 || page >= k.n_pages) return -1;
    return (int64_t)page * k.page_size + slot;
}

}  // namespace csa2
