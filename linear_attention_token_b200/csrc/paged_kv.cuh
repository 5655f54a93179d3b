// Device view of the paged key-value cache (include/attn.h), shared by its kernels.
#pragma once

#include "common.cuh"
#include "../../include/attn.h"

namespace gdn {

constexpr size_t kErrorBytes = 256;        // the error word at a workspace's start, padded

struct PagedView {
    unsigned char *k, *v;
    const int32_t *table;          // [num_seqs, max_pages]
    int num_pages, max_pages, page_shift, H_kv;
};

inline PagedView paged_view(const gdn_paged_kv &kv) {
    PagedView p;
    p.k = static_cast<unsigned char *>(kv.k);
    p.v = static_cast<unsigned char *>(kv.v);
    p.table = kv.page_table;
    p.num_pages = kv.num_pages;
    p.max_pages = kv.max_pages;
    p.page_shift = 0;
    while ((1 << p.page_shift) < kv.page_size) ++p.page_shift;
    p.H_kv = kv.H_kv;
    return p;
}

// Row of the cache (page x page_size + slot; multiply by H_kv d in 64 bits) that holds token t
// of sequence n, or -1 when the token is absent (include/attn.h).  t may be any value.
__device__ __forceinline__ int cache_row(const PagedView &c, int n, long long t) {
    const long long page = t >> c.page_shift;
    if (t < 0 || page >= c.max_pages) return -1;
    const int id = __ldg(c.table + (size_t)n * c.max_pages + page);
    if ((unsigned)id >= (unsigned)c.num_pages) return -1;
    return (id << c.page_shift) + (int)(t & ((1 << c.page_shift) - 1));
}

// Tokens the table of one sequence can hold.
__device__ __forceinline__ long long cache_capacity(const PagedView &c) {
    return (long long)c.max_pages << c.page_shift;
}

// Programmatic dependent launch: the join starts while the main kernel drains, and waits for its
// completion (and its memory) before it reads anything.
__device__ __forceinline__ void pdl_trigger() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace gdn
