// tp_paged.cuh -- what the kernels over a paged key/value cache share: the
// index arithmetic (tp_paged_index.h), the status bit of a page outside the
// cache, and the view's construction on the host.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "tp_device.cuh"
#include "tp_internal.h"
#include "tp_paged_index.h"

namespace tpk {

// Status bit: a position whose page is not one of the cache's was met.
constexpr unsigned kStatusPage = 4u;

}  // namespace tpk

namespace tpi {

inline tpk::PagedView paged_view(const PagedArgs& a) {
    tpk::PagedView v{};
    v.table = a.page_table;
    v.q_start = a.q_start;
    v.kv_len = a.kv_len;
    v.n_pages = a.n_pages;
    v.rows = static_cast<int>(a.tokens);
    v.n_seqs = a.n_seqs;
    v.max_pages = a.max_pages;
    while ((1 << v.page_log2) < a.page_size) ++v.page_log2;
    v.kv_heads = a.kv_heads;
    v.d = a.head_dim;
    return v;
}

}  // namespace tpi
