// rlk_paged.h -- the paged key-value cache as the kernels see it, and what the
// translation units that work on it share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rlk_rollout.h"

namespace rlk {

struct PagedParams {
  const void* k;
  const void* v;
  int64_t num_pages, page_stride, token_stride, head_stride;
  int page_size, kv_heads, max_pages;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  const int32_t* new_lens;
  int n;
  int32_t* err;
};

// Length and number of new tokens of sequence b, or false where they do not
// agree with each other or with the page table's width.
__device__ __forceinline__ bool seq_lens(const PagedParams& P, int b, int& len, int& nnew) {
  len = P.lens[b];
  nnew = P.new_lens ? P.new_lens[b] : P.n;
  return nnew >= 0 && nnew <= P.n && len >= nnew &&
         len <= static_cast<int64_t>(P.max_pages) * P.page_size;
}

rlk_status check_cache(const rlk_kv_cache* c);
rlk_status check_bth(const void* p, const rlk_bth_strides* s, const char* what);
PagedParams paged_params(const rlk_kv_cache* c);

}  // namespace rlk
