// The paged KV cache as the kernels see it, and the host checks its entry
// points share.
#pragma once

#include "tv_common.cuh"

namespace tv {

struct PagedCache {
  long long page_stride, head_stride, row_stride;  // elements
  int num_pages, page_shift;                       // page_size = 1 << page_shift
};

// Strides of extent-one dimensions are never used by an address; they are set
// to a legal value, so that whatever the caller has there is not refused.
inline long long stride_or(long long stride, long long extent, long long other) {
  return extent == 1 ? other : stride;
}

// Checks a cache descriptor; fills `out`.
inline tv_status check_cache(const tv_paged_cache* c, PagedCache* out) {
  if (!c) return TV_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->Hkv < 1 || c->D < 1) return TV_ERR_INVALID_ARG;
  if (c->dtype != TV_BF16 && c->dtype != TV_FP16) return TV_ERR_UNSUPPORTED;
  int shift = 3;
  while (shift < 8 && (1 << shift) < c->page_size) ++shift;
  if (c->page_size != (1 << shift)) return TV_ERR_UNSUPPORTED;
  out->num_pages = c->num_pages;
  out->page_shift = shift;
  out->row_stride = c->row_stride;
  out->head_stride = stride_or(c->head_stride, c->Hkv, 8);
  out->page_stride = stride_or(c->page_stride, c->num_pages, 8);
  if (!c->k || !c->v) return TV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15)
    return TV_ERR_INVALID_ARG;
  if (out->row_stride < 0 || out->head_stride < 0 || out->page_stride < 0 ||
      ((out->row_stride | out->head_stride | out->page_stride) & 7))
    return TV_ERR_INVALID_ARG;
  return TV_OK;
}

// New tokens of sequence b: false for a malformed q_start.
__device__ __forceinline__ bool seq_range(const int32_t* q_start, int b, int T, int& t0, int& n) {
  t0 = __ldg(q_start + b);
  const int t1 = __ldg(q_start + b + 1);
  n = t1 - t0;
  return t0 >= 0 && t1 >= t0 && t1 <= T;
}

}  // namespace tv
