// The accepted branch's rows to consecutive positions of a paged cache, of 16-bit values
// (tv_commit_paged) or of 8-bit codes with a scale byte a row (tv_commit_paged_q8).
#pragma once

#include "tv_paged.cuh"

namespace tv {
namespace {

// As commit_kernel of the dense cache: one CTA per (sequence, kv head); the
// path is strictly increasing from 0, so path[d] >= d and a destination never
// lies past the sources still to be read; a batch reads all its rows before
// it writes any.  Row addresses come from the block table; every page that
// a moving row touches is checked before the first row moves.
constexpr int kCommitThreads = 256;
constexpr int kCommitChunks = 4;  // 16-byte chunks a thread carries per batch

// E: uint16_t, or uint8_t for codes, whose scale bytes ks, vs [num_pages, Hkv, page_size] move along.
template <typename E>
__global__ void __launch_bounds__(kCommitThreads)
commit_paged_kernel(E* __restrict__ k, E* __restrict__ v, uint8_t* __restrict__ ks,
                    uint8_t* __restrict__ vs, const PagedCache c, const int32_t* __restrict__ table,
                    const int32_t* __restrict__ kv_len, const int32_t* __restrict__ path,
                    const int32_t* __restrict__ accept_len, int N, int Hkv, int C, int P,
                    int32_t* __restrict__ new_kv_len, int32_t* __restrict__ status) {
  constexpr bool kScales = sizeof(E) == 1;
  __shared__ int32_t s_path[kMaxNodes];
  __shared__ long long s_src[kMaxNodes], s_dst[kMaxNodes];  // element offsets; -1: the row stays
  __shared__ long long s_sc[kScales ? 2 : 1][kScales ? kMaxNodes : 1];  // scales' offsets, from and to
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x / Hkv, h = blockIdx.x % Hkv;
  const int tid = threadIdx.x;
  const int L = __ldg(kv_len + b), a = __ldg(accept_len + b);
  int bad = !(L >= 0 && a >= 0 && a < N && TV_CHECK(N <= kMaxNodes));
  if (!bad)
    for (int d = tid; d <= a; d += kCommitThreads) {
      const int p = __ldg(path + (size_t)b * N + d);
      s_path[d] = p;
      bad |= (d == 0) ? (p != 0) : (p < d || p >= N);
    }
  bad = __syncthreads_or(bad);
  if (!bad) bad = (long long)L + s_path[a] >= ((long long)P << c.page_shift);
  if (!bad)
    for (int d = tid; d <= a; d += kCommitThreads) {
      if (d > 0) bad |= s_path[d] <= s_path[d - 1];
      long long off[2] = {-1, -1};
      if (d > 0 && s_path[d] != d) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int pos = L + (e ? d : s_path[d]), j = pos >> c.page_shift;
          const int row = pos & ((1 << c.page_shift) - 1);
          // (a path that does not rise may lead past the table before its end is seen)
          const int page = j < P ? __ldg(table + (size_t)b * P + j) : -1;
          bad |= page < 0 || page >= c.num_pages;
          off[e] = page * c.page_stride + h * c.head_stride + row * c.row_stride;
          if (kScales) s_sc[e % (kScales ? 2 : 1)][d] = (((long long)page * Hkv + h) << c.page_shift) + row;
        }
      }
      s_src[d] = off[0];
      s_dst[d] = off[1];
    }
  bad = __syncthreads_or(bad);
  if (h == 0 && tid == 0) {
    status[b] = bad ? TV_ERR_INVALID_ARG : TV_OK;
    new_kv_len[b] = bad ? L : L + a + 1;
  }
  if (bad) return;
  const int per_row = 2 * C;  // K and V chunks of a row
  const int rows_per_batch = max(1, kCommitThreads * kCommitChunks / per_row);
  for (int d0 = 1; d0 <= a; d0 += rows_per_batch) {
    const int rows = min(a + 1, d0 + rows_per_batch) - d0, items = rows * per_row;
    uint4 buf[kCommitChunks];
    uint8_t scale[kCommitChunks];  // (a batch has 512 rows at most)
#pragma unroll
    for (int u = 0; u < kCommitChunks; ++u) {
      const int w = tid + u * kCommitThreads;
      if (w < items) {
        const int d = d0 + w / per_row, t = (w / C) & 1, x = w % C;
        if (s_src[d] >= 0) buf[u] = reinterpret_cast<const uint4*>((t ? v : k) + s_src[d])[x];
      }
      if (kScales && w < 2 * rows && s_src[d0 + (w >> 1)] >= 0)
        scale[u] = ((w & 1) ? vs : ks)[s_sc[0][d0 + (w >> 1)]];
    }
    __syncthreads();  // every source of the batch is read before any destination is written
#pragma unroll
    for (int u = 0; u < kCommitChunks; ++u) {
      const int w = tid + u * kCommitThreads;
      if (w < items) {
        const int d = d0 + w / per_row, t = (w / C) & 1, x = w % C;
        if (s_dst[d] >= 0) reinterpret_cast<uint4*>((t ? v : k) + s_dst[d])[x] = buf[u];
      }
      if (kScales && w < 2 * rows && s_dst[d0 + (w >> 1)] >= 0)
        ((w & 1) ? vs : ks)[s_sc[kScales ? 1 : 0][d0 + (w >> 1)]] = scale[u];
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace tv
