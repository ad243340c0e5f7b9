// The paged KV cache's bookkeeping and writes: tv_page_map (block tables and
// slot maps from lengths), tv_paged_append (new K/V rows into their slots) and
// tv_commit_paged (the accepted branch's rows to consecutive positions:
// Speculative Decoding concept page, "The protocol" step 4; OPT-Tree §2).
//
// page map: the free pages are a stack.  With held_b pages and the target
// g_b = ceil((kv_len_b + n_b) / page_size), sequence b gives back
// r_b = max(0, held_b - g_b) pages and misses m_b = max(0, g_b - held_b).  R and M are
// the inclusive prefix sums of r and m over the sequences, F = R_last; b is
// served iff M_b <= n_free + F (so the served sequences that miss pages are a
// prefix of those that do).  Freed page f (0 <= f < F) is found by a binary
// search for the first b with R_b > f; the virtual stack is the old one with
// the freed pages on top, and the a-th popped page is entry n_free + F - 1 - a
// of it.  Every page that moves is thus found from the two prefix sums alone,
// by any thread, in any order: no atomics, and the result depends on the
// inputs only.  One cluster of 1 or 8 CTAs: each CTA scans all sequences into its
// shared memory, and once all have read the old n_pages and n_free (a cluster barrier)
// they share the writes.  No other word that a thread reads is written: pops
// read list entries below n_free and table entries at or past a target, while
// pushes write list entries at or past n_free and tables grow past held_b.
#define TV_UNIT 10
#include "tv_paged.cuh"
#include "tv_sm100.cuh"

namespace tv {
namespace {

constexpr int kMaxSeqs = 4096;

struct PageMapParams {
  const int32_t* q_start;
  const int32_t* kv_len;
  int32_t* table;
  int32_t* n_pages;
  int32_t* free_list;
  int32_t* n_free;
  int64_t* slots;
  int32_t* status;
  int B, T, P, shift, num_pages;
  int map_slots;  // this launch writes the slots too
};

// First index i in [0, n) with a[i] > x (a ascending), or n.
__device__ __forceinline__ int first_above(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// The sequence that token t belongs to, or n: end[b] is one past sequence b's last token (its first
// where its range is malformed), ascending unless q_start descends somewhere; then all are looked at.
__device__ __forceinline__ int owner_of(const int* end, const int32_t* q_start, int n, int t, bool descends) {
  if (!descends) return first_above(end, n, t);
  int b = 0;
  while (b < n && !(__ldg(q_start + b) >= 0 && t >= __ldg(q_start + b) && t < end[b])) ++b;
  return b;
}

__device__ __forceinline__ long long slot_of(int page, int pos, int shift, int num_pages) {
  return (page >= 0 && page < num_pages)
             ? ((long long)page << shift) + (pos & ((1 << shift) - 1)) : -1ll;
}

__global__ void __launch_bounds__(1024) page_map_kernel(const PageMapParams p) {
  extern __shared__ int s_dyn[];
  int* s_miss = s_dyn;         // inclusive prefix sums of the missing pages
  int* s_back = s_dyn + p.B;   // ... of the pages given back
  int* s_held = s_back + p.B;
  int* s_kv = s_held + p.B;    // cached tokens; -1: the sequence has a status already
  int* s_end = s_kv + p.B;     // one past each sequence's last token
  __shared__ int2 s_warp[32];
  __shared__ int s_taken;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, ctas = gridDim.x;
  const int per = ceil_div(p.B, nt), b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  if (tid == 0) s_taken = 0;
  const int n_free = *(volatile const int32_t*)p.n_free;
  int2 sum = make_int2(0, 0);
  bool falls = false;
  for (int b = b0; b < b1; ++b) {
    int t0, n;
    const bool range = seq_range(p.q_start, b, p.T, t0, n);
    falls |= t0 > __ldg(p.q_start + b + 1);
    const int kv = __ldg(p.kv_len + b), held = *(volatile const int32_t*)(p.n_pages + b);
    const long long want = ((long long)kv + n + (1 << p.shift) - 1) >> p.shift;
    const bool ok = range && kv >= 0 && held >= 0 && held <= p.P && want <= p.P;
    if (ok) {
      sum.x += max(0, (int)want - held);
      sum.y += max(0, held - (int)want);
    }
    s_miss[b] = sum.x;
    s_back[b] = sum.y;
    s_held[b] = held;
    s_kv[b] = ok ? kv : -1;
    s_end[b] = range ? t0 + n : t0;  // a malformed range owns no token
  }
  // block scan of the threads' sums
  int2 inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc.x, o), y = __shfl_up_sync(0xffffffffu, inc.y, o);
    if (lane >= o) {
      inc.x += x;
      inc.y += y;
    }
  }
  if (lane == 31) s_warp[warp] = inc;
  const bool descends = __syncthreads_or(falls);
  int2 base = make_int2(inc.x - sum.x, inc.y - sum.y), total = make_int2(0, 0);
  for (int w = 0; w < nt / 32; ++w) {
    if (w < warp) {
      base.x += s_warp[w].x;
      base.y += s_warp[w].y;
    }
    total.x += s_warp[w].x;
    total.y += s_warp[w].y;
  }
  const int F = total.y;
  const bool bad = n_free < 0 || n_free > p.num_pages || F > p.num_pages - n_free;
  const int size = n_free + F;
  int taken = 0, before = base.x;
  for (int b = b0; b < b1; ++b) {
    const int m = (s_miss[b] += base.x);
    s_back[b] += base.y;
    if (m > before && m <= size) taken = m;
    before = m;
  }
  if (taken) atomicMax(&s_taken, taken);
  __syncthreads();
  if (ctas > 1) sm100::cluster_sync();  // n_pages and n_free have been read everywhere
  const int A = bad ? 0 : s_taken;

  auto miss_before = [&](int b) { return b ? s_miss[b - 1] : 0; };
  auto back_before = [&](int b) { return b ? s_back[b - 1] : 0; };
  auto freed_page = [&](int f) {
    const int b = first_above(s_back, p.B, f);
    if (!TV_IN(b, p.B)) return -1;
    const int target = s_held[b] - (s_back[b] - back_before(b));
    const int j = target + f - back_before(b);
    return TV_IN(j, p.P) ? p.table[(size_t)b * p.P + j] : -1;
  };
  auto popped_page = [&](int a) {
    const int i = size - 1 - a;
    if (!TV_IN(i, p.num_pages)) return -1;
    return i < n_free ? p.free_list[i] : freed_page(i - n_free);
  };
  const int g0 = rank * nt + tid, gs = ctas * nt;
  for (int b = g0; b < p.B; b += gs) {
    const int miss = s_miss[b] - miss_before(b), back = s_back[b] - back_before(b);
    int st = TV_OK;
    if (bad || s_kv[b] < 0) st = TV_ERR_INVALID_ARG;
    else if (miss > 0 && s_miss[b] > size) st = TV_ERR_NO_PAGES;
    else if (miss | back) p.n_pages[b] = s_held[b] + miss - back;
    p.status[b] = st;
  }
  if (!bad) {
    // (four pages a thread at a time: their reads overlap)
    for (int a0 = g0; a0 < A; a0 += 4 * gs) {
      int page[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (a0 + u * gs < A) page[u] = popped_page(a0 + u * gs);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int a = a0 + u * gs;
        if (a >= A) break;
        const int b = first_above(s_miss, p.B, a);
        if (!TV_IN(b, p.B)) continue;
        const int j = s_held[b] + a - miss_before(b);
        if (TV_IN(j, p.P)) p.table[(size_t)b * p.P + j] = page[u];
      }
    }
    for (int f0 = g0; f0 < F - A; f0 += 4 * gs) {
      int page[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (f0 + u * gs < F - A) page[u] = freed_page(f0 + u * gs);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int f = f0 + u * gs;
        if (f < F - A && TV_IN(n_free + f, p.num_pages)) p.free_list[n_free + f] = page[u];
      }
    }
    if (g0 == 0) *p.n_free = size - A;
  }
  if (!p.map_slots) return;
  for (int t = g0; t < p.T; t += gs) {
    const int b = owner_of(s_end, p.q_start, p.B, t, descends);
    long long slot = -1;
    if (!bad && b < p.B && s_kv[b] >= 0) {
      const int first = __ldg(p.q_start + b);
      const int miss = s_miss[b] - miss_before(b);
      if (t >= first && !(miss > 0 && s_miss[b] > size)) {
        const int pos = s_kv[b] + t - first, j = pos >> p.shift;
        const int page = j < s_held[b]
                             ? (TV_IN(j, p.P) ? p.table[(size_t)b * p.P + j] : -1)
                             : popped_page(miss_before(b) + j - s_held[b]);
        slot = slot_of(page, pos, p.shift, p.num_pages);
      }
    }
    p.slots[t] = slot;
  }
}

// Slots from tables that are already at their lengths (many tokens: one
// cluster's eight SMs would take longer than this second, wider launch).
constexpr int kSlotThreads = 256, kSlotTokens = 1024;

__global__ void __launch_bounds__(kSlotThreads) page_slots_kernel(const PageMapParams p) {
  extern __shared__ int s_dyn[];
  int* s_end = s_dyn;
  pdl_trigger();
  pdl_wait();
  bool falls = false;
  for (int b = threadIdx.x; b < p.B; b += kSlotThreads) {
    int t0, n;
    s_end[b] = seq_range(p.q_start, b, p.T, t0, n) ? t0 + n : t0;
    falls |= t0 > __ldg(p.q_start + b + 1);
  }
  const bool descends = __syncthreads_or(falls);
  const int base = blockIdx.x * kSlotTokens + threadIdx.x;
#pragma unroll
  for (int u = 0; u < kSlotTokens / kSlotThreads; ++u) {
    const int t = base + u * kSlotThreads;
    if (t >= p.T) return;
    const int b = owner_of(s_end, p.q_start, p.B, t, descends);
    long long slot = -1;
    if (b < p.B && __ldg(p.status + b) == TV_OK) {
      const int first = __ldg(p.q_start + b);
      const int pos = __ldg(p.kv_len + b) + t - first, j = pos >> p.shift;
      if (t >= first && j < __ldg(p.n_pages + b) && TV_IN(j, p.P))
        slot = slot_of(__ldg(p.table + (size_t)b * p.P + j), pos, p.shift, p.num_pages);
    }
    p.slots[t] = slot;
  }
}

// ------------------------------------------------------------------- append
// A thread carries U 16-byte chunks (all its loads in flight before its first
// store), chunk c of the flat order token, K then V, head, chunk of the row.
constexpr int kAppendThreads = 256;

struct AppendParams {
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* kp;
  uint16_t* vp;
  const int64_t* slots;
  int32_t* status;
  long long token_stride, head_stride;
  PagedCache c;
  int T, Hkv, C;  // C: 16-byte chunks per row
};

template <int U>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  pdl_trigger();
  pdl_wait();
  const unsigned per_side = (unsigned)p.Hkv * p.C, per_token = 2 * per_side;
  const unsigned items = (unsigned)p.T * per_token;
  const unsigned base = blockIdx.x * (kAppendThreads * U) + threadIdx.x;
  const long long limit = (long long)p.c.num_pages << p.c.page_shift;
  uint4 x[U];
  uint4* dst[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const unsigned i = base + u * kAppendThreads;
    dst[u] = nullptr;
    if (i < items) {
      const unsigned t = i / per_token, w = i - t * per_token;
      const unsigned side = w >= per_side, r = w - side * per_side;
      const unsigned h = r / p.C, c = r - h * p.C;
      const long long slot = __ldg(reinterpret_cast<const long long*>(p.slots) + t);
      const bool in = slot >= 0 && slot < limit;
      if (w == 0 && p.status) p.status[t] = slot >= limit ? TV_ERR_INVALID_ARG : TV_OK;
      if (in) {
        const long long page = slot >> p.c.page_shift, row = slot & ((1ll << p.c.page_shift) - 1);
        dst[u] = reinterpret_cast<uint4*>((side ? p.vp : p.kp) + page * p.c.page_stride +
                                          h * p.c.head_stride + row * p.c.row_stride) + c;
        x[u] = __ldg(reinterpret_cast<const uint4*>((side ? p.v : p.k) + t * p.token_stride +
                                                    h * p.head_stride) + c);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (dst[u]) *dst[u] = x[u];
}

// ------------------------------------------------------------------- commit
// As commit_kernel of the dense cache: one CTA per (sequence, kv head); the
// path is strictly increasing from 0, so path[d] >= d and a destination never
// lies past the sources still to be read; a batch reads all its rows before
// it writes any.  Row addresses come from the block table; every page that
// a moving row touches is checked before the first row moves.
constexpr int kCommitThreads = 256;
constexpr int kCommitChunks = 4;  // 16-byte chunks a thread carries per batch

__global__ void __launch_bounds__(kCommitThreads)
commit_paged_kernel(uint16_t* __restrict__ k, uint16_t* __restrict__ v, const PagedCache c,
                    const int32_t* __restrict__ table, const int32_t* __restrict__ kv_len,
                    const int32_t* __restrict__ path, const int32_t* __restrict__ accept_len, int N,
                    int Hkv, int C, int P, int32_t* __restrict__ new_kv_len,
                    int32_t* __restrict__ status) {
  __shared__ int32_t s_path[kMaxNodes];
  __shared__ long long s_src[kMaxNodes], s_dst[kMaxNodes];  // element offsets; -1: the row stays
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
          // (a path that does not rise may lead past the table before its end is seen)
          const int page = j < P ? __ldg(table + (size_t)b * P + j) : -1;
          bad |= page < 0 || page >= c.num_pages;
          off[e] = page * c.page_stride + h * c.head_stride +
                   (pos & ((1 << c.page_shift) - 1)) * c.row_stride;
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
    const int items = (min(a + 1, d0 + rows_per_batch) - d0) * per_row;
    uint4 buf[kCommitChunks];
#pragma unroll
    for (int u = 0; u < kCommitChunks; ++u) {
      const int w = tid + u * kCommitThreads;
      if (w < items) {
        const int d = d0 + w / per_row, t = (w / C) & 1, x = w % C;
        if (s_src[d] >= 0) buf[u] = reinterpret_cast<const uint4*>((t ? v : k) + s_src[d])[x];
      }
    }
    __syncthreads();  // every source of the batch is read before any destination is written
#pragma unroll
    for (int u = 0; u < kCommitChunks; ++u) {
      const int w = tid + u * kCommitThreads;
      if (w < items) {
        const int d = d0 + w / per_row, t = (w / C) & 1, x = w % C;
        if (s_dst[d] >= 0) reinterpret_cast<uint4*>((t ? v : k) + s_dst[d])[x] = buf[u];
      }
    }
    __syncthreads();
  }
}

tv_status launched(cudaError_t e) {
  if (e == cudaSuccess) return TV_OK;
  (void)cudaGetLastError();
  return TV_ERR_CUDA;
}

}  // namespace
}  // namespace tv

extern "C" tv_status tv_page_map(const int32_t* q_start, const int32_t* kv_len, int B, int T, int P,
                                 int page_size, int num_pages, int32_t* block_table,
                                 int32_t* n_pages, int32_t* free_list, int32_t* n_free,
                                 int64_t* slots, int32_t* status, cudaStream_t stream) {
  TV_NVTX_RANGE("tv_page_map");
  if (B < 0 || T < 0 || P < 1 || num_pages < 1) return TV_ERR_INVALID_ARG;
  int shift = 3;
  while (shift < 8 && (1 << shift) < page_size) ++shift;
  if (page_size != (1 << shift)) return TV_ERR_UNSUPPORTED;
  if (B > tv::kMaxSeqs || (long long)B * P > 0x7fffffffll) return TV_ERR_UNSUPPORTED;
  if (T > 0x7fffffff - tv::kSlotTokens || ((long long)P << shift) > 0x7fffffffll)
    return TV_ERR_UNSUPPORTED;
  if (B == 0 && T == 0) return TV_OK;
  if (!q_start || !free_list || !n_free || (T > 0 && !slots)) return TV_ERR_INVALID_ARG;
  if (B > 0 && (!kv_len || !block_table || !n_pages || !status)) return TV_ERR_INVALID_ARG;
  tv::PageMapParams p{q_start, kv_len, block_table, n_pages, free_list, n_free, slots,
                      status,  B,      T,           P,       shift,     num_pages, 1};
  // (growing by prompts of 40 to 2,000 tokens and back: 16 of them 9.6 us with the slots in the first launch,
  // 12.2 us with the wide one behind it; 64 of them 21.0 and 17.6 us)
  const bool wide = T > 16384;
  p.map_slots = !wide;
  const int smem = 5 * B * (int)sizeof(int);
  // The pages that move are known to the device alone; the tables' size bounds them.  Growing by
  // 200 prompts (12,600 pages) and releasing them again takes 36 us where the release runs on one CTA,
  // 16 us on a cluster; a decode step of 64 sequences and its way back 6.6 and 7.8 us.
  const long long most = (long long)B * P;
  const int ctas = (T > 1024 || B > 512 || most > 8192) ? 8 : 1;
  // (a decode step of 64 and its way back 7.8 us with 256 threads a CTA, 8.2 with 512; 200 prompts 17.4,
  // 15.5 and with 1,024 threads 16.8 us; 4,000 decode sequences 36.7, 24.2 and 21.0 us)
  const int threads = B > 1024 ? 1024 : (T > 1024 || B > 128) ? 512 : 256;
  if (!tv::set_dyn_smem(tv::page_map_kernel, 5 * tv::kMaxSeqs * (int)sizeof(int)))
    return TV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  const tv_status st = tv::launched(cudaLaunchKernelEx(&cfg, tv::page_map_kernel, p));
  if (st != TV_OK || !wide) return st;
  return tv::launched(tv::launch_pdl(tv::page_slots_kernel, dim3(tv::ceil_div(T, tv::kSlotTokens)),
                                     dim3(tv::kSlotThreads), B * sizeof(int), stream, p));
}

extern "C" tv_status tv_paged_append(const void* k, const void* v, int64_t token_stride,
                                     int64_t head_stride, const int64_t* slots, int T,
                                     const tv_paged_cache* cache, int32_t* status,
                                     cudaStream_t stream) {
  TV_NVTX_RANGE("tv_paged_append");
  if (T < 0) return TV_ERR_INVALID_ARG;
  tv::AppendParams p;
  const tv_status st = tv::check_cache(cache, &p.c);
  if (st != TV_OK) return st;
  const int Hkv = cache->Hkv, D = cache->D;
  if (D % 8 != 0 || D > 1024) return TV_ERR_UNSUPPORTED;
  if ((long long)T * Hkv * (D / 8) > (1ll << 30) - 4096) return TV_ERR_UNSUPPORTED;
  if (T == 0) return TV_OK;
  if (!k || !v || !slots) return TV_ERR_INVALID_ARG;
  p.token_stride = tv::stride_or(token_stride, T, 8);
  p.head_stride = tv::stride_or(head_stride, Hkv, 8);
  if (p.token_stride < 0 || p.head_stride < 0 || ((p.token_stride | p.head_stride) & 7))
    return TV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15)
    return TV_ERR_INVALID_ARG;
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.kp = static_cast<uint16_t*>(cache->k);
  p.vp = static_cast<uint16_t*>(cache->v);
  p.slots = slots;
  p.status = status;
  p.T = T;
  p.Hkv = Hkv;
  p.C = D / 8;
  const long long items = 2ll * T * Hkv * p.C;
  const int per = tv::kAppendThreads;
  // Rows of 8 heads of 128: 64 and 2,000 tokens take 1.4 and 3.2 us with one chunk a thread, 2.3 and 4.9 us
  // with four; 8,192 tokens 14.0 and 12.0 us (78 % of what a copy reaches).
  if (items <= (long long)per * 24 * tv::device_sm_count())
    return tv::launched(tv::launch_pdl(tv::append_kernel<1>, dim3((unsigned)((items + per - 1) / per)),
                                       dim3(per), 0, stream, p));
  return tv::launched(tv::launch_pdl(tv::append_kernel<4>,
                                     dim3((unsigned)((items + 4 * per - 1) / (4 * per))), dim3(per),
                                     0, stream, p));
}

extern "C" tv_status tv_commit_paged(const tv_paged_cache* cache, const int32_t* block_table,
                                     const int32_t* kv_len, const int32_t* path,
                                     const int32_t* accept_len, int B, int N, int P,
                                     int32_t* new_kv_len, int32_t* status, cudaStream_t stream) {
  TV_NVTX_RANGE("tv_commit_paged");
  if (B < 0 || N < 1 || N > TV_MAX_NODES || P < 1) return TV_ERR_INVALID_ARG;
  tv::PagedCache c;
  const tv_status st = tv::check_cache(cache, &c);
  if (st != TV_OK) return st;
  if (cache->D % 8 != 0 || cache->D > 1024) return TV_ERR_UNSUPPORTED;
  if ((long long)B * P > 0x7fffffffll || (long long)B * cache->Hkv > 0x7fffffffll ||
      ((long long)P << c.page_shift) > 0x7fffffffll - TV_MAX_NODES)
    return TV_ERR_UNSUPPORTED;
  if (B == 0) return TV_OK;
  if (!block_table || !kv_len || !path || !accept_len || !new_kv_len || !status)
    return TV_ERR_INVALID_ARG;
  if (new_kv_len == kv_len) return TV_ERR_INVALID_ARG;
  return tv::launched(tv::launch_pdl(
      tv::commit_paged_kernel, dim3((unsigned)(B * cache->Hkv)), dim3(tv::kCommitThreads), 0, stream,
      static_cast<uint16_t*>(cache->k), static_cast<uint16_t*>(cache->v), c, block_table, kv_len,
      path, accept_len, N, cache->Hkv, cache->D / 8, P, new_kv_len, status));
}
