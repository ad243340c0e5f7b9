// The 8-bit paged cache's writes and reads: tv_paged_append_q8 (new K and V rows quantised into their
// slots), tv_paged_read_q8 (rows of sequences as 16-bit values) and tv_commit_paged_q8 (the accepted
// branch's rows: Speculative Decoding concept page, "The protocol" step 4; OPT-Tree §2).
//
// A row x of D values becomes codes c_i and a scale byte s: with e = s - 127 the least exponent from
// -126 on with max |x_i| <= M 2^e, c_i = x_i 2^-e to the nearest e4m3 (M = 448) or whole number (M = 127),
// ties to even.  A power of two costs e4m3 nothing (its step goes with the value, off by at most 2^-4 of
// it) and int8 up to a bit (a step is at most max|x| / 63.5, half of it the error); in return scaling is
// exact, so a code is off by one rounding and the same on every machine, and a code's value is a bf16
// number, so reading back rounds nothing and a row that is written again keeps its codes' values.
#define TV_UNIT 14
#include "tv_commit_paged.cuh"
#include "tv_quant.cuh"

namespace tv {
namespace {

tv_status launched(cudaError_t e) {
  if (e == cudaSuccess) return TV_OK;
  (void)cudaGetLastError();
  return TV_ERR_CUDA;
}

// ------------------------------------------------------------------- append
// A row goes to 1 << row_lanes lanes, U units of 16 values each, all loads in flight ahead of the
// row's maximum, which takes row_lanes shuffles.  Bound by HBM (3 D + 1 bytes a row): 8,192 tokens of 8 heads of 128
// take 9.6 us, 73 % of the copy rate (10.4 us when a lane stored 8 codes at a time); 64 tokens 1.6 us, a launch's
// latency.
constexpr int kRowThreads = 256;

struct AppendQ8Params {
  const uint16_t* k;
  const uint16_t* v;
  const int64_t* slots;
  int32_t* status;
  long long token_stride, head_stride;
  Q8Cache c;
  int T, units, row_lanes;  // units: of 16 values in a row
};

template <bool E4M3, bool F16, int U>
__global__ void __launch_bounds__(kRowThreads) append_q8_kernel(const AppendQ8Params p) {
  pdl_trigger();
  pdl_wait();
  const unsigned item = blockIdx.x * kRowThreads + threadIdx.x, lanes = 1u << p.row_lanes;
  const unsigned r = item >> p.row_lanes, lane = item & (lanes - 1);
  const unsigned per_token = 2 * p.c.Hkv, t = r / per_token, w = r - t * per_token;
  const bool side = w >= (unsigned)p.c.Hkv;
  const int h = side ? w - p.c.Hkv : w;
  const bool is_row = t < (unsigned)p.T;
  const long long slot = is_row ? __ldg(reinterpret_cast<const long long*>(p.slots) + t) : -1;
  const long long limit = (long long)p.c.num_pages << p.c.page_shift;
  const bool in = slot >= 0 && slot < limit;
  if (is_row && w == 0 && lane == 0 && p.status) p.status[t] = slot >= limit ? TV_ERR_INVALID_ARG : TV_OK;
  uint4 x[U][2];
  const uint4* src = reinterpret_cast<const uint4*>((side ? p.v : p.k) + (long long)t * p.token_stride +
                                                    h * p.head_stride);
#pragma unroll
  for (int c = 0; c < 2 * U; ++c) {
    const int at = lane + (c >> 1) * lanes;
    x[c >> 1][c & 1] = in && at < p.units ? __ldg(src + 2 * at + (c & 1)) : make_uint4(0, 0, 0, 0);
  }
  // the largest magnitude: 16-bit floats without their sign are in the order of their bits
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < 2 * U; ++c) {
    const uint32_t m = 0x7fff7fffu;
    const uint4 v = x[c >> 1][c & 1];
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m)));
  }
  top = max(top & 0xffffu, top >> 16);
  for (int o = 1; o < (int)lanes; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (!in) return;
  const int s = q8::scale_of<E4M3>(q8::unpack<F16>(top).x);
  // (2^-e; rows that are no numbers get codes of 0)
  const float f = s == q8::kNaN ? 0.0f : __int_as_float((254 - s) << 23);
  const long long page = slot >> p.c.page_shift;
  const int row = (int)(slot & ((1ll << p.c.page_shift) - 1));
  uint4* dst = reinterpret_cast<uint4*>((side ? p.c.v : p.c.k) + p.c.code_at(page, h, row));
#pragma unroll
  for (int c = 0; c < U; ++c) {
    const uint32_t in8[8] = {x[c][0].x, x[c][0].y, x[c][0].z, x[c][0].w, x[c][1].x, x[c][1].y, x[c][1].z, x[c][1].w};
    uint32_t out4[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 y[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        y[k] = q8::unpack<F16>(s == q8::kNaN ? 0u : in8[2 * i + k]);
        y[k].x *= f;
        y[k].y *= f;
      }
      out4[i] = q8::encode4<E4M3>(y[0], y[1]);
    }
    const int at = lane + c * lanes;
    if (at < p.units) dst[at] = make_uint4(out4[0], out4[1], out4[2], out4[3]);
  }
  if (lane == 0) (side ? p.c.vs : p.c.ks)[p.c.scale_at(page, h, row)] = (uint8_t)s;
}

template <bool E4M3, bool F16>
cudaError_t launch_append(const AppendQ8Params& p, int U, unsigned blocks, cudaStream_t stream) {
  if (U == 1) return launch_pdl(append_q8_kernel<E4M3, F16, 1>, dim3(blocks), dim3(kRowThreads), 0, stream, p);
  return launch_pdl(append_q8_kernel<E4M3, F16, 2>, dim3(blocks), dim3(kRowThreads), 0, stream, p);
}

// --------------------------------------------------------------------- read
// A CTA takes `tokens` consecutive tokens: a thread each finds its token's sequence (a binary search of
// the starts) and row, then all stream the rows, 16 codes a step, four steps in flight (two take as long, eight
// 103 us for the 85 that four took then: fewer warps).  Bound by HBM (3 D + 1 bytes a row): 16 sequences of 512 to 8,192
// tokens, 8 heads of 128, take 73 us, 86 % of the copy rate; 84.5 us while each step divided for its place and
// every value was held against the type's largest.
constexpr int kReadTokens = 32, kReadFlight = 4;

struct ReadQ8Params {
  Q8Cache c;
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* start;
  uint16_t* k;
  uint16_t* v;
  int32_t* status;
  int B, T, P, tokens, units;  // units: of 16 codes in a row
  int step_c, step_w, step_t;  // kRowThreads units as units of a row, rows of a token and tokens
  int blocks;                  // CTAs of tokens; those behind them write the sequences' status
};

// The last sequence that starts at or before token t, or -1, if the starts ascend.
__device__ __forceinline__ int seq_of(const ReadQ8Params& p, int t) {
  int lo = 0, hi = p.B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.q_start + mid) <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

// Whether a sequence's rows lie within the table.
__device__ __forceinline__ bool read_fits(const ReadQ8Params& p, int start, int n) {
  return start >= 0 && (long long)start + n <= ((long long)p.P << p.c.page_shift);
}

// Scale bytes up to this one give no value (448 2^e or 128 2^e at most) past the type's largest.
template <bool E4M3, bool F16>
constexpr int kSafeScale = 127 + (E4M3 ? (F16 ? 7 : 119) : (F16 ? 8 : 120));

template <bool F16>
__device__ __forceinline__ uint32_t narrow(float2 y, float f, bool safe) {
  y.x *= f;
  y.y *= f;
  if (!safe) {
    const float most = F16 ? 65504.0f : 3.38953139e38f;  // (a code's value may be past it; a NaN stays)
    if (fabsf(y.x) > most) y.x = copysignf(most, y.x);
    if (fabsf(y.y) > most) y.y = copysignf(most, y.y);
  }
  if (F16) {
    const __half2 o = __floats2half2_rn(y.x, y.y);
    return *reinterpret_cast<const uint32_t*>(&o);
  }
  const __nv_bfloat162 o = __floats2bfloat162_rn(y.x, y.y);
  return *reinterpret_cast<const uint32_t*>(&o);
}

template <bool E4M3, bool F16>
__global__ void __launch_bounds__(kRowThreads) read_q8_kernel(const ReadQ8Params p) {
  __shared__ int s_page[kReadTokens], s_row[kReadTokens];  // page -1: zeros, -2: nobody's token
  __shared__ int s_owner[kReadTokens];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= p.blocks) {  // a warp per sequence
    const int b = ((int)blockIdx.x - p.blocks) * (kRowThreads / 32) + (tid >> 5);
    if (b >= p.B) return;
    int t0, n;
    bool ok = seq_range(p.q_start, b, p.T, t0, n);
    const int start = __ldg(p.start + b);
    ok = ok && read_fits(p, start, n);
    if (ok && n > 0)
      for (int j = (start >> p.c.page_shift) + (tid & 31); j <= (start + n - 1) >> p.c.page_shift; j += 32) {
        const int page = TV_IN(j, p.P) ? __ldg(p.table + (size_t)b * p.P + j) : -1;
        ok = ok && page >= 0 && page < p.c.num_pages;
      }
    // (a search that finds its first and last token finds those between, as one path through the starts does.  One that
    // does not means starts that descend: its rows are its own then if no other sequence has tokens of it)
    if (seq_range(p.q_start, b, p.T, t0, n) && n > 0 && (seq_of(p, t0) != b || seq_of(p, t0 + n - 1) != b))
      for (int o = tid & 31; o < p.B; o += 32) {
        int s0, sn;
        if (o != b && seq_range(p.q_start, o, p.T, s0, sn)) ok = ok && (s0 >= t0 + n || s0 + sn <= t0 || sn == 0);
      }
    ok = __all_sync(0xffffffffu, ok);
    if ((tid & 31) == 0 && p.status) p.status[b] = ok ? TV_OK : TV_ERR_INVALID_ARG;
    return;
  }
  const int first = blockIdx.x * p.tokens, count = min(p.tokens, p.T - first);
  const int token = first + tid;
  int b = -1, t0 = 0, n = 0;
  if (tid < count) {
    b = seq_of(p, token);
    if (b >= 0 && !(seq_range(p.q_start, b, p.T, t0, n) && token >= t0 && token - t0 < n)) b = -1;
    s_owner[tid] = p.B;
  }
  if (__syncthreads_or(tid < count && b < 0)) {  // nobody's tokens, or starts that descend: the first that has them
    for (int o = tid; o < p.B; o += kRowThreads) {
      int s0, sn;
      if (seq_range(p.q_start, o, p.T, s0, sn))
        for (int i = max(s0 - first, 0); i < min(s0 + sn - first, count); ++i) atomicMin(&s_owner[i], o);
    }
    __syncthreads();
    if (tid < count && b < 0 && s_owner[tid] < p.B) {
      b = s_owner[tid];
      seq_range(p.q_start, b, p.T, t0, n);
    }
  }
  if (tid < count) {
    int page = -2, row = 0;
    if (b >= 0) {
      const int start = __ldg(p.start + b);
      page = -1;
      if (read_fits(p, start, n)) {
        const int pos = start + token - t0, j = pos >> p.c.page_shift;
        page = TV_IN(j, p.P) ? __ldg(p.table + (size_t)b * p.P + j) : -1;
        if (page < 0 || page >= p.c.num_pages) page = -1;
        row = pos & ((1 << p.c.page_shift) - 1);
      }
    }
    s_page[tid] = page;
    s_row[tid] = row;
  }
  __syncthreads();
  const int rows = 2 * p.c.Hkv;  // of a token, K's ahead of V's
  int c = tid % p.units, w = tid / p.units % rows, t = tid / p.units / rows;
  while (t < count) {
    uint4 x[kReadFlight], *dst[kReadFlight];
    int s[kReadFlight];
#pragma unroll
    for (int u = 0; u < kReadFlight; ++u) {
      dst[u] = nullptr;
      if (t < count) {
        const bool side = w >= p.c.Hkv;
        const int h = side ? w - p.c.Hkv : w, page = s_page[t];
        x[u] = make_uint4(0, 0, 0, 0);
        s[u] = 1;
        if (page >= -1)
          dst[u] = reinterpret_cast<uint4*>(
              (side ? p.v : p.k) + (((long long)(first + t) * p.c.Hkv + h) * p.units + c) * 16);
        if (page >= 0) {
          x[u] = __ldg(reinterpret_cast<const uint4*>((side ? p.c.v : p.c.k) + p.c.code_at(page, h, s_row[t])) + c);
          s[u] = __ldg((side ? p.c.vs : p.c.ks) + p.c.scale_at(page, h, s_row[t]));
        }
      }
      // kRowThreads units of 16 codes on
      c += p.step_c;
      w += p.step_w;
      t += p.step_t;
      if (c >= p.units) {
        c -= p.units;
        ++w;
      }
      if (w >= rows) {
        w -= rows;
        ++t;
      }
    }
#pragma unroll
    for (int u = 0; u < kReadFlight; ++u) {
      if (!dst[u]) continue;
      const float f = q8::factor(s[u]);
      const bool safe = s[u] <= kSafeScale<E4M3, F16>;
      const uint32_t c4[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 a, b;
        q8::decode4<E4M3>(c4[i], a, b);
        o[2 * i] = narrow<F16>(a, f, safe);
        o[2 * i + 1] = narrow<F16>(b, f, safe);
      }
      dst[u][0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[u][1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

}  // namespace
}  // namespace tv

extern "C" tv_status tv_paged_append_q8(const void* k, const void* v, int64_t token_stride,
                                        int64_t head_stride, const int64_t* slots, int T,
                                        const tv_q8_cache* cache, int32_t* status,
                                        cudaStream_t stream) {
  TV_NVTX_RANGE("tv_paged_append_q8");
  if (T < 0) return TV_ERR_INVALID_ARG;
  tv::AppendQ8Params p;
  const tv_status st = tv::check_q8_cache(cache, &p.c);
  if (st != TV_OK) return st;
  const int Hkv = cache->Hkv, D = cache->D;
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
  p.slots = slots;
  p.status = status;
  p.T = T;
  p.units = D / 16;
  // Half the threads where a unit each would be more than half as many again as the GPU holds (8 CTAs an SM): 8,192,
  // 4,096 and 2,048 tokens of 8 heads of 128 take 9.6, 6.1 and 4.4 us with two units, 10.3, 6.2 and 4.1 us with one.
  const bool many = 2ll * T * Hkv * p.units > 12ll * tv::kRowThreads * tv::device_sm_count();
  const int U = p.units > 32 || (p.units > 1 && many) ? 2 : 1;
  p.row_lanes = 0;
  while (p.row_lanes < 5 && (U << p.row_lanes) < p.units) ++p.row_lanes;
  const long long threads = (2ll * T * Hkv) << p.row_lanes;
  const unsigned blocks = (unsigned)((threads + tv::kRowThreads - 1) / tv::kRowThreads);
  const bool f16 = cache->dtype == TV_FP16;
  if (cache->format == TV_E4M3)
    return tv::launched(f16 ? tv::launch_append<true, true>(p, U, blocks, stream)
                            : tv::launch_append<true, false>(p, U, blocks, stream));
  return tv::launched(f16 ? tv::launch_append<false, true>(p, U, blocks, stream)
                          : tv::launch_append<false, false>(p, U, blocks, stream));
}

extern "C" tv_status tv_paged_read_q8(const tv_q8_cache* cache, const int32_t* block_table,
                                      const int32_t* q_start, const int32_t* start, int B, int T, int P,
                                      void* k, void* v, int32_t* status, cudaStream_t stream) {
  TV_NVTX_RANGE("tv_paged_read_q8");
  if (B < 0 || T < 0 || P < 1) return TV_ERR_INVALID_ARG;
  tv::ReadQ8Params p;
  const tv_status st = tv::check_q8_cache(cache, &p.c);
  if (st != TV_OK) return st;
  const int Hkv = cache->Hkv, D = cache->D;
  if (B > tv::kMaxSeqs || (long long)B * P > 0x7fffffffll ||
      ((long long)P << p.c.page_shift) > 0x7fffffffll || (long long)Hkv * (D / 16) > (1 << 20))
    return TV_ERR_UNSUPPORTED;
  if (B == 0) return TV_OK;
  if (!block_table || !q_start || !start || (T > 0 && (!k || !v))) return TV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15)
    return TV_ERR_INVALID_ARG;
  p.table = block_table;
  p.q_start = q_start;
  p.start = start;
  p.k = static_cast<uint16_t*>(k);
  p.v = static_cast<uint16_t*>(v);
  p.status = status;
  p.B = B;
  p.T = T;
  p.P = P;
  p.units = D / 16;
  p.step_c = tv::kRowThreads % p.units;
  p.step_w = tv::kRowThreads / p.units % (2 * Hkv);
  p.step_t = tv::kRowThreads / p.units / (2 * Hkv);
  p.tokens = tv::kReadTokens;
  while (p.tokens > 1 && T / p.tokens < 4 * tv::device_sm_count()) p.tokens /= 2;
  p.blocks = T / p.tokens + (T % p.tokens != 0);
  const int per = tv::kRowThreads / 32;
  const dim3 grid((unsigned)p.blocks + (status ? (B + per - 1) / per : 0));
  if (grid.x == 0) return TV_OK;
  const bool f16 = cache->dtype == TV_FP16;
  if (cache->format == TV_E4M3)
    return tv::launched(
        f16 ? tv::launch_pdl(tv::read_q8_kernel<true, true>, grid, dim3(tv::kRowThreads), 0, stream, p)
            : tv::launch_pdl(tv::read_q8_kernel<true, false>, grid, dim3(tv::kRowThreads), 0, stream, p));
  return tv::launched(
      f16 ? tv::launch_pdl(tv::read_q8_kernel<false, true>, grid, dim3(tv::kRowThreads), 0, stream, p)
          : tv::launch_pdl(tv::read_q8_kernel<false, false>, grid, dim3(tv::kRowThreads), 0, stream, p));
}

extern "C" tv_status tv_commit_paged_q8(const tv_q8_cache* cache, const int32_t* block_table,
                                        const int32_t* kv_len, const int32_t* path,
                                        const int32_t* accept_len, int B, int N, int P,
                                        int32_t* new_kv_len, int32_t* status, cudaStream_t stream) {
  TV_NVTX_RANGE("tv_commit_paged_q8");
  if (B < 0 || N < 1 || N > TV_MAX_NODES || P < 1) return TV_ERR_INVALID_ARG;
  tv::Q8Cache c;
  const tv_status st = tv::check_q8_cache(cache, &c);
  if (st != TV_OK) return st;
  if ((long long)B * P > 0x7fffffffll || (long long)B * cache->Hkv > 0x7fffffffll ||
      ((long long)P << c.page_shift) > 0x7fffffffll - TV_MAX_NODES)
    return TV_ERR_UNSUPPORTED;
  if (B == 0) return TV_OK;
  if (!block_table || !kv_len || !path || !accept_len || !new_kv_len || !status)
    return TV_ERR_INVALID_ARG;
  if (new_kv_len == kv_len) return TV_ERR_INVALID_ARG;
  return tv::launched(tv::launch_pdl(
      tv::commit_paged_kernel<uint8_t>, dim3((unsigned)(B * cache->Hkv)), dim3(tv::kCommitThreads), 0,
      stream, c.k, c.v, c.ks, c.vs, static_cast<const tv::PagedCache&>(c), block_table, kv_len, path,
      accept_len, N, cache->Hkv, cache->D / 16, P, new_kv_len, status));
}
