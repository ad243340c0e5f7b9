// tv_attn_paged: attention of a ragged batch of new tokens over a paged cache.
#define TV_UNIT 11
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tv_paged.cuh"

namespace tv {
namespace {

struct PagedAttnParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  long long q_token_stride, q_head_stride;
  PagedCache c;
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* kv_len;
  const uint64_t* anc;
  const float* slopes;
  uint16_t* out;
  float* lse;
  int32_t* status;
  int B, T, P, Hq, Hkv, G, W, window;
  float scale, softcap;
};

template <bool F16>
__device__ __forceinline__ float to_f(uint16_t x) {
  if (F16) return __half2float(__ushort_as_half(x));
  return __uint_as_float((uint32_t)x << 16);
}
template <bool F16>
__device__ __forceinline__ uint16_t from_f(float x) {
  if (F16) return __half_as_ushort(__float2half_rn(x));
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// One warp per (token, query head); a lane scores one key of 32, the warp
// then adds the 32 value rows.
template <int D, bool F16>
__global__ void __launch_bounds__(128) attn_simple_kernel(const PagedAttnParams p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const long long items = (long long)p.T * p.Hq;
  if (item >= items) {  // one warp per sequence: its status
    const long long b = item - items;
    if (b >= p.B || !p.status) return;
    int t0, n;
    int bad = !seq_range(p.q_start, (int)b, p.T, t0, n);
    const int L = __ldg(p.kv_len + b);
    if (!bad) bad = L < 0 || (long long)L + n > ((long long)p.P << p.c.page_shift) ||
                    (p.anc && n > 64 * p.W);
    if (!bad) {
      const int lo = p.window > 0 ? max(0, L - p.window + 1) : 0;
      for (int j = (lo >> p.c.page_shift) + lane; n > 0 && ((long long)j << p.c.page_shift) < L + n; j += 32) {
        const int page = __ldg(p.table + (size_t)b * p.P + j);
        bad |= page < 0 || page >= p.c.num_pages;
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) p.status[b] = bad ? TV_ERR_INVALID_ARG : TV_OK;
    return;
  }
  const int t = (int)(item / p.Hq), h = (int)(item % p.Hq), kvh = h / p.G;
  int b = -1, t0 = 0, n = 0;
  for (int x = 0; x < p.B; ++x) {
    int f, m;
    if (seq_range(p.q_start, x, p.T, f, m) && t >= f && t < f + m) {
      b = x;
      t0 = f;
      n = m;
    }
  }
  if (b < 0) return;
  const int L = __ldg(p.kv_len + b), i = t - t0;
  float acc[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) acc[e] = 0.0f;
  float m_run = -INFINITY, l_run = 0.0f;
  const bool bad = L < 0 || (long long)L + n > ((long long)p.P << p.c.page_shift) ||
                   (p.anc && n > 64 * p.W);
  if (!bad) {
    const uint64_t* anc = p.anc ? p.anc + (size_t)t * p.W : nullptr;
    int pos = L + i;
    if (anc) {
      int c = 0;
      for (int w = 0; w < p.W; ++w) c += __popcll(anc[w]);
      pos = L + c - 1;
    }
    const float slope = p.slopes ? p.slopes[h] : 0.0f;
    const uint16_t* q = p.q + t * p.q_token_stride + h * p.q_head_stride;
    const int keys = anc ? L + n : L + i + 1;
    for (int j0 = 0; j0 < keys; j0 += 32) {
      const int j = j0 + lane;
      float x = -INFINITY;
      long long row = -1;
      if (j < keys) {
        int kpos = j;
        bool see = true;
        if (anc && j >= L) {
          const int a = j - L;
          see = (anc[a >> 6] >> (a & 63)) & 1;
          int c = 0;
          for (int w = 0; w <= (a >> 6); ++w)
            c += __popcll(w < (a >> 6) ? anc[w] : anc[w] & (~0ull >> (63 - (a & 63))));
          kpos = L + c - 1;
        }
        if (p.window > 0) see = see && pos - kpos < p.window;
        if (see) {
          const int page = p.table[(size_t)b * p.P + (j >> p.c.page_shift)];
          if (page >= 0 && page < p.c.num_pages) {
            row = page * p.c.page_stride + kvh * p.c.head_stride +
                  (j & ((1 << p.c.page_shift) - 1)) * p.c.row_stride;
            float s = 0.0f;
            for (int e = 0; e < D; ++e) s += to_f<F16>(q[e]) * to_f<F16>(p.k[row + e]);
            x = s * p.scale;
            if (p.softcap > 0.0f) x = p.softcap * tanhf(x / p.softcap);
            x -= slope * (float)(pos - kpos);
          }
        }
      }
      const float m_new = fmaxf(m_run, warp_max(x));
      if (m_new == -INFINITY) continue;
      const float corr = expf(m_run - m_new), w = expf(x - m_new);
      m_run = m_new;
      l_run = l_run * corr + warp_sum(w);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) acc[e] *= corr;
      for (int s = 0; s < 32; ++s) {
        const long long r = __shfl_sync(0xffffffffu, row, s);
        const float ws = __shfl_sync(0xffffffffu, w, s);
        if (r < 0) continue;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[e] += ws * to_f<F16>(p.v[r + 32 * e + lane]);
      }
    }
  }
  const float inv = l_run > 0.0f ? 1.0f / l_run : 0.0f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    p.out[((size_t)t * p.Hq + h) * D + 32 * e + lane] = from_f<F16>(acc[e] * inv);
  if (p.lse && lane == 0)
    p.lse[(size_t)t * p.Hq + h] = bad ? 0.0f : (l_run > 0.0f ? m_run + logf(l_run) : -INFINITY);
}

}  // namespace
}  // namespace tv

extern "C" size_t tv_attn_paged_workspace_size(int max_q, int Hq, int Hkv, int D) {
  (void)max_q, (void)Hq, (void)Hkv, (void)D;
  return 0;
}

extern "C" tv_status tv_attn_paged(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                   const tv_paged_cache* cache, const int32_t* block_table,
                                   const int32_t* q_start, const int32_t* kv_len,
                                   const uint64_t* anc_mask, const float* slopes, int B, int T,
                                   int P, int Hq, int max_q, float scale, float softcap, int window,
                                   void* out, float* lse, int32_t* status, void* workspace,
                                   size_t ws_bytes, cudaStream_t stream) {
  TV_NVTX_RANGE("tv_attn_paged");
  if (B < 0 || T < 0 || P < 1 || Hq < 1 || max_q < 1 || window < 0) return TV_ERR_INVALID_ARG;
  if (!(scale >= 0.0f) || !isfinite(scale) || !(softcap >= 0.0f) || !isfinite(softcap))
    return TV_ERR_INVALID_ARG;
  tv::PagedAttnParams p;
  const tv_status st = tv::check_cache(cache, &p.c);
  if (st != TV_OK) return st;
  const int Hkv = cache->Hkv, D = cache->D;
  if (Hq % Hkv != 0) return TV_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || Hq / Hkv > 128 || B > 4096) return TV_ERR_UNSUPPORTED;
  if (anc_mask && max_q > TV_MAX_NODES) return TV_ERR_UNSUPPORTED;
  if ((long long)T * Hq > 0x7fffffffll || (long long)B * P > 0x7fffffffll ||
      ((long long)P << p.c.page_shift) > 0x7fffffffll)
    return TV_ERR_UNSUPPORTED;
  if (B == 0) return TV_OK;
  if (!block_table || !q_start || !kv_len || (T > 0 && (!q || !out))) return TV_ERR_INVALID_ARG;
  p.q_token_stride = tv::stride_or(q_token_stride, T, 8);
  p.q_head_stride = tv::stride_or(q_head_stride, Hq, 8);
  if (p.q_token_stride < 0 || p.q_head_stride < 0 || ((p.q_token_stride | p.q_head_stride) & 7))
    return TV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15)
    return TV_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(cache->k);
  p.v = static_cast<const uint16_t*>(cache->v);
  p.table = block_table;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.anc = anc_mask;
  p.slopes = slopes;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.status = status;
  p.B = B;
  p.T = T;
  p.P = P;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.W = (max_q + 63) / 64;
  p.window = window;
  p.scale = scale == 0.0f ? 1.0f / sqrtf((float)D) : scale;
  p.softcap = softcap;
  const bool f16 = cache->dtype == TV_FP16;
  auto kernel = D == 128 ? (f16 ? tv::attn_simple_kernel<128, true> : tv::attn_simple_kernel<128, false>)
                         : (f16 ? tv::attn_simple_kernel<64, true> : tv::attn_simple_kernel<64, false>);
  const long long warps = (long long)T * Hq + B;
  if (tv::launch_pdl(kernel, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, stream, p) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return TV_ERR_CUDA;
  }
  return TV_OK;
}
