// tv_attn_paged: the merge of split units, the plan and the entry point (tv_attn_paged.cuh
// says how the work is shared).
#define TV_UNIT 11
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cfloat>
#include <chrono>

#include "tv_attn_paged.cuh"

namespace tv {
namespace paged {
namespace {

// Joins the parts of split units.  Block (i, y): the unit that share i ends inside, if any; its
// parts are slots 2 i + 1, 2 (i + 1), 2 (i + 2), ..  Rows of the tcgen05 kernel (TC) lie chunk by
// chunk ([D / 4][256] of four floats, the order its threads write), small units' row by row.
constexpr int kMergeThreads = 256, kMergeBatch = 2;

// The merge's blocks also write the sequences' status: it costs nothing here, while a scan of
// a long block table held up the attention kernel's first tiles by some 1.5 us.
__device__ __forceinline__ void merge_status(const PagedAttnParams& p) {
  if (!p.status) return;
  for (int b = blockIdx.y * gridDim.x + blockIdx.x; b < p.B; b += gridDim.x * gridDim.y) {
    const bool late = is_late(p, b, threadIdx.x, kMergeThreads);
    const bool bad = !seq_ok(p, b, threadIdx.x, kMergeThreads);
    const int any_late = __syncthreads_or(late), any_bad = __syncthreads_or(bad);
    if (threadIdx.x == 0)
      p.status[b] = any_late ? TV_ERR_TIMEOUT : any_bad ? TV_ERR_INVALID_ARG : TV_OK;
  }
}

// A thread joins kC chunks (of four floats) of one row, all its loads of a batch of parts
// in flight.
template <int D, bool F16, bool TC>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedAttnParams p, int nb) {
  constexpr int kChunks = D / 4, kRows = TC ? 256 : 16;
  constexpr int kC = TC ? 4 : kChunks * kRows / kMergeThreads;  // a small unit: one block
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.x;
  const int4 d = p.desc[i];
  merge_status(p);
  if (d.w == 0) return;
  const int row = TC ? threadIdx.x : threadIdx.x / (kChunks / kC);
  const int c0 = TC ? blockIdx.y * kC : (threadIdx.x % (kChunks / kC)) * kC;
  // a row block of the tcgen05 kernel holds nb tokens in its 128 rows
  const int rl = TC ? row & 127 : row, tr = rl / p.G;
  const int tl = (TC ? (row >> 7) * nb : 0) + tr;
  if (tl >= d.y || (TC && tr >= nb)) return;
  const int h = d.z * p.G + rl - tr * p.G;
  const size_t oidx = (size_t)(d.x + tl) * p.Hq + h;
  if (!TV_CHECK(oidx < (size_t)p.T * p.Hq)) return;
  float M = -INFINITY, l = 0.0f;
  float4 a[kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) a[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < d.w; j0 += kMergeBatch) {
    float2 ml[kMergeBatch];
    float4 v[kMergeBatch][kC];
#pragma unroll
    for (int j = 0; j < kMergeBatch; ++j) {
      ml[j] = make_float2(-INFINITY, 0.0f);
      if (j0 + j < d.w && TV_CHECK(i + j0 + j < (int)gridDim.x)) {
        const size_t slot = j0 + j == 0 ? 2 * i + 1 : 2 * (i + j0 + j);
        ml[j] = p.part_ml[slot * kRows + row];
        const float4* src = reinterpret_cast<const float4*>(p.part) + slot * kRows * kChunks;
#pragma unroll
        for (int c = 0; c < kC; ++c)
          v[j][c] = src[TC ? (c0 + c) * kRows + row : row * kChunks + c0 + c];
      }
    }
    float mx = M;
#pragma unroll
    for (int j = 0; j < kMergeBatch; ++j) mx = fmaxf(mx, ml[j].x);
    // (maxima leave a NaN out, sums carry it: 0 times NaN is NaN)
    const float f = M == -INFINITY ? 0.0f : ex2(M - mx);
    M = mx;
    l *= f;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      a[c].x *= f;
      a[c].y *= f;
      a[c].z *= f;
      a[c].w *= f;
    }
#pragma unroll
    for (int j = 0; j < kMergeBatch; ++j) {
      const float e = ml[j].x == -INFINITY ? 0.0f : ex2(ml[j].x - M);
      l = fmaf(e, ml[j].y, l);
      if (e == 0.0f) continue;  // (a part whose keys are all hidden: select, do not multiply)
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        a[c].x = fmaf(e, v[j][c].x, a[c].x);
        a[c].y = fmaf(e, v[j][c].y, a[c].y);
        a[c].z = fmaf(e, v[j][c].z, a[c].z);
        a[c].w = fmaf(e, v[j][c].w, a[c].w);
      }
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint2* out = reinterpret_cast<uint2*>(p.out + oidx * D) + c0;
#pragma unroll
  for (int c = 0; c < kC; ++c)
    out[c] = make_uint2(pack2<F16>(a[c].x * inv, a[c].y * inv), pack2<F16>(a[c].z * inv, a[c].w * inv));
  if (c0 == 0 && p.lse) p.lse[oidx] = l == 0.0f ? -INFINITY : (M + log2f(l)) * kLn2;
}

// --------------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      return nullptr;
    }
    f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    fn.store(f, std::memory_order_release);
  }
  return f;
}

// The outer dimensions of a tensor map in the order of their strides, which a map wants
// to be multiples of one another; a dimension of extent one takes a stride that fits.
// order[i] = which dimension comes i-th.
bool order_strides(const long long (&extent)[3], long long (&stride)[3], int D, int (&order)[3]) {
  long long most = D;
  for (int i = 0; i < 3; ++i)
    if (extent[i] > 1) most = stride[i] > most ? stride[i] : most;
  for (int i = 0; i < 3; ++i)
    if (extent[i] == 1) stride[i] = most;
  for (int i = 0; i < 3; ++i) order[i] = i;
  for (int i = 1; i < 3; ++i)
    for (int j = i; j > 0 && stride[order[j]] < stride[order[j - 1]]; --j) {
      const int x = order[j];
      order[j] = order[j - 1];
      order[j - 1] = x;
    }
  const long long a = stride[order[0]], b = stride[order[1]], c = stride[order[2]];
  return a > 0 && a % 8 == 0 && b % a == 0 && c % b == 0 && c < (1ll << 39);
}

// A cache side: D by rows, heads and pages; a box is 64 dims of `rows` rows of one
// page and head.
bool map_cache(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* map, void* base,
               const tv_paged_cache* cache, const long long (&stride)[3], const int (&order)[3],
               int rows) {
  const cuuint64_t extent[3] = {(cuuint64_t)cache->page_size, (cuuint64_t)cache->Hkv,
                                (cuuint64_t)cache->num_pages};
  cuuint64_t dims[4] = {(cuuint64_t)cache->D}, strides[3];
  cuuint32_t box[4] = {64};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = extent[order[i]];
    strides[i] = (cuuint64_t)stride[order[i]] * 2;
    box[i + 1] = order[i] == 0 ? (cuuint32_t)rows : 1u;
  }
  return encode(map, cache->dtype == TV_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                4, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr long long kWholeRowsKeys = 960, kWholeTcKeys = 512;

// A mark of its own for every call, which nothing that a workspace held before is taken for: counted
// on from a start that differs from process to process.
unsigned long long next_token() {
  static std::atomic<unsigned long long> token{
      ((unsigned long long)std::chrono::system_clock::now().time_since_epoch().count() << 20) ^
      (unsigned long long)reinterpret_cast<uintptr_t>(&tensor_map_encoder)};
  return token.fetch_add(1, std::memory_order_relaxed) | 1ull << 63;
}


// Limits of the kernels' waits, less the regular one (so that 0 is that); by device.
std::atomic<long long> g_wait_limit[kMaxDevicesCached];
long long wait_limit() {
  const int dev = current_device();
  return kWaitLimitCycles + (dev >= 0 && dev < kMaxDevicesCached ? g_wait_limit[dev].load() : 0);
}

// Which kernel runs, by the rows of the largest unit.
PagedPlan paged_plan(int max_q, int Hkv, int G, int D, int B, int T, long long keys) {
  PagedPlan pl;
  const long long rows = (long long)max_q * G;
  // 64 decode sequences of 512 to 8,192 keys, 8 kv heads: 4 rows a unit 186 us here and 198 us on the
  // tcgen05 kernel (D 64: 102 and 149 us), 16 rows 171 and 180 us; 32 rows took 430 us with two row
  // tiles a warp here (its registers spill) and 185 us there.
  pl.small = rows <= 16;
  if (pl.small) {
    pl.rows = 16;
    pl.nb = pl.tq = (rows <= 8 ? 8 : 16) / G;
    pl.ctas = 2 * device_sm_count();
    // (4 sequences of 1,000 keys 11.4, 12.0 and 13.9 us at 5, 6 and 9; one of 10,000, whose parts are many,
    // 20.7, 19.4 and 18.6 us)
    pl.min_share = 6;
  } else {
    pl.rows = 256;
    pl.nb = 128 / G;
    pl.tq = 2 * pl.nb;
    pl.ctas = device_sm_count();
    // (a unit's fixed cost and one tile; one tree of 64 behind 2,000 keys 21.2, 22.2 and 23.1 us at 4, 5 and 6)
    pl.min_share = 4;
  }
  // Units short enough for a CTA each (keys: the most that the block table has room for, as the
  // host knows no lengths; short sequences in a wide table are split) are not split, and
  // the merge is not launched: decode of 4 sequences of 500, 1,000 and 1,500 keys 8.9, 12.6 and 16.2 us,
  // split 11.2, 11.8 and 12.2 us (D 64: 1,000 keys 9.9 and 10.5 us; 16 rows: 13.5 and 14.1 us); 2 trees of 64
  // behind 200, 440 and 900 keys 14.3, 14.7 and 20.3 us, split 18.1, 18.9 and 19.5 us.
  pl.whole = keys <= (pl.small ? kWholeRowsKeys : kWholeTcKeys) &&
             (long long)Hkv * (T / pl.tq + B) <= device_sm_count();
  if (pl.whole) pl.min_share = 1;
  // At least Hkv ceil(T / tokens of a unit) units: with two CTAs a unit or fewer the CTAs join
  // split units themselves (16 trees of 64 nodes 77 us, 82 us with the merge kernel; one tree of 64
  // behind 32,000 keys, 19 CTAs a unit, 86 and 47 us).  Small units always take the merge kernel:
  // joining in the CTAs took 199 instead of 187 us for a decode of 64.
  const int unit_tokens = pl.tq < max_q ? pl.tq : max_q;
  pl.merge = !pl.whole &&
             (pl.small || 2 * Hkv * (((long long)T + unit_tokens - 1) / unit_tokens) < pl.ctas);
  const size_t r = 2 * (size_t)pl.ctas * pl.rows;
  pl.part_bytes = align_up(r * D * 4, 256);
  pl.ml_bytes = align_up(r * 8, 256);
  pl.desc_bytes = align_up((size_t)pl.ctas * 16, 256);
  pl.late_bytes = align_up((size_t)pl.ctas * sizeof(Late) + 8, 256);
  pl.ready_bytes = align_up((size_t)pl.ctas * 64, 256);
  return pl;
}

template <int D, bool F16>
cudaError_t launch_merge(const PagedPlan& pl, const PagedAttnParams& p, cudaStream_t stream) {
  if (pl.small)
    return launch_pdl(paged_merge_kernel<D, F16, false>, dim3(pl.ctas, 1), dim3(kMergeThreads), 0,
                      stream, p, pl.nb);
  return launch_pdl(paged_merge_kernel<D, F16, true>, dim3(pl.ctas, D / 16), dim3(kMergeThreads), 0,
                    stream, p, pl.nb);
}

}  // namespace

void set_wait_limit(long long cycles) {
  const int dev = current_device();
  if (dev >= 0 && dev < kMaxDevicesCached) g_wait_limit[dev] = cycles - kWaitLimitCycles;
}

}  // namespace paged
}  // namespace tv

extern "C" size_t tv_attn_paged_workspace_size(int max_q, int Hq, int Hkv, int D) {
  if (max_q < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq / Hkv > 128 || (D != 64 && D != 128))
    return 0;
  return tv::paged::paged_plan(max_q, Hkv, Hq / Hkv, D, 0, 0, 0).bytes();  // (whatever B, T and keys are)
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
  tv::paged::PagedAttnParams p;
  tv::PagedCache c;
  const tv_status st = tv::check_cache(cache, &c);
  if (st != TV_OK) return st;
  const int Hkv = cache->Hkv, D = cache->D;
  if (Hq % Hkv != 0) return TV_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || Hq / Hkv > 128 || B > tv::paged::kMaxSeqs) return TV_ERR_UNSUPPORTED;
  if (anc_mask && max_q > TV_MAX_NODES) return TV_ERR_UNSUPPORTED;
  if ((long long)T * Hq > 0x7fffffffll || (long long)B * P > 0x7fffffffll ||
      ((long long)P << c.page_shift) > 0x7fffffffll - 512)
    return TV_ERR_UNSUPPORTED;
  if (B == 0) return TV_OK;
  if (!block_table || !q_start || !kv_len || (T > 0 && (!q || !out))) return TV_ERR_INVALID_ARG;
  p.q_head_stride = tv::stride_or(q_head_stride, Hq, D);
  p.q_token_stride = tv::stride_or(q_token_stride, T, Hq * p.q_head_stride);
  if (p.q_token_stride < 0 || p.q_head_stride < 0 || ((p.q_token_stride | p.q_head_stride) & 7))
    return TV_ERR_INVALID_ARG;
  if (p.q_head_stride == 0 || p.q_token_stride == 0) return TV_ERR_UNSUPPORTED;
  if (Hq == 1) p.q_head_stride = p.q_token_stride;
  if (p.q_token_stride % p.q_head_stride != 0 || p.q_token_stride >= (1ll << 39))
    return TV_ERR_UNSUPPORTED;
  const long long extent[3] = {cache->page_size, Hkv, cache->num_pages};
  long long stride[3] = {c.row_stride, c.head_stride, c.page_stride};
  int order[3];
  if (!tv::paged::order_strides(extent, stride, D, order)) return TV_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15)
    return TV_ERR_INVALID_ARG;
  const tv::paged::PagedPlan pl =
      tv::paged::paged_plan(max_q, Hkv, Hq / Hkv, D, B, T, (long long)P << c.page_shift);
  if (!workspace || ws_bytes < pl.bytes() || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return TV_ERR_WORKSPACE;
  auto encode = tv::paged::tensor_map_encoder();
  if (!encode) return TV_ERR_CUDA;
  CUtensorMap tmQ, tmK, tmV;
  const int rows = min(cache->page_size, pl.small && !pl.whole ? 64 : 128);
  if (!tv::paged::map_cache(encode, &tmK, cache->k, cache, stride, order, rows) ||
      !tv::paged::map_cache(encode, &tmV, cache->v, cache, stride, order, rows))
    return TV_ERR_INVALID_ARG;
  if (!pl.small && T > 0) {
    // q as [tokens][heads][D]; a box is 64 dims of the group's heads of nb tokens
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)p.q_head_stride * 2, (cuuint64_t)p.q_token_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)(Hq / Hkv), (cuuint32_t)pl.nb}, estr[3] = {1, 1, 1};
    if (encode(&tmQ, cache->dtype == TV_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
               3, const_cast<void*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return TV_ERR_INVALID_ARG;
  } else {
    tmQ = tmK;  // not read
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.part_bytes);
  p.desc = reinterpret_cast<int4*>(ws + pl.part_bytes + pl.ml_bytes);
  p.late = reinterpret_cast<tv::paged::Late*>(ws + pl.part_bytes + pl.ml_bytes + pl.desc_bytes);
  p.any_late = reinterpret_cast<unsigned long long*>(p.late + pl.ctas);
  p.wait_limit = tv::paged::wait_limit();
  p.q = static_cast<const uint16_t*>(q);
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
  p.num_pages = c.num_pages;
  p.page_shift = c.page_shift;
  for (int i = 0; i < 3; ++i) {
    if (order[i] == 0) p.row_dim = i + 1;
    if (order[i] == 1) p.head_dim = i + 1;
  }
  p.tq = pl.tq;
  p.min_share = pl.min_share;
  p.share_lanes = 0;  // (a lane per query tile of the largest chunk, where the kernels' threads suffice)
  while (p.share_lanes < 5 && (pl.tq << p.share_lanes) < max_q && (B << (p.share_lanes + 1)) <= 192)
    ++p.share_lanes;
  p.whole = pl.whole;
  p.out_sectors = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  p.merge = pl.merge;
  p.ready = reinterpret_cast<unsigned long long*>(ws + pl.part_bytes + pl.ml_bytes + pl.desc_bytes +
                                                  pl.late_bytes);
  p.token = tv::paged::next_token();
  const float sc = scale == 0.0f ? 1.0f / sqrtf((float)D) : scale;
  p.scale_log2 = sc * tv::paged::kLog2e;
  // (caps at the ends of the 32-bit range: a product of 0 has a score of 0 all the same)
  p.softcap_log2 = fminf(softcap * tv::paged::kLog2e, FLT_MAX);
  p.cap_in = softcap > 0.0f ? fminf(sc / softcap, 1e30f) : 0.0f;
  // The cubic's coefficients for products as they are, in the log2 domain.  For a large cap the higher
  // ones fade to 0 and nearly every score is taken by it: the function for the others is off by
  // some 2^-23 of the cap, not of the score.  For caps below 1e-5 of the scale, whose coefficients would
  // leave the 32-bit range, that is small, and it takes all.
  p.cap_top = -1.0f;
  for (float& c : p.cap_q) c = 0.0f;
  if (p.cap_in <= 1e5f) {
    const float a2 = p.cap_in * p.cap_in;
    float f = p.scale_log2;
    for (int i = 0; i < 4; ++i, f *= a2) p.cap_q[i] = f * tv::paged::kTanhC[i];
    p.cap_top = fminf(tv::paged::kTanhSmall * tv::paged::kTanhSmall / a2, 1e36f);  // (squares stay finite)
  }
  const bool bias = slopes || (anc_mask && window > 0 && window < 64 * p.W);
  const bool f16 = cache->dtype == TV_FP16;
  cudaError_t e = pl.small ? tv::paged::launch_rows(pl, D, f16, bias || softcap > 0.0f, tmK, tmV, p, stream)
                        : tv::paged::launch_tc(pl, D, f16, bias, tmQ, tmK, tmV, p, stream);
  if (e == cudaSuccess && pl.merge)
    e = D == 128 ? (f16 ? tv::paged::launch_merge<128, true>(pl, p, stream)
                        : tv::paged::launch_merge<128, false>(pl, p, stream))
                 : (f16 ? tv::paged::launch_merge<64, true>(pl, p, stream)
                        : tv::paged::launch_merge<64, false>(pl, p, stream));
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return TV_ERR_CUDA;
  }
  return TV_OK;
}
