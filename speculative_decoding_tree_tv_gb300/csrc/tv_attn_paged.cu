// tv_attn_paged: the merge of split units, the plan and the entry point (tv_attn_paged.cuh
// says how the work is shared).
#define TV_UNIT 11
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cfloat>
#include <chrono>

#include "tv_attn_paged.cuh"
#include "tv_quant.cuh"

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
      // (a part whose keys are all hidden: select, do not multiply; 8-bit rows that are no numbers stay)
      if (e == 0.0f && (!p.k_scale || ml[j].x == -INFINITY)) continue;
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

// A cache as the entry point sees it, of 16-bit values or of 8-bit codes.
struct CacheArg {
  PagedCache c;
  void* k;
  void* v;
  int Hkv, D, dtype;
  int format;  // tv_q8_format, or -1
  const uint8_t* k_scale;
  const uint8_t* v_scale;
};

// A cache side: D by rows, heads and pages; a box is 64 dims (of codes: all) of `rows` rows of one
// page and head, for codes that go on as they are (plain) not swizzled.
bool map_cache(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* map, void* base, const CacheArg& a,
               const long long (&stride)[3], const int (&order)[3], int rows, bool plain) {
  const cuuint64_t extent[3] = {(cuuint64_t)1 << a.c.page_shift, (cuuint64_t)a.Hkv, (cuuint64_t)a.c.num_pages};
  const bool codes = a.format >= 0;
  cuuint64_t dims[4] = {(cuuint64_t)a.D}, strides[3];
  cuuint32_t box[4] = {codes ? (cuuint32_t)a.D : 64u};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = extent[order[i]];
    strides[i] = (cuuint64_t)stride[order[i]] * (codes ? 1 : 2);
    box[i + 1] = order[i] == 0 ? (cuuint32_t)rows : 1u;
  }
  return encode(map,
                codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                      : a.dtype == TV_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                4, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                plain                ? CU_TENSOR_MAP_SWIZZLE_NONE
                : codes && a.D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                     : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
PagedPlan paged_plan(int max_q, int Hkv, int G, int D, int B, int T, long long keys, bool q8 = false) {
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
    // 20.7, 19.4 and 18.6 us.  Tiles of 8-bit codes have 128 keys: 4 sequences of 1,500 keys 14, 14 to 15, 18 and 22 us
    // at 3, 4, 6 and 9, one of 10,000 19.0, 18.9, 20.0 and 23.4 us)
    pl.min_share = q8 ? 4 : 6;
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
  // behind 200, 440 and 900 keys 14.3, 14.7 and 20.3 us, split 18.1, 18.9 and 19.5 us.  8-bit caches: decode of 4
  // sequences of 500, 940 and 1,500 keys 10.4, 14.0 and 18.3 us, split 14.5, 16.9 and 17.9 us (at shares of 6; 14 to 15
  // at 4); 2 trees of 64 behind 200, 440 and 900 keys 19.6, 20.4 and 30.9 us, split 25.1, 26.2 and 27.6 us.
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
cudaError_t launch_merge(const PagedPlan& pl, int D, bool f16, const PagedAttnParams& p, cudaStream_t stream) {
  if (D == 128) return f16 ? launch_merge<128, true>(pl, p, stream) : launch_merge<128, false>(pl, p, stream);
  return f16 ? launch_merge<64, true>(pl, p, stream) : launch_merge<64, false>(pl, p, stream);
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


namespace tv {
namespace paged {
namespace {

tv_status cache_arg(const tv_paged_cache* cache, CacheArg* c) {
  const tv_status st = check_cache(cache, &c->c);
  if (st != TV_OK) return st;
  c->k = cache->k;
  c->v = cache->v;
  c->Hkv = cache->Hkv;
  c->D = cache->D;
  c->dtype = cache->dtype;
  c->format = -1;
  return TV_OK;
}

// What an attention call is given, whatever the cache.
struct AttnArgs {
  const void* q;
  int64_t q_token_stride, q_head_stride;
  const int32_t* block_table;
  const int32_t* q_start;
  const int32_t* kv_len;
  const uint64_t* anc_mask;
  const float* slopes;
  int B, T, P, Hq, max_q;
  float scale, softcap;
  int window;
  void* out;
  float* lse;
  int32_t* status;
  void* workspace;
  size_t ws_bytes;
  cudaStream_t stream;
};

// The prefixes that groups of sequences share.
struct PrefixArgs {
  const int32_t* table;
  const int32_t* len;
  const int32_t* group_start;
  int groups, P;
};

// Checks what the host can see; strides of extent-one dimensions are set to ones that fit.
tv_status check_attn(AttnArgs& a, const CacheArg& cache) {
  const int Hkv = cache.Hkv, D = cache.D;
  if (a.B < 0 || a.T < 0 || a.P < 1 || a.Hq < 1 || a.max_q < 1 || a.window < 0) return TV_ERR_INVALID_ARG;
  if (!(a.scale >= 0.0f) || !isfinite(a.scale) || !(a.softcap >= 0.0f) || !isfinite(a.softcap))
    return TV_ERR_INVALID_ARG;
  if (a.Hq % Hkv != 0) return TV_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || a.Hq / Hkv > 128 || a.B > kMaxSeqs) return TV_ERR_UNSUPPORTED;
  if (a.anc_mask && a.max_q > TV_MAX_NODES) return TV_ERR_UNSUPPORTED;
  if ((long long)a.T * a.Hq > 0x7fffffffll || (long long)a.B * a.P > 0x7fffffffll ||
      ((long long)a.P << cache.c.page_shift) > 0x7fffffffll - 512)
    return TV_ERR_UNSUPPORTED;
  if (a.B == 0) return TV_OK;
  if (!a.block_table || !a.q_start || !a.kv_len || (a.T > 0 && (!a.q || !a.out))) return TV_ERR_INVALID_ARG;
  a.q_head_stride = stride_or(a.q_head_stride, a.Hq, D);
  a.q_token_stride = stride_or(a.q_token_stride, a.T, a.Hq * a.q_head_stride);
  if (a.q_token_stride < 0 || a.q_head_stride < 0 || ((a.q_token_stride | a.q_head_stride) & 7))
    return TV_ERR_INVALID_ARG;
  if (a.q_head_stride == 0 || a.q_token_stride == 0) return TV_ERR_UNSUPPORTED;
  if (a.Hq == 1) a.q_head_stride = a.q_token_stride;
  if (a.q_token_stride % a.q_head_stride != 0 || a.q_token_stride >= (1ll << 39))
    return TV_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.out)) & 15)
    return TV_ERR_INVALID_ARG;
  return TV_OK;
}

// One pass over a paged cache: a plan, the kernels' arguments and tensor maps.
struct Pass {
  PagedPlan pl;
  PagedAttnParams p;
  CUtensorMap tmQ, tmK, tmV;
  bool bias;
};

// chunk: the tokens of a sequence, as far as the host knows them.
tv_status make_pass(const AttnArgs& a, const CacheArg& cache, const PagedPlan& pl, int chunk, uint8_t* ws,
                    Pass* out) {
  out->pl = pl;
  PagedAttnParams& p = out->p;
  p = PagedAttnParams{};
  const PagedCache& c = cache.c;
  const int Hkv = cache.Hkv, D = cache.D;
  const bool q8 = cache.format >= 0, f16 = cache.dtype == TV_FP16;
  p.q_head_stride = a.q_head_stride;
  p.q_token_stride = a.q_token_stride;
  const long long extent[3] = {1ll << c.page_shift, Hkv, c.num_pages};
  long long stride[3] = {c.row_stride, c.head_stride, c.page_stride};
  int order[3];
  if (!order_strides(extent, stride, D, order)) return TV_ERR_UNSUPPORTED;
  auto encode = tensor_map_encoder();
  if (!encode) return TV_ERR_CUDA;
  CUtensorMap &tmQ = out->tmQ, &tmK = out->tmK, &tmV = out->tmV;
  const int rows = min(1 << c.page_shift, pl.small && !pl.whole && !q8 ? 64 : 128);
  const bool plain = q8 && !pl.small;  // (codes on their way to 16-bit tiles)
  if (!map_cache(encode, &tmK, cache.k, cache, stride, order, rows, plain) ||
      !map_cache(encode, &tmV, cache.v, cache, stride, order, rows, plain))
    return TV_ERR_INVALID_ARG;
  if (!pl.small && a.T > 0) {
    // q as [tokens][heads][D]; a box is 64 dims of the group's heads of nb tokens
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
    const cuuint64_t strides[2] = {(cuuint64_t)p.q_head_stride * 2, (cuuint64_t)p.q_token_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)(a.Hq / Hkv), (cuuint32_t)pl.nb}, estr[3] = {1, 1, 1};
    if (encode(&tmQ, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
               3, const_cast<void*>(a.q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return TV_ERR_INVALID_ARG;
  } else {
    tmQ = tmK;  // not read
  }
  p.part = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.part_bytes);
  p.desc = reinterpret_cast<int4*>(ws + pl.part_bytes + pl.ml_bytes);
  p.late = reinterpret_cast<Late*>(ws + pl.part_bytes + pl.ml_bytes + pl.desc_bytes);
  p.any_late = reinterpret_cast<unsigned long long*>(p.late + pl.ctas);
  p.wait_limit = wait_limit();
  p.q = static_cast<const uint16_t*>(a.q);
  p.k_scale = cache.k_scale;
  p.v_scale = cache.v_scale;
  p.f16 = f16;
  p.e4m3 = cache.format == TV_E4M3;
  p.table = a.block_table;
  p.q_start = a.q_start;
  p.kv_len = a.kv_len;
  p.anc = a.anc_mask;
  p.slopes = a.slopes;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.status = a.status;
  p.B = a.B;
  p.T = a.T;
  p.P = a.P;
  p.Hq = a.Hq;
  p.Hkv = Hkv;
  p.G = a.Hq / Hkv;
  p.W = (a.max_q + 63) / 64;
  p.window = a.window;
  p.num_pages = c.num_pages;
  p.page_shift = c.page_shift;
  for (int i = 0; i < 3; ++i) {
    if (order[i] == 0) p.row_dim = i + 1;
    if (order[i] == 1) p.head_dim = i + 1;
  }
  p.tq = pl.tq;
  p.ctas = pl.ctas;
  p.min_share = pl.min_share;
  p.share_lanes = 0;  // (a lane per query tile of the largest chunk, where the kernels' threads suffice)
  while (p.share_lanes < 5 && (pl.tq << p.share_lanes) < chunk && (a.B << (p.share_lanes + 1)) <= 192)
    ++p.share_lanes;
  p.whole = pl.whole;
  p.unit_cost = kUnitCost;
  p.out_sectors = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
  p.merge = pl.merge;
  p.ready = reinterpret_cast<unsigned long long*>(ws + pl.part_bytes + pl.ml_bytes + pl.desc_bytes +
                                                  pl.late_bytes);
  p.token = next_token();
  const float sc = a.scale == 0.0f ? 1.0f / sqrtf((float)D) : a.scale;
  p.scale_log2 = sc * kLog2e;
  // (caps at the ends of the 32-bit range: a product of 0 has a score of 0 all the same)
  p.softcap_log2 = fminf(a.softcap * kLog2e, FLT_MAX);
  p.cap_in = a.softcap > 0.0f ? fminf(sc / a.softcap, 1e30f) : 0.0f;
  // The cubic's coefficients for products as they are, in the log2 domain.  For a large cap the higher
  // ones fade to 0 and nearly every score is taken by it: the function for the others is off by
  // some 2^-23 of the cap, not of the score.  For caps below 1e-5 of the scale, whose coefficients would
  // leave the 32-bit range, that is small, and it takes all.
  p.cap_top = -1.0f;
  for (float& c : p.cap_q) c = 0.0f;
  if (p.cap_in <= 1e5f) {
    const float a2 = p.cap_in * p.cap_in;
    float f = p.scale_log2;
    for (int i = 0; i < 4; ++i, f *= a2) p.cap_q[i] = f * kTanhC[i];
    p.cap_top = fminf(kTanhSmall * kTanhSmall / a2, 1e36f);  // (squares stay finite)
  }
  out->bias = a.slopes || (a.anc_mask && a.window > 0 && a.window < 64 * p.W);
  return TV_OK;
}

cudaError_t launch_pass(const Pass& s, const CacheArg& cache, cudaStream_t stream) {
  const PagedPlan& pl = s.pl;
  const PagedAttnParams& p = s.p;
  const int D = cache.D;
  const bool f16 = cache.dtype == TV_FP16, mod = s.bias || p.softcap_log2 > 0.0f;
  cudaError_t e;
  if (cache.format >= 0 && !pl.small)
    e = launch_tc_q8(pl, D, f16, s.bias, s.tmQ, s.tmK, s.tmV, p, stream);
  else if (cache.format >= 0)
    e = cache.format == TV_E4M3 ? launch_rows_e4m3(pl, D, mod, s.tmK, s.tmV, p, stream)
                                : launch_rows_int8(pl, D, mod, s.tmK, s.tmV, p, stream);
  else if (p.groups > 0)
    return launch_prefix(pl, D, f16, s.bias, s.tmQ, s.tmK, s.tmV, p, stream);
  else if (pl.small)
    e = launch_rows(pl, D, f16, mod, s.tmK, s.tmV, p, stream);
  else
    e = launch_tc(pl, D, f16, s.bias, s.tmQ, s.tmK, s.tmV, p, stream);
  if (e == cudaSuccess && pl.merge) e = launch_merge(pl, D, f16, p, stream);
  return e;
}

tv_status launched(cudaError_t e) {
  if (e == cudaSuccess) return TV_OK;
  (void)cudaGetLastError();
  return TV_ERR_CUDA;
}

tv_status attend(AttnArgs a, const CacheArg& cache) {
  tv_status st = check_attn(a, cache);
  if (st != TV_OK || a.B == 0) return st;
  const PagedPlan pl = paged_plan(a.max_q, cache.Hkv, a.Hq / cache.Hkv, cache.D, a.B, a.T,
                                  (long long)a.P << cache.c.page_shift, cache.format >= 0);
  if (!a.workspace || a.ws_bytes < pl.bytes() || (reinterpret_cast<uintptr_t>(a.workspace) & 255))
    return TV_ERR_WORKSPACE;
  Pass s;
  st = make_pass(a, cache, pl, a.max_q, static_cast<uint8_t*>(a.workspace), &s);
  return st != TV_OK ? st : launched(launch_pass(s, cache, a.stream));
}

// The plan of a call with shared prefixes, and where the rows of units that are not split lie behind its workspace.
struct PrefixPlan {
  PagedPlan pl;
  size_t raw, raw_ml, src, bytes;
};
PrefixPlan prefix_plan(int T, int groups, int Hq, int Hkv, int D, int B, long long keys) {
  PrefixPlan f;
  PagedPlan& pl = f.pl;
  pl = paged_plan(TV_MAX_NODES, Hkv, Hq / Hkv, D, B, T, 1ll << 40);  // (the tcgen05 kernel's)
  // (units of prefixes and of sequences)
  pl.whole = keys <= kWholeTcKeys && (long long)Hkv * (2ll * (T / pl.tq) + groups + B) <= device_sm_count();
  if (pl.whole) pl.min_share = 1;
  pl.merge = true;  // split units' rows are left in slots
  f.raw = pl.bytes();
  f.raw_ml = f.raw + align_up(2 * (size_t)T * Hq * D * 4, 256);
  f.src = f.raw_ml + align_up(2 * (size_t)T * Hq * 8, 256);
  f.bytes = f.src + align_up(2 * (size_t)T * Hkv * 16, 256);
  return f;
}

tv_status attend_prefix(AttnArgs a, const PrefixArgs& f, const CacheArg& cache) {
  if (f.groups < 0 || f.P < 1) return TV_ERR_INVALID_ARG;
  tv_status st = check_attn(a, cache);
  if (st != TV_OK) return st;
  const int shift = cache.c.page_shift;
  if (f.groups > kMaxSeqs || (long long)f.groups * f.P > 0x7fffffffll ||
      ((long long)a.P + f.P) << shift > 0x7fffffffll - 512)
    return TV_ERR_UNSUPPORTED;
  if (a.B == 0) return TV_OK;
  if (f.groups == 0) return attend(a, cache);
  if (!f.table || !f.len || !f.group_start) return TV_ERR_INVALID_ARG;
  const PrefixPlan pl = prefix_plan(a.T, f.groups, a.Hq, cache.Hkv, cache.D, a.B,
                                    (long long)(a.P > f.P ? a.P : f.P) << shift);
  if (!a.workspace || a.ws_bytes < pl.bytes || (reinterpret_cast<uintptr_t>(a.workspace) & 255))
    return TV_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  Pass s;
  const int per_group = a.T / f.groups + 1;  // (the host knows no groups' lengths)
  if ((st = make_pass(a, cache, pl.pl, per_group > a.max_q ? per_group : a.max_q, ws, &s)) != TV_OK) return st;
  PagedAttnParams& p = s.p;
  p.groups = f.groups;
  // (small own units, of decode tokens, are not worth their sequences' weight beside a prefix's tiles of 256 rows: 64
  // of them behind 8,000 rows 59.8, 46.6, 51.2 and 54.4 us at 0 to 3; trees of 16 to 48 nodes behind four prefixes 36.7,
  // 31.7, 28.2 and 27.6 us)
  p.unit_cost = a.max_q * (a.Hq / cache.Hkv) <= 16 ? 1 : kUnitCost;
  p.prefix_P = f.P;
  p.group_start = f.group_start;
  p.prefix_len = f.len;
  p.prefix_table = f.table;
  p.raw = reinterpret_cast<float*>(ws + pl.raw);
  p.raw_ml = reinterpret_cast<float2*>(ws + pl.raw_ml);
  p.src = reinterpret_cast<int4*>(ws + pl.src);
  while (p.share_lanes > 0 && (f.groups + a.B) << p.share_lanes > 384) --p.share_lanes;  // (a thread each at most)
  return launched(launch_pass(s, cache, a.stream));
}

}  // namespace
}  // namespace paged
}  // namespace tv

extern "C" tv_status tv_attn_paged(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                   const tv_paged_cache* cache, const int32_t* block_table,
                                   const int32_t* q_start, const int32_t* kv_len,
                                   const uint64_t* anc_mask, const float* slopes, int B, int T,
                                   int P, int Hq, int max_q, float scale, float softcap, int window,
                                   void* out, float* lse, int32_t* status, void* workspace,
                                   size_t ws_bytes, cudaStream_t stream) {
  TV_NVTX_RANGE("tv_attn_paged");
  tv::paged::CacheArg c{};
  const tv_status st = tv::paged::cache_arg(cache, &c);
  if (st != TV_OK) return st;
  return tv::paged::attend({q, q_token_stride, q_head_stride, block_table, q_start, kv_len, anc_mask, slopes, B, T, P,
                            Hq, max_q, scale, softcap, window, out, lse, status, workspace, ws_bytes, stream}, c);
}

extern "C" size_t tv_attn_paged_q8_workspace_size(int max_q, int Hq, int Hkv, int D) {
  if (max_q < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq / Hkv > 128 || (D != 64 && D != 128))
    return 0;
  return tv::paged::paged_plan(max_q, Hkv, Hq / Hkv, D, 0, 0, 0).bytes();
}

extern "C" tv_status tv_attn_paged_q8(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                      const tv_q8_cache* cache, const int32_t* block_table,
                                      const int32_t* q_start, const int32_t* kv_len,
                                      const uint64_t* anc_mask, const float* slopes, int B, int T,
                                      int P, int Hq, int max_q, float scale, float softcap, int window,
                                      void* out, float* lse, int32_t* status, void* workspace,
                                      size_t ws_bytes, cudaStream_t stream) {
  TV_NVTX_RANGE("tv_attn_paged_q8");
  tv::paged::CacheArg c{};
  tv::Q8Cache rows;
  const tv_status st = tv::check_q8_cache(cache, &rows);
  if (st != TV_OK) return st;
  c.c = rows;
  c.k = cache->k;
  c.v = cache->v;
  c.Hkv = cache->Hkv;
  c.D = cache->D;
  c.dtype = cache->dtype;
  c.format = cache->format;
  c.k_scale = cache->k_scale;
  c.v_scale = cache->v_scale;
  return tv::paged::attend({q, q_token_stride, q_head_stride, block_table, q_start, kv_len, anc_mask, slopes, B, T, P,
                            Hq, max_q, scale, softcap, window, out, lse, status, workspace, ws_bytes, stream}, c);
}

extern "C" size_t tv_attn_paged_prefix_workspace_size(int max_q, int T, int groups, int Hq, int Hkv, int D) {
  if (max_q < 1 || T < 0 || groups < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq / Hkv > 128 ||
      (D != 64 && D != 128) || (long long)T * Hq > 0x7fffffffll)
    return 0;
  if (groups == 0) return tv_attn_paged_workspace_size(max_q, Hq, Hkv, D);
  return tv::paged::prefix_plan(T, groups, Hq, Hkv, D, 0, 0).bytes;
}

extern "C" tv_status tv_attn_paged_prefix(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, const tv_paged_cache* cache,
    const int32_t* prefix_table, const int32_t* prefix_len, const int32_t* group_start, int groups, int prefix_P,
    const int32_t* block_table, const int32_t* q_start, const int32_t* kv_len, const uint64_t* anc_mask,
    const float* slopes, int B, int T, int P, int Hq, int max_q, float scale, float softcap, int window,
    void* out, float* lse, int32_t* status, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  TV_NVTX_RANGE("tv_attn_paged_prefix");
  tv::paged::CacheArg c{};
  const tv_status st = tv::paged::cache_arg(cache, &c);
  if (st != TV_OK) return st;
  return tv::paged::attend_prefix(
      {q, q_token_stride, q_head_stride, block_table, q_start, kv_len, anc_mask, slopes, B, T, P, Hq, max_q, scale,
       softcap, window, out, lse, status, workspace, ws_bytes, stream},
      {prefix_table, prefix_len, group_start, groups, prefix_P}, c);
}
