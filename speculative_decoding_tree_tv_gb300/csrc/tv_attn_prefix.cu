// tv_attn_paged_prefix's kernels: paged_tc_kernel over one line of prefixes and sequences, and the kernel that
// joins their rows.
//
// A prefix's unit holds up to 256 rows of its group's tokens, whatever sequences they are of, so its keys are
// read once for them; a sequence's own units follow on the same line, and the line is cut into equal shares as
// always: prefixes and own rows are worked on side by side in one launch.  Small own units (decode tokens)
// stay on this kernel too: it streams their pages at 94 % of the small kernel's rate (64 decode
// sequences 198 and 186 us), and a launch of their own waits for the prefixes' one (52 for 46.5 us, 64 sequences behind
// 8,000 rows).  As two passes, own rows behind the prefixes' joined ones, that took 71 us.
//
// Bound by latency: a prefix has few bytes when it is read once.  64 decode tokens behind 8,000 rows with 30 to 600 of
// their own take 46 us (floor 16): the share is known at 3.4 us, the first product issued at 8, the first tile done at
// 12.5 (its code is new to the SM), then 1.9 us a tile, and 9 us for the rows' stores and their joining.  Trees of 16 to
// 48 nodes behind four prompts take 27 us, three short sequences 16.5.
#define TV_UNIT 17
#include "tv_attn_paged_tc.cuh"

namespace tv {
namespace paged {
namespace {

constexpr int kJoinThreads = 128;

// The status of the sequence of a block.  Beside tv_attn_paged's reasons: a malformed group at or ahead of it, a group with
// starts that descend, a prefix that does not fit, and a page of it that is none, as far as the sequence's window reaches.
__device__ __forceinline__ void prefix_status(const PagedAttnParams& p, int b) {
  const int lane = threadIdx.x, lanes = kJoinThreads;
  bool bad = !seq_ok(p, b, lane, lanes);
  const int good = p.desc[0].x;  // (their starts ascend)
  const int g = last_at_most(p.group_start, good, b);
  const int next = __ldg(p.group_start + g + 1);
  int t0, n, s0, sn, of = -1;
  if (g >= 0 && b < next) {
    of = g;
    bad |= !group_range(p, g, t0, n) || !seq_range(p.q_start, b, p.T, s0, sn) || s0 < t0 || s0 + sn > t0 + n;
    // (the positions of a group's tokens are searched for among its starts)
    if (!bad)
      for (int j = __ldg(p.group_start + g) + lane; j < next; j += lanes) bad |= __ldg(p.q_start + j + 1) < __ldg(p.q_start + j);
    const int L = __ldg(p.prefix_len + g);
    bad |= L < 0 || L > ((long long)p.prefix_P << p.page_shift);
    if (!bad && sn > 0) {
      const long long lo = p.window > 0 ? max(0ll, (long long)L + __ldg(p.kv_len + b) - p.window + 1) : 0;
      for (long long j = (lo >> p.page_shift) + lane; j << p.page_shift < L; j += lanes) {
        const int page = TV_IN(j, p.prefix_P) ? __ldg(p.prefix_table + (size_t)g * p.prefix_P + j) : 0;
        bad |= page < 0 || page >= p.num_pages;
      }
    }
  } else {  // behind the last group or ahead of the first
    bad |= good < p.groups && (good == 0 || b >= __ldg(p.group_start + good));
  }
  const bool late = is_late(p, b, lane, lanes, of);
  const int any_late = __syncthreads_or(late), any_bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) p.status[b] = any_late ? TV_ERR_TIMEOUT : any_bad ? TV_ERR_INVALID_ARG : TV_OK;
}

// A thread joins kC chunks of a row: the parts of its prefix's unit and of its own, or the whole
// units' rows, kBatch parts' loads in flight.  Lanes are consecutive rows (token, head) of one kv head, which lie
// side by side in the large units' parts.  Blocks behind the first row_blocks write the status.
template <int D, bool F16, int kC, int kBatch>
__global__ void __launch_bounds__(kJoinThreads)
prefix_join_kernel(const PagedAttnParams p, int nb, int row_blocks) {
  pdl_trigger();
  pdl_wait();
  if ((int)blockIdx.x >= row_blocks) {
    const int b = (((int)blockIdx.x - row_blocks) * gridDim.y + blockIdx.y) * gridDim.z + blockIdx.z;
    if (b < p.B) prefix_status(p, b);
    return;
  }
  const int r = blockIdx.x * kJoinThreads + threadIdx.x, kvh = blockIdx.y, c0 = blockIdx.z * kC;
  const int t = r / p.G, h_in = r - t * p.G;
  if (t >= p.T) return;
  // A token's units were noted by the kernel ahead; what is noted of a token that has none is old or
  // anything, and does not agree with the lengths (if it does, it was noted anew).  The rows are asked for before
  // that is known.
  const int4 mine = p.src[((size_t)p.T + t) * p.Hkv + kvh], pfx = p.src[(size_t)t * p.Hkv + kvh];
  const int b = min(max(mine.w, 0), p.B - 1), g = min(max(pfx.w, 0), p.groups - 1);
  const Seq s_own = load_own(p, b);
  const int good = p.desc[0].x;
  int gt, gn;
  const bool is_group = group_range(p, g, gt, gn);
  const bool is_own = mine.w == b && t >= s_own.t0 && t - s_own.t0 < s_own.n;
  const bool pre = pfx.w == g && g < good && is_group && t >= gt && t - gt < gn && b >= __ldg(p.group_start + g) &&
                   b < __ldg(p.group_start + g + 1);
  const size_t oidx = (size_t)t * p.Hq + kvh * p.G + h_in, rows = (size_t)p.T * p.Hq;
  uint2* out = reinterpret_cast<uint2*>(p.out + oidx * D) + c0;
  float M = -INFINITY, l = 0.0f;
  float4 a[kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) a[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int side = 1; side >= 0; --side) {
    if (side == 0 && !pre) break;
    const int4 s = side ? mine : pfx;
    // a part's rows lie chunk by chunk ([D / 4][256]): two row blocks of nb tokens in 128 each
    const int parts = s.x < 0 ? 1 : min(s.y, p.ctas), tl = (int)((unsigned)t - (unsigned)s.z), rb = tl >= nb;
    // (what nobody noted, of nobody's token or where a CTA gave up, may be anything)
    if (s.x >= 0 && (tl < 0 || tl >= 2 * nb || s.x >= 2 * p.ctas)) continue;
    const int crow = rb * 128 + (tl - rb * nb) * p.G + h_in;
    for (int j0 = 0; j0 < parts; j0 += kBatch) {
      float2 ml[kBatch];
      float4 v[kBatch][kC];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        ml[j] = make_float2(-INFINITY, 0.0f);
        // (the part that begins a unit is its share's last, the others are their shares' first)
        const int slot = j0 + j == 0 ? s.x : s.x - 1 + 2 * (j0 + j);
        if (j0 + j < parts && s.x < 0) {
          ml[j] = p.raw_ml[side * rows + oidx];
          const float4* src = reinterpret_cast<const float4*>(p.raw + (side * rows + oidx) * D) + c0;
#pragma unroll
          for (int c = 0; c < kC; ++c) v[j][c] = src[c];
        } else if (j0 + j < parts && slot < 2 * p.ctas) {
          ml[j] = p.part_ml[(size_t)slot * 256 + crow];
          const float4* src = reinterpret_cast<const float4*>(p.part) + (size_t)slot * 256 * (D / 4) + crow;
#pragma unroll
          for (int c = 0; c < kC; ++c) v[j][c] = src[(c0 + c) * 256];
        }
      }
      float mx = M;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) mx = fmaxf(mx, ml[j].x);
      // (maxima leave a NaN out, sums carry it: 0 times NaN is NaN)
      const float f = M == -INFINITY ? 0.0f : ex2(M - mx);
      M = mx;
      l *= f;
#pragma unroll
      for (int c = 0; c < kC; ++c) a[c] = make_float4(a[c].x * f, a[c].y * f, a[c].z * f, a[c].w * f);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const float e = ml[j].x == -INFINITY ? 0.0f : ex2(ml[j].x - M);
        l = fmaf(e, ml[j].y, l);
        if (e == 0.0f) continue;  // (a part whose keys are all hidden: select, do not multiply)
#pragma unroll
        for (int c = 0; c < kC; ++c)
          a[c] = make_float4(fmaf(e, v[j][c].x, a[c].x), fmaf(e, v[j][c].y, a[c].y), fmaf(e, v[j][c].z, a[c].z),
                             fmaf(e, v[j][c].w, a[c].w));
      }
    }
  }
  if (!is_own) return;  // nobody's token
  if (s_own.bad) {
    l = 0.0f;
#pragma unroll
    for (int c = 0; c < kC; ++c) a[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int c = 0; c < kC; ++c)
    out[c] = make_uint2(pack2<F16>(a[c].x * inv, a[c].y * inv), pack2<F16>(a[c].z * inv, a[c].w * inv));
  if (c0 == 0 && p.lse) p.lse[oidx] = s_own.bad ? 0.0f : l == 0.0f ? -INFINITY : (M + log2f(l)) * kLn2;
}

template <int D, bool F16, int kC, int kBatch>
cudaError_t launch_join(const PagedPlan& pl, const PagedAttnParams& p, cudaStream_t stream) {
  const int z = D / 4 / kC, per = p.Hkv * z;
  const int row_blocks = (int)(((long long)p.T * p.G + kJoinThreads - 1) / kJoinThreads);
  const int status_blocks = p.status ? ceil_div(p.B, per) : 0;
  if (row_blocks + status_blocks == 0) return cudaSuccess;
  return launch_pdl(prefix_join_kernel<D, F16, kC, kBatch>, dim3(row_blocks + status_blocks, p.Hkv, z),
                    dim3(kJoinThreads), 0, stream, p, pl.nb, row_blocks);
}
template <int D, bool F16>
cudaError_t launch_size(const PagedPlan& pl, const PagedAttnParams& p, cudaStream_t stream) {
  // Few rows have many parts: 64 decode tokens of 32 heads behind 8,000 rows 46.1 us at two chunks and four parts a
  // thread, 44.2 at one and eight; trees of 500 nodes of 16 heads 27.0 and 28.2 us.
  if ((long long)p.T * p.Hq <= 4096) return launch_join<D, F16, 1, 8>(pl, p, stream);
  return launch_join<D, F16, 2, 4>(pl, p, stream);
}

}  // namespace

cudaError_t launch_prefix(const PagedPlan& pl, int D, bool f16, bool bias, const CUtensorMap& tmQ,
                          const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedAttnParams& p,
                          cudaStream_t stream) {
  const cudaError_t e = launch_any<true, false>(pl, D, f16, bias, tmQ, tmK, tmV, p, stream);
  if (e != cudaSuccess) return e;
  if (D == 128) return f16 ? launch_size<128, true>(pl, p, stream) : launch_size<128, false>(pl, p, stream);
  return f16 ? launch_size<64, true>(pl, p, stream) : launch_size<64, false>(pl, p, stream);
}

}  // namespace paged
}  // namespace tv
