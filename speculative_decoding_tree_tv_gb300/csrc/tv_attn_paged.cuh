// tv_attn_paged: attention of a ragged batch of new tokens over a paged cache -- what its
// kernels share.
//
// Work.  A unit is (sequence, kv head, query tile): the tile's rows are the
// (token, head) pairs of the GQA group, token-major, and they share every K/V
// tile.  Its keys are the tiles of [lo, hi): from the first key the window
// leaves to the last one that the tile's last token sees.  The units, in the
// order sequence, head, query tile, are laid end to end on one line, each as
// long as its key tiles plus kUnitCost (what starting and finishing a unit costs,
// in tiles), and the line is cut into equal shares, one per resident CTA.
// So a ragged batch is balanced whatever its lengths are, without the host
// knowing them: every CTA finds its share from q_start and kv_len alone.  A unit
// that a cut splits leaves 32-bit partial rows (running maximum, sum, unnormalised
// output) in the workspace, and they are joined in one of two ways.  Where units
// are many, so that one is split over few CTAs, the CTA that a unit begins in (with the
// last item of its share) joins the rows of those that go on with it (with the
// first of theirs, so they are there as a rule).  Where few units are split
// over many CTAs, a merge kernel joins them, chained by programmatic dependent launch.
// The cuts depend on the lengths alone, so results do not vary from run to run.
//
// Two kernels take units: paged_rows_kernel (tv_attn_paged_rows.cu) those of at most 16 rows
// (decode tokens and small trees: HBM-bound, warp-level mma), and
// paged_tc_kernel (tv_attn_paged_tc.cuh, tcgen05) larger ones.  Over an 8-bit cache the former has a twin,
// paged_rows_q8_kernel (tv_attn_q8_rows.cuh), the latter a variant.  With shared prefixes (tv_attn_prefix.cu) the line
// holds the groups' prefixes, as sequences whose rows are all their group's tokens, ahead of the sequences.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>

#include "tv_paged.cuh"
#include "tv_sm100.cuh"

namespace tv {
namespace paged {

using namespace sm100;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kRescaleLog2 = 8.0f;  // keep a stale maximum while within 2^8

// A CTA whose waits gave up: rows of the sequences first .. last with tokens may not be there.  It counts
// only with this call's token.
struct Late {
  unsigned long long token;
  int first, last;
};

struct PagedAttnParams {
  const uint16_t* q;
  long long q_token_stride, q_head_stride;
  const uint8_t* k_scale;  // of an 8-bit cache: [pages, heads, rows]
  const uint8_t* v_scale;
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* kv_len;
  const uint64_t* anc;
  const float* slopes;
  uint16_t* out;
  float* lse;
  int32_t* status;
  float* part;      // [2 * CTAs] slots of partial rows
  float2* part_ml;  // their (running maximum, log2 domain; running sum)
  int4* desc;       // [CTAs]: the unit a CTA's share ends inside (first token, tokens, kv head, parts);
                    // with shared prefixes [0].x: the groups that count
  Late* late;       // [CTAs]
  unsigned long long* any_late;  // this call's token: some CTA is late
  long long wait_limit;          // SM cycles; 0: the producers of K and V give up before they load anything
  int B, T, P, Hq, Hkv, G, W, window;
  int ctas;         // of the attention kernel
  int num_pages, page_shift;
  int row_dim, head_dim;  // which of a cache map's dimensions 1, 2, 3 they are (the pages: the third)
  int tq;           // tokens per query tile
  int min_share;    // least cost of a share
  int share_lanes;  // log2 of the lanes that look at one sequence (1 << share_lanes) * B threads at most
  int whole;        // one unit a CTA, none is split
  int unit_cost;    // of starting and finishing a unit, in tiles
  int f16;          // 16-bit tensors are fp16 (the 8-bit cache's small units)
  int e4m3;         // codes of an 8-bit cache are e4m3, else int8
  int out_sectors;  // out lies on a 32-byte boundary
  int merge;        // a merge kernel joins the parts of split units, else the CTA a unit begins in
  unsigned long long token;      // this call's mark in `ready`
  unsigned long long* ready;     // [CTAs][8]: a warp of a share's first part has left its rows
  // Shared prefixes (tv_attn_prefix.cu): the line holds groups + B sequences, of which the first `groups` are the
  // prefixes: a group's tokens are its sequences', its keys the prefix's rows.  Rows of either kind are left
  // as they are (not divided by their sums) and joined by a kernel behind.
  int groups;                  // 0: none
  int prefix_P;
  const int32_t* group_start;  // [groups + 1] sequences
  const int32_t* prefix_len;   // [groups]
  const int32_t* prefix_table; // [groups, prefix_P]
  float* raw;                  // [2][T * Hq][D]: rows of units that are not split (0: prefixes', 1: own)
  float2* raw_ml;              // [2][T * Hq]
  int4* src;                   // [2][T * Hkv]: a token's unit: first slot (-1: in raw), parts, its first
                               // token, its prefix or sequence
  float scale_log2, softcap_log2, cap_in;  // cap_in: scale / softcap
  float cap_q[4], cap_top;  // capped scores s of s^2 <= cap_top: s (q0 + q1 s^2 + q2 s^4 + q3 s^6)
};

// ------------------------------------------------------------ small helpers
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (F16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
        "l"(*reinterpret_cast<const uint64_t*>(&c)));
  return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&d);
}
// 2^x on the special-function unit (flush-to-zero); 2^-inf = +0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// One box of a cache map: 64 dims from d0 of the rows from `row` of (page, head).  The map's
// outer dimensions lie in the order of their strides.
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, uint64_t* bar, int d0,
                                              int row, int head, int page, int row_dim, int head_dim) {
  const int c1 = row_dim == 1 ? row : head_dim == 1 ? head : page;
  const int c2 = row_dim == 2 ? row : head_dim == 2 ? head : page;
  const int c3 = row_dim == 3 ? row : head_dim == 3 ? head : page;
  tma_load_4d(dst, map, bar, d0, c1, c2, c3);
}
// A wait that gives up after `limit` SM cycles.  (The limit is looked at where a barrier is not ready: a
// chunk of 2048 157 us, with a branch on it ahead of every wait 166.5 us.)
__device__ __forceinline__ bool wait_within(uint64_t* bar, uint32_t parity, long long limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > limit) return false;
  return true;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, long long limit) {
  return __all_sync(0xffffffffu, wait_within(bar, parity, limit));
}
// Eight bytes to shared memory, zeros where `valid` is not set; they count on the barrier that
// the thread arrives at next with cp_arrive.
__device__ __forceinline__ void cp_async8(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(valid ? 8 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// tanh(y) as 1 - 2 / (1 + e^2y), y2 = 2 log2(e) y.  The subtraction leaves an
// absolute error of a few 2^-24, times the cap what a probability feels; tanh.approx is off by
// 2^-11 of the value.
__device__ __forceinline__ float tanh_any(float y2) { return fmaf(-2.0f, rcp(1.0f + ex2(y2)), 1.0f); }
// For |y| <= kTanhSmall tanh(y) / y is a cubic in y^2, fitted at Chebyshev nodes (relative
// error 2^-22 in 32-bit arithmetic), on the FMA pipe where the function above takes
// two special-function instructions.
constexpr float kTanhSmall = 0.4f;
constexpr float kTanhC[4] = {0.999999903f, -0.333313733f, 0.132711566f, -0.047561077f};

// Bits [a, b) of a 32-bit word (a, b any integers).
__device__ __forceinline__ uint32_t range_bits(int a, int b) {
  const uint32_t hi = b >= 32 ? 0xffffffffu : (b <= 0 ? 0u : (1u << b) - 1u);
  const uint32_t lo = a >= 32 ? 0xffffffffu : (a <= 0 ? 0u : (1u << a) - 1u);
  return hi & ~lo;
}
// 32 bits of the mask row starting at bit `pos` (-32 < pos < 64 W); 0 beyond it.
__device__ __forceinline__ uint32_t anc_bits32(const uint64_t* anc, int W, int pos) {
  if (pos < 0) return (uint32_t)anc[0] << -pos;
  const int wi = pos >> 6, sh = pos & 63;
  if (!TV_IN(wi, W)) return 0;
  const uint64_t lo = anc[wi], hi = (sh > 32 && wi + 1 < W) ? anc[wi + 1] : 0ull;
  return (uint32_t)((lo >> sh) | (sh ? hi << (64 - sh) : 0ull));
}
// Number of mask bits below bit `pos` (pos <= 64 W): a visible node a is at depth
// count(a + 1) - 1, as the mask's bits up to a are a and its own ancestors.
__device__ __forceinline__ int anc_count(const uint64_t* anc, int W, int pos) {
  int c = 0;
  for (int w = 0; w < W && 64 * w < pos; ++w)
    c += __popcll(pos - 64 * w >= 64 ? anc[w] : anc[w] & ((1ull << (pos - 64 * w)) - 1ull));
  return c;
}

// Depth of the node with this mask row: its ancestors.  A node whose mask is empty (of a tree that
// was refused) is taken at the root's depth, so that it reaches no further back than a window's pages.
__device__ __forceinline__ int anc_depth(const uint64_t* anc, int W) {
  return max(0, anc_count(anc, W, 64 * W) - 1);
}

// ------------------------------------------------------- shares of the work
// (16 trees of 64 nodes, a capped ragged batch and biased prompts of 200 to 1,500: 79.1, 64.2 and 29.5 us at 1;
// 75.7, 63.8 and 28.7 us at 3; 80.3, 63.0 and 33.0 us at 8)
constexpr int kUnitCost = 3;

// Whether group g's sequences are none.  The first such group and those behind it do not count (they may name
// sequences of the ones ahead).
__device__ __forceinline__ bool group_malformed(const PagedAttnParams& p, int g) {
  const int b0 = __ldg(p.group_start + g), b1 = __ldg(p.group_start + g + 1);
  return b0 < 0 || b1 < b0 || b1 > p.B;
}
// Tokens of group g: false for a malformed group_start or q_start.
__device__ __forceinline__ bool group_range(const PagedAttnParams& p, int g, int& t0, int& n) {
  const int b0 = __ldg(p.group_start + g), b1 = __ldg(p.group_start + g + 1);
  t0 = n = 0;
  if (b0 < 0 || b1 < b0 || b1 > p.B) return false;
  t0 = __ldg(p.q_start + b0);
  const int t1 = __ldg(p.q_start + b1);
  n = t1 - t0;
  return t0 >= 0 && t1 >= t0 && t1 <= p.T;
}
// The last of `n` ascending values that is at most x, or -1.
__device__ __forceinline__ int last_at_most(const int32_t* v, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(v + mid) <= x) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}
// The position of token t of group g behind a prefix of L rows.
__device__ __forceinline__ int prefix_pos(const PagedAttnParams& p, int g, int t, int L) {
  if (p.window == 0 && !p.slopes) return L;  // (not looked at)
  const int b0 = __ldg(p.group_start + g), n = __ldg(p.group_start + g + 1) - b0;
  const int b = b0 + max(0, last_at_most(p.q_start + b0, n, t));
  return L + __ldg(p.kv_len + b) +
         (p.anc ? anc_depth(p.anc + (size_t)t * p.W, p.W) : t - __ldg(p.q_start + b));
}

struct Seq {
  int t0, n, L;
  int lo;       // a prefix: the first row that a window reaches
  bool bad;     // rows are zeroed
  bool shared;  // a prefix
};

// The first row of a prefix of L that the window of some token of group g reaches: the sequence with the fewest
// rows of its own reaches back furthest.
__device__ __forceinline__ int prefix_reach(const PagedAttnParams& p, int g, int L) {
  const int b1 = __ldg(p.group_start + g + 1);
  int least = INT_MAX;
#pragma unroll 8
  for (int b = __ldg(p.group_start + g); b < b1; ++b) {
    const int own = __ldg(p.kv_len + b);
    if (__ldg(p.q_start + b + 1) > __ldg(p.q_start + b)) least = min(least, own);
  }
  return (int)min((long long)L, max(0ll, (long long)L + max(least, 0) - p.window + 1));
}

__device__ __forceinline__ Seq load_own(const PagedAttnParams& p, int b) {
  Seq s;
  s.shared = false;
  s.lo = 0;
  s.L = __ldg(p.kv_len + b);
  if (!seq_range(p.q_start, b, p.T, s.t0, s.n)) s.n = 0;
  s.bad = s.L < 0 || (long long)s.L + s.n > ((long long)p.P << p.page_shift) ||
          (p.anc && s.n > 64 * p.W);
  return s;
}
// PRE: with shared prefixes, which lie on the line (b) ahead of the sequences (a variant of its own: 4 short sequences
// took 11.6 us for 11.3 with groups looked for at run time).  good: the groups that count.
template <bool PRE>
__device__ __forceinline__ Seq load_seq(const PagedAttnParams& p, int b, int good) {
  if (!PRE || b >= p.groups) return load_own(p, PRE ? b - p.groups : b);
  Seq s;
  s.shared = true;
  s.L = __ldg(p.prefix_len + b);
  const bool is_group = group_range(p, b, s.t0, s.n);
  if (b >= good || !is_group) s.n = 0;
  s.bad = !is_group || s.L < 0 || s.L > ((long long)p.prefix_P << p.page_shift);
  s.lo = p.window > 0 && s.n > 0 && !s.bad ? prefix_reach(p, b, s.L) : 0;
  return s;
}

// Keys [lo, hi) that some token of query tile qt sees.
template <bool PRE>
__device__ __forceinline__ void key_range(const PagedAttnParams& p, const Seq& s, int qt, int& lo,
                                          int& hi) {
  const int first = qt * p.tq;
  if (PRE && s.shared) {  // (its tokens are all behind the prefix; no tiles where no window reaches it)
    lo = s.lo < s.L ? s.lo : 0;
    hi = s.lo < s.L ? s.L : 0;
    return;
  }
  hi = p.anc ? s.L + s.n : s.L + min(s.n, first + p.tq);
  // (the root of a tree sees furthest back)
  lo = p.window > 0 ? max(0, (p.anc ? s.L : s.L + first) - p.window + 1) : 0;
}
template <int KT, bool PRE>
__device__ __forceinline__ int key_tiles(const PagedAttnParams& p, const Seq& s, int qt) {
  if (s.bad) return 0;
  int lo, hi;
  key_range<PRE>(p, s, qt, lo, hi);
  return (hi + KT - 1) / KT - lo / KT;
}

// Shares are handed out against the CTAs' order: a CTA waits for the rows of later shares alone, whose
// CTAs have started before it.
__device__ __forceinline__ int share_index() { return (int)(gridDim.x - 1 - blockIdx.x); }

struct Part {
  Seq s;
  int b;             // its sequence; -1: the share is at its end
  int kvh;
  int first, ntok;   // the query tile's tokens: first, count
  int lo, hi;        // its keys
  int begin, end;    // key tiles of this part
  int slot;          // partial slot, or -1: the whole unit is here
  int parts;         // a unit that this part begins: how many parts it has
};

// (64-bit division costs some hundred cycles; the quotients here are small)
__device__ __forceinline__ long long div_fast(long long a, long long b) {
  if (((a | b) >> 31) == 0) return (unsigned)a / (unsigned)b;
  return a / b;
}

// A CTA's walk over its share of the line.
template <int KT, bool PRE = false>
struct Cursor {
  long long rest, share;  // cost left, cost of a share
  long long at;           // cost behind the share's start
  int b, kvh, qt, pos;    // unit, and cost of it that lies behind
  int last;               // the share's last sequence (or one behind it, where a thread looks at several)
  int good;               // groups that count
  Seq s;

  static __device__ __forceinline__ int line(const PagedAttnParams& p) { return PRE ? p.groups + p.B : p.B; }
  __device__ __forceinline__ int unit_cost(const PagedAttnParams& p) const { return PRE ? p.unit_cost : kUnitCost; }
  __device__ __forceinline__ int cost_of(const PagedAttnParams& p, int tiles) const {
    return p.whole ? 1 : tiles + unit_cost(p);
  }
  __device__ __forceinline__ bool next(const PagedAttnParams& p, Part& o) {
    while (rest > 0) {
      const int tiles = key_tiles<KT, PRE>(p, s, qt), cost = cost_of(p, tiles);
      const int take = (int)min((long long)(cost - pos), rest);
      const int a = p.whole ? 0 : max(0, pos - unit_cost(p));
      const int e = p.whole ? tiles : max(0, pos + take - unit_cost(p));
      const bool ends = pos + take == cost;
      const bool emit = e > a || (tiles == 0 && ends);
      if (emit) {
        key_range<PRE>(p, s, qt, o.lo, o.hi);
        o.s = s;
        o.b = b;
        o.kvh = kvh;
        o.first = qt * p.tq;
        o.ntok = min(p.tq, s.n - o.first);
        o.begin = o.lo / KT + a;
        o.end = o.lo / KT + e;
        o.slot = (a == 0 && e == tiles) ? -1 : p.merge ? 2 * share_index() + (a == 0) : share_index();
        o.parts = (o.slot >= 0 && a == 0) ? (int)div_fast(at - pos + cost - 1, share) + 1 : 0;
      }
      rest -= take;
      at += take;
      pos += take;
      if (ends) {
        pos = 0;
        if (++qt * (long long)p.tq >= s.n) {
          qt = 0;
          if (++kvh == p.Hkv) {
            kvh = 0;
            do {
              if (++b >= line(p)) break;
              s = load_seq<PRE>(p, b, good);
            } while (s.n == 0);
            if (b >= line(p)) rest = 0;
          }
        }
      }
      if (emit) return true;
    }
    o.b = -1;
    return false;
  }
};

// Lines of the lengths and of the block table into the L2, shared out over the CTAs, while
// the previous kernel finishes: a hint, which changes no result if that kernel writes them.
template <int THREADS, bool PRE = false>
__device__ __forceinline__ void prefetch_lengths(const PagedAttnParams& p) {
  const int first = (blockIdx.x * THREADS + threadIdx.x) * 32, step = gridDim.x * THREADS * 32;
  for (int i = first; i < p.B; i += step) {
    line_prefetch_l2(p.q_start + i);
    line_prefetch_l2(p.kv_len + i);
  }
  const long long words = min((long long)p.B * p.P, (long long)step);  // (one line a thread)
  if (first < words) line_prefetch_l2(p.table + first);
  if (!PRE) return;
  for (int i = first; i < p.groups; i += step) {
    line_prefetch_l2(p.group_start + i);
    line_prefetch_l2(p.prefix_len + i);
  }
  if (first < (long long)p.groups * p.prefix_P) line_prefetch_l2(p.prefix_table + first);
}

// The first malformed group, or p.groups (all THREADS threads; a function of its own, as hardly any call needs it and code
// at a kernel's start is new to the SM: the three cases of shared prefixes took 0.5 to 1.5 us longer with it in find_share).
template <int THREADS>
__device__ __noinline__ int first_malformed(const PagedAttnParams& p) {
  __shared__ int s_first;
  __syncthreads();
  if (threadIdx.x == 0) s_first = p.groups;
  __syncthreads();
  for (int g = threadIdx.x; g < p.groups; g += THREADS)
    if (group_malformed(p, g)) atomicMin(&s_first, g);
  __syncthreads();
  return s_first;
}

// Finds this CTA's share (s_cur: shared; rest is 0 where there is none); returns the groups that count.  All THREADS
// threads call it; ends with a barrier.  Where sequences are few and chunks long, 2^share_lanes lanes share one's query tiles
// (a lane that walked the 32 of a chunk of 2048 alone held up the first tile by some 3,000 cycles).
template <int KT, int THREADS, bool PRE>
__device__ __forceinline__ int find_share(const PagedAttnParams& p, Cursor<KT, PRE>& s_cur) {
  __shared__ long long s_warp[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lanes = 1 << p.share_lanes;
  const int seqs = Cursor<KT, PRE>::line(p), per = ceil_div(seqs, THREADS);  // (1 where lanes > 1)
  const int own = tid >> p.share_lanes, b0 = min(seqs, own * per), b1 = min(seqs, b0 + per);
  Cursor<KT, PRE> c;
  c.good = PRE ? p.groups : 0;
  int qt0 = 0, qt1 = 0;  // this lane's query tiles
  auto tiles_cost = [&](const Seq& s) {  // of one kv head's units among them
    const int nq = s.n > 0 ? (s.n - 1) / p.tq + 1 : 0, each = (nq + lanes - 1) >> p.share_lanes;
    qt0 = min(nq, (tid & (lanes - 1)) * each);
    qt1 = min(nq, qt0 + each);
    long long v = 0;
    for (int qt = qt0; qt < qt1; ++qt) v += c.cost_of(p, key_tiles<KT, PRE>(p, s, qt));
    return v;
  };
  long long sum, one, before = 0, inc;  // (before: of the head's units ahead of this lane's)
  for (;;) {
    bool look = false;
    sum = one = 0;
    for (int b = b0; b < b1; ++b) {
      c.s = load_seq<PRE>(p, b, c.good);
      look |= c.s.bad && b < c.good;
      one = tiles_cost(c.s);
      sum += one * p.Hkv;
    }
    inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) s_warp[warp] = inc;
    if (tid == 0) s_cur.rest = 0;
    if (!PRE) {
      __syncthreads();
      break;
    }
    if (!__syncthreads_or(look)) break;
    const int good = first_malformed<THREADS>(p);
    if (good == c.good) break;
    c.good = good;  // (the lengths anew)
  }
  long long base = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) base += s_warp[w];
    total += s_warp[w];
  }
  if (lanes > 1) {  // the sequence's start and cost, from its lanes
    const int first = lane & ~(lanes - 1), last = first + lanes - 1;
    const long long end = __shfl_sync(0xffffffffu, base + sum, last);
    const long long mine = base;
    base = __shfl_sync(0xffffffffu, base, first);
    sum = end - base;
    before = div_fast(mine - base, p.Hkv);
    one = div_fast(sum, p.Hkv);
  }
  const long long base0 = base;
  c.share = max(div_fast(total + gridDim.x - 1, gridDim.x), (long long)p.min_share);
  const long long x0 = share_index() * c.share;
  c.rest = min(total - x0, c.share);
  if (c.rest > 0 && x0 >= base && x0 < base + sum) {  // this lane's sequences hold the share's start
    c.b = b0;
    if (per > 1) {
      for (;; ++c.b) {
        c.s = load_seq<PRE>(p, c.b, c.good);
        one = tiles_cost(c.s);
        if (x0 < base + one * p.Hkv) break;
        base += one * p.Hkv;
      }
    }
    c.at = 0;
    c.kvh = (int)div_fast(x0 - base, one);
    long long left = x0 - base - c.kvh * one - before;
    for (c.qt = qt0; left >= 0 && c.qt < qt1; ++c.qt) {
      const int cost = c.cost_of(p, key_tiles<KT, PRE>(p, c.s, c.qt));
      if (left < cost) {
        c.pos = (int)left;
        s_cur.rest = c.rest;
        s_cur.share = c.share;
        s_cur.at = c.at;
        s_cur.b = c.b;
        s_cur.kvh = c.kvh;
        s_cur.qt = c.qt;
        s_cur.pos = c.pos;
        s_cur.s = c.s;
        s_cur.good = c.good;
        break;
      }
      left -= cost;
    }
  }
  const long long x1 = x0 + c.rest;  // the share's end, among this lane's sequences?
  if (c.rest > 0 && x1 > base0 && x1 <= base0 + sum) s_cur.last = b1 - 1;
  __syncthreads();
  return c.good;
}

// The parts of a CTA's share, published by the one warp that walks it: the other
// warps read a part from shared memory when they come to it.
constexpr int kPartRing = 4;
struct PartRing {
  Part part[kPartRing];
  uint64_t full[kPartRing], empty[kPartRing];

  __device__ __forceinline__ void init(int readers) {  // one thread
    for (int i = 0; i < kPartRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], readers);
    }
  }
  // (a whole warp)
  __device__ __forceinline__ bool publish(uint32_t n, const Part& w, long long limit) {
    const uint32_t i = n % kPartRing;
    if (!warp_wait(&empty[i], ((n / kPartRing) & 1) ^ 1, limit)) return false;
    if ((threadIdx.x & 31) == 0) {
      part[i] = w;
      mbar_arrive(&full[i]);
    }
    __syncwarp();
    return true;
  }
  __device__ __forceinline__ bool ready(uint32_t n, long long limit) {
    return wait_within(&full[n % kPartRing], (n / kPartRing) & 1, limit);
  }
  __device__ __forceinline__ const Part& at(uint32_t n) const { return part[n % kPartRing]; }
  __device__ __forceinline__ void done(uint32_t n) { mbar_arrive(&empty[n % kPartRing]); }  // one thread
};

// Whether sequence b's lengths fit and its pages are pages, as far as the window reaches;
// `lane` of `lanes` threads looks at its share of the pages.
__device__ __forceinline__ bool seq_ok(const PagedAttnParams& p, int b, int lane, int lanes) {
  int t0, n;
  if (!seq_range(p.q_start, b, p.T, t0, n)) return false;
  const Seq s = load_own(p, b);
  if (s.bad) return false;
  if (n == 0) return true;
  int lo, hi, any = 0;
  key_range<false>(p, s, 0, lo, hi);
  hi = s.L + n;
  const int32_t* row = p.table + (size_t)b * p.P;
#pragma unroll 8
  for (int j = (lo >> p.page_shift) + lane; j <= (hi - 1) >> p.page_shift; j += lanes) {
    const int page = TV_IN(j, p.P) ? __ldg(row + j) : 0;
    any |= page < 0 || page >= p.num_pages;
  }
  return any == 0;
}
// Whether a CTA that gave up may have left rows of sequence b (of group g) undone; `lane` of `lanes` threads
// looks at its share of the CTAs.
__device__ __forceinline__ bool is_late(const PagedAttnParams& p, int b, int lane, int lanes, int g = -1) {
  if (*(volatile unsigned long long*)p.any_late != p.token) return false;
  int t0, n;
  bool late = false;
  for (int c = lane; c < p.ctas; c += lanes) {
    volatile Late* l = p.late + c;
    late |= l->token == p.token && ((b + p.groups >= l->first && b + p.groups <= l->last) ||
                                    (g >= l->first && g <= l->last));
  }
  return late && seq_range(p.q_start, b, p.T, t0, n) && n > 0;
}
// status[b] of the sequences b = CTA, CTA + grid, .., by one warp, where no merge kernel follows
// to write it.  A CTA that gives up (report_late) leaves its mark, then the status; here the status comes
// first, then a look at the marks: with a fence between the two on either side, a look that misses
// the mark comes before it, and the status here before the one there.
__device__ __forceinline__ void write_status(const PagedAttnParams& p) {
  if (!p.status || blockIdx.x >= p.B) return;
  const int lane = threadIdx.x & 31;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const bool ok = __all_sync(0xffffffffu, seq_ok(p, b, lane, 32));
    if (lane == 0) *(volatile int32_t*)(p.status + b) = ok ? TV_OK : TV_ERR_INVALID_ARG;
  }
  __threadfence();
  for (int b = blockIdx.x; b < p.B; b += gridDim.x)
    if (__any_sync(0xffffffffu, is_late(p, b, lane, 32)) && lane == 0)
      *(volatile int32_t*)(p.status + b) = TV_ERR_TIMEOUT;
}
// A wait of this CTA gave up: the sequences of its share from `first` on may lack rows (one thread).
template <int KT, bool PRE>
__device__ __forceinline__ void report_late(const PagedAttnParams& p, const Cursor<KT, PRE>& share, int first) {
  if (share.rest <= 0) return;
  volatile Late* l = p.late + blockIdx.x;
  l->first = first;
  l->last = share.last;
  __threadfence();
  l->token = p.token;
  *(volatile unsigned long long*)p.any_late = p.token;
  __threadfence();
  if (p.merge || !p.status) return;  // (the merge kernel looks at the marks)
  for (int b = first; b <= share.last; ++b) {
    int t0, n;
    if (seq_range(p.q_start, b, p.T, t0, n) && n > 0) *(volatile int32_t*)(p.status + b) = TV_ERR_TIMEOUT;
  }
}

// Hand-over of partial rows within the launch, warp by warp (a warp holds the same rows of a
// unit in every CTA).  `ready` needs no clearing: a mark counts only if it is this
// call's, and a replayed graph, whose calls keep their mark, finds it taken away again.
__device__ __forceinline__ void leave_rows(const PagedAttnParams& p, int share, int warp) {
  __threadfence();
  __syncwarp();
  if ((threadIdx.x & 31) == 0)
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p.ready + share * 8 + warp), "l"(p.token) : "memory");
}
// False if the rows did not come within the limit.
__device__ __forceinline__ bool await_rows(const PagedAttnParams& p, int share, int warp) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) {
    unsigned long long* at = p.ready + share * 8 + warp;
    const long long t0 = clock64();
    for (;;) {
      unsigned long long v;
      asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(at) : "memory");
      if (v == p.token) break;
      if (clock64() - t0 > p.wait_limit) {
        ok = false;
        break;
      }
      __nanosleep(100);
    }
    if (ok) *at = 0;
  }
  return __all_sync(0xffffffffu, ok);
}

// The page ids of a part's tiles, last tile first, for a warp that issues their loads: one
// coalesced read of the block table covers 32 pages, and the next is on its way
// (a read per tile held the loads to a tile per memory latency).
template <int KT, bool PRE = false>
struct PageFeed {
  int rows, per_tile, tiles;  // rows of a box; pages of a tile; tiles of a read
  int page, next;             // this lane's page, and what the table says of the next read's
  bool next_needed;
  uint32_t bad;               // bit l: lane l's page is needed and is none

  // (the value is not looked at here, so that the read does not hold up the warp)
  __device__ __forceinline__ void read(const PagedAttnParams& p, const Part& w, int t0) {
    const int lane = threadIdx.x & 31, back = lane / per_tile, t = t0 - back;
    const int key = t * KT + (lane - back * per_tile) * rows, j = key >> p.page_shift;
    next_needed = back < tiles && t >= w.begin && key < w.hi && key + rows > w.lo;
    const bool shared = PRE && w.s.shared;
    const int P = shared ? p.prefix_P : p.P;
    const int32_t* row = (shared ? p.prefix_table : p.table) + (size_t)(PRE && !shared ? w.b - p.groups : w.b) * P;
    next = next_needed && TV_IN(j, P) ? __ldg(row + j) : -1;
  }
  __device__ __forceinline__ void take(const PagedAttnParams& p) {
    const bool is_page = next >= 0 && next < p.num_pages;
    page = is_page ? next : p.num_pages;  // (a tensor map reads zeros there)
    bad = __ballot_sync(0xffffffffu, next_needed && !is_page);
  }
  __device__ __forceinline__ void start(const PagedAttnParams& p, const Part& w) {
    rows = min(1 << p.page_shift, KT);
    per_tile = KT / rows;
    tiles = 32 / per_tile;
    read(p, w, w.end - 1);
  }
  // For tile t (they come in order): the page of the box at row `pg` * rows, and bits of 8
  // keys each that have no page.
  __device__ __forceinline__ int get(const PagedAttnParams& p, const Part& w, int t, int pg,
                                     uint32_t& bad8) {
    const int off = (w.end - 1 - t) & (tiles - 1);
    if (off == 0) {
      take(p);
      read(p, w, t - tiles);
    }
    bad8 = 0;
    if (bad) {
      const uint32_t b = bad >> (off * per_tile);
      for (int g = 0; g < KT / 8; ++g) bad8 |= ((b >> (8 * g / rows)) & 1u) << g;
    }
    return __shfl_sync(0xffffffffu, page, off * per_tile + pg);
  }
};

// The scale bytes of the eight rows from `row` of (page, head), zeros where there is no page.
__device__ __forceinline__ void load_scales(const PagedAttnParams& p, uint8_t* dst, const uint8_t* src, int page,
                                            int head, int row) {
  const bool valid = TV_CHECK(page >= 0) && page < p.num_pages;
  const long long at = valid ? (((long long)page * p.Hkv + head) << p.page_shift) + row : 0;
  cp_async8(dst, src + at, valid);
}

// How a call runs: the kernel, its CTAs, and the layout of the workspace.
struct PagedPlan {
  bool small;  // units of at most 16 rows: paged_rows_kernel
  int rows;  // rows of a unit
  int tq, nb, ctas, min_share;
  int whole;  // units are not split
  int merge;  // the merge kernel follows
  size_t part_bytes, ml_bytes, desc_bytes, late_bytes, ready_bytes;
  size_t bytes() const { return part_bytes + ml_bytes + desc_bytes + late_bytes + ready_bytes; }
};

constexpr int kTcKeys = 128;  // keys of a tile of the tcgen05 kernel
constexpr int kQ8Keys = 128;  // keys of a stage of the 8-bit cache's small kernel

// bias: slopes, or tree distances that the window reaches (mod: those or a cap)
cudaError_t launch_rows(const PagedPlan& pl, int D, bool f16, bool mod, const CUtensorMap& tmK,
                        const CUtensorMap& tmV, const PagedAttnParams& p, cudaStream_t stream);
cudaError_t launch_tc_q8(const PagedPlan& pl, int D, bool f16, bool bias, const CUtensorMap& tmQ,
                         const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedAttnParams& p,
                         cudaStream_t stream);
cudaError_t launch_rows_e4m3(const PagedPlan& pl, int D, bool mod, const CUtensorMap& tmK,
                             const CUtensorMap& tmV, const PagedAttnParams& p, cudaStream_t stream);
cudaError_t launch_rows_int8(const PagedPlan& pl, int D, bool mod, const CUtensorMap& tmK,
                             const CUtensorMap& tmV, const PagedAttnParams& p, cudaStream_t stream);
// a call with shared prefixes: paged_tc_kernel and the kernel that joins the rows
cudaError_t launch_prefix(const PagedPlan& pl, int D, bool f16, bool bias, const CUtensorMap& tmQ,
                          const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedAttnParams& p,
                          cudaStream_t stream);
cudaError_t launch_tc(const PagedPlan& pl, int D, bool f16, bool bias, const CUtensorMap& tmQ,
                      const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedAttnParams& p,
                      cudaStream_t stream);

}  // namespace paged
}  // namespace tv
