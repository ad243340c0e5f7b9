// paged_rows_q8_kernel: units of at most 16 rows over an 8-bit cache.  Its shape is paged_rows_kernel's
// (tv_attn_paged_rows.cu): a producer warp each for K and V, consumer warps with keys of their own and
// no barrier between them until the unit's end.  A stage is 128 keys: its codes take the bytes that 64
// keys of a 16-bit cache take, and the scales come with them (a byte a key).
//
// Codes become fp16 operands in registers (e4m3 and int8 values are exact there), and scales never meet
// them: with q_r = 2^a_r q'_r (a row's largest |q'| in [1, 2)), k_j = 2^s_j k'_j, v_j = 2^t_j v'_j,
//   x_rj = 2^(a_r + s_j) q'_r . k'_j,   O_r = sum_j (p_rj 2^t_j) v'_j,
// a score takes its key's factor behind the first product, a probability its row's ahead of the second.
// p_rj 2^t_j is rounded to fp16 (half a step: 2^-11 of it) as p 2^(t_j - c + 6), c about the warp's largest t: from
// 2^-20 of that on with all its bits, below to multiples of 2^-30.  Where the warp's t differ by more
// than kNear allows, c is the row's own, that of its largest p_rj 2^t_j: a row that it does not see, or hardly, has no say
// in its bits.
//
// An operand's 16 dims (or rows) are in the order in which the bytes lie: ldmatrix takes byte
// pairs for 16-bit values, so a lane gets dims 4c .. 4c + 3 of a key, which serve as the mma's k = 2c, 2c + 1,
// 2c + 8, 2c + 9 (q' in the same order), and of V, transposed, dims 2g and 2g + 1 of keys 2c and 2c + 1.
//
// Bound by HBM, 2 D + 2 bytes a key: a decode of 64 sequences of 512 to 8,192 keys (8 kv heads, D 128) takes 108 us
// with e4m3, 85 % of the copy rate (7 us of it the merge, some 8 the start and the drain; 186 us over 16 bits), and 121 us
// with int8, whose codes take more instructions on their way to fp16.  At D 64, where a key has half the bytes and the
// same scores to turn into probabilities, 89 us (52 %).  V rows too far apart for one power of two: 134 us.
#pragma once

#include <cfloat>

#include "tv_quant.cuh"
#include "tv_warp_mma.cuh"

namespace tv {
namespace paged {
namespace {

constexpr int kUnitRows = 16;  // rows of a slot
constexpr int kPBias = 6;      // probabilities of up to 2^8 (a stale maximum) stay below 2^15

// NW consumer warps share a stage's keys: 4 and two CTAs an SM, or 8 and one where every unit has an SM to
// itself (p.whole).
template <int D, int NW>
struct RowsQ8Layout {
  static constexpr int kSide = kQ8Keys * D;  // codes of K or V of a stage
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kScratch = NW * 16 * 32 * 4;  // [warp][row][32 dims]; the unit's Q rows ahead of that
  static constexpr int kDyn = 2 * kStages * (kSide + kQ8Keys) + kScratch + 1024;
};

// 16-byte chunk c of a row of codes, as TMA lays it out (128-byte swizzle, for D 64 the 64-byte one).
template <int D>
__device__ __forceinline__ int chunk_at(int key, int c) {
  return key * D + ((D == 128 ? c ^ (key & 7) : c ^ ((key >> 1) & 3)) << 4);
}

// fp16 pairs of four codes: the first two and the last two.
template <bool E4M3>
__device__ __forceinline__ void halves(uint32_t x, uint32_t& lo, uint32_t& hi) {
  if (E4M3) {
    asm("{.reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
  } else {  // 1024 + (code + 128), less 1152
    const uint32_t u = x ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x0 = __hsub2(*reinterpret_cast<__half2*>(&a), off), x1 = __hsub2(*reinterpret_cast<__half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x0);
    hi = *reinterpret_cast<const uint32_t*>(&x1);
  }
}
// Two dims of two keys (dims of the first key in the low half): pairs of keys for either dim.
template <bool E4M3>
__device__ __forceinline__ void halves_t(uint32_t x, uint32_t& even, uint32_t& odd) {
  halves<E4M3>(__byte_perm(x, 0, 0x3120), even, odd);
}

// Q's and the outputs' type makes no variant: it matters at a unit's ends alone.
__device__ __forceinline__ float2 unpack16(int f16, uint32_t x) {
  return f16 ? q8::unpack<true>(x) : q8::unpack<false>(x);
}
__device__ __forceinline__ uint32_t pack16(int f16, float lo, float hi) {
  return f16 ? pack2<true>(lo, hi) : pack2<false>(lo, hi);
}

// A row's sum with that of a warp's (maximum, sum) on top (a NaN stays: maxima leave it out, sums do not).
__device__ __forceinline__ float row_sum(float2 v, float top, float sum) {
  return fmaf(v.x == -INFINITY ? 0.0f : ex2(v.x - top), v.y, sum);
}

// NR: the most rows of a unit.  16: S = Q K^T and O = P V.  8: S^T = K Q^T and O^T = V^T P^T, keys and
// dims in the mma's 16 and rows in its 8.
template <int D, bool E4M3, bool MOD, int NW, int NR>
__global__ void __launch_bounds__(32 * (NW + 2), NW == 4 ? 2 : 1)
paged_rows_q8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const PagedAttnParams p) {
  using Lay = RowsQ8Layout<D, NW>;
  constexpr int KB = kQ8Keys / (16 * NW), kWarpKeys = 16 * KB;  // blocks of 16 keys, keys of a warp
  constexpr int kSteps = D / 16, kThreads = 32 * (NW + 2), kStages = Lay::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sK = smem;
  uint8_t* sV = smem + kStages * Lay::kSide;
  uint8_t* s_q = smem + 2 * kStages * Lay::kSide;
  float* s_acc = reinterpret_cast<float*>(s_q);
  uint8_t* s_ks = s_q + Lay::kScratch;
  uint8_t* s_vs = s_ks + kStages * kQ8Keys;
  __shared__ __align__(8) uint64_t bar_full[kStages], bar_empty[kStages];
  __shared__ uint32_t s_bad_pages[kStages];  // bit g: keys 8 g .. 8 g + 7 have no page
  __shared__ float2 s_ml[NW][kUnitRows];
  __shared__ float s_qf[kUnitRows];          // 2^a of the unit's rows
  __shared__ volatile int s_abort;           // a consumer's wait ran out
  __shared__ PartRing s_ring;
  __shared__ Cursor<kQ8Keys> s_cur;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  if (tid == 0) {
    s_abort = 0;
    s_ring.init(NW + 1);  // V, consumers
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar_full[s], 2 + 64);  // (K's and V's bytes, and their lanes' scales)
      mbar_init(&bar_empty[s], NW);
    }
    mbar_fence_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  prefetch_lengths<kThreads>(p);
  pdl_wait();
  find_share<kQ8Keys, kThreads>(p, s_cur);
  uint32_t st = 0, phase = 0, np = 0;  // stage, its ring's phase; parts so far
  auto next_stage = [&]() {
    phase ^= st == kStages - 1;
    st = st == kStages - 1 ? 0 : st + 1;
  };

  if (warp >= NW) {
    // ------------------------------------------------- K, V producers
    // (K's also walks the share.)  Lane l < 16 has the keys 8 l .. 8 l + 7: their scales, and the
    // box of their page if they are its first.
    const bool isV = warp > NW;
    const CUtensorMap* map = isV ? &tmV : &tmK;
    uint8_t* ring = isV ? sV : sK;
    uint8_t* scales = isV ? s_vs : s_ks;
    const uint8_t* scale_src = isV ? p.v_scale : p.k_scale;
    Part w;
    Cursor<kQ8Keys> cur = s_cur;
    if (p.merge && !isV && lane == 0) p.desc[share_index()] = make_int4(0, 0, 0, 0);
    PageFeed<kQ8Keys> feed;
    const int rows_page = min(1 << p.page_shift, kQ8Keys);  // rows of one box
    const int row0 = (lane & 15) * 8, pg = row0 / rows_page;
    const bool issues = lane < 16 && row0 % rows_page == 0;
    uint32_t issued = 0;
    bool ok = p.wait_limit > 0;
    for (; ok; ++np) {
      if (isV) {
        ok = __all_sync(0xffffffffu, s_ring.ready(np, p.wait_limit));
        if (!ok) break;
        w = s_ring.at(np);
        __syncwarp();
        if (lane == 0) s_ring.done(np);
        if (w.b < 0) break;
      } else {
        const bool more = cur.next(p, w);
        ok = s_ring.publish(np, w, p.wait_limit);
        if (!ok || !more) break;
        if (w.parts && lane == 0)
          p.desc[share_index()] = make_int4(w.s.t0 + w.first, w.ntok, w.kvh, w.parts);
      }
      feed.start(p, w);
      for (int t = w.end - 1; t >= w.begin; --t) {
        const int row = (t * kQ8Keys + row0) & ((1 << p.page_shift) - 1);
        uint32_t bad8;
        const int page = feed.get(p, w, t, pg, bad8);
        ok = warp_wait(&bar_empty[st], phase ^ 1, p.wait_limit);
        if (!ok) break;
        if (lane == 0) {
          if (!isV) s_bad_pages[st] = bad8;
          mbar_expect_tx(&bar_full[st], Lay::kSide);
        }
        __syncwarp();
        if (issues)
          tma_load_rows(ring + st * Lay::kSide + row0 * D, map, &bar_full[st], 0, row, w.kvh, page, p.row_dim,
                        p.head_dim);
        if (lane < 16) load_scales(p, scales + st * kQ8Keys + row0, scale_src, page, w.kvh, row);
        cp_arrive(&bar_full[st]);
        next_stage();
        ++issued;
      }
      if (!ok) break;
    }
    if (!p.merge && !isV) write_status(p);
    // no copy may be in flight when the CTA leaves (where the other producer gave up, its half of a
    // stage never comes: this one's has landed long before the limit)
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (uint32_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
      if (!mbar_wait(&bar_full[i % kStages], (i / kStages) & 1)) break;
    return;  // (what a producer that gave up did not load, the consumers wait for in vain, and report)
  }

  // ---------------------------------------------------------------- consumers
  const float cap_in2 = 2.0f * kLog2e * p.cap_in;
  const int g = lane >> 2, c = lane & 3, c2 = 2 * c;  // fragment row; first column (of two) of this lane
  // A lane's two rows, and the kKeys keys of a block of 16 that it holds of both
  constexpr int kKeys = NR == 16 ? 4 : 2, kAll = KB * kKeys;
  constexpr int kAcc = NR == 16 ? D / 8 : D / 16;
  auto row_of = [&](int r) { return NR == 16 ? r * 8 + g : c2 + r; };
  auto key_of = [&](int i) {  // among the warp's
    const int k = i % kKeys;
    return 16 * (i / kKeys) + (NR == 16 ? 8 * (k >> 1) + c2 + (k & 1) : 8 * k + g);
  };
  auto at = [](int r, int i) {
    const int k = i % kKeys;
    return 8 * (i / kKeys) + (NR == 16 ? 4 * (k >> 1) + 2 * r + (k & 1) : 2 * k + r);
  };
  auto reduce = [](float x, auto op) {  // over the lanes that hold a row's keys
#pragma unroll
    for (int o = NR == 16 ? 1 : 4; o < (NR == 16 ? 4 : 32); o *= 2)
      x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  };
  int b = s_cur.b;
  for (;; ++np) {
    // (a warp that gives up still joins the others at the unit's end, where all see it)
    if (!__all_sync(0xffffffffu, s_ring.ready(np, p.wait_limit))) s_abort = 1;
    named_sync(1, NW * 32);
    if (s_abort) {
      if (tid == 0) report_late(p, s_cur, b);
      break;
    }
    const Part w = s_ring.at(np);
    if (w.b < 0) break;
    b = w.b;
    const int rows = w.ntok * p.G;
    // the unit's Q rows to shared memory, in fp16 and scaled (rows past the unit repeat its last one);
    // 16-byte chunk x of row r lies at x ^ (r & 7)
    for (int x = tid; x < NR * (D / 8); x += NW * 32) {
      const int r = x / (D / 8), ch = x % (D / 8), row = min(r, rows - 1);
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(
                                p.q + (w.s.t0 + w.first + row / p.G) * p.q_token_stride +
                                (w.kvh * p.G + row % p.G) * p.q_head_stride) + ch);
      const uint32_t in[4] = {v.x, v.y, v.z, v.w}, m = 0x7fff7fffu;
      uint32_t top = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
      top = max(top & 0xffffu, top >> 16);
#pragma unroll
      for (int o = 1; o < D / 8; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = min(max(__float_as_int(unpack16(p.f16, top).x) >> 23, 1), 253);
      const float f = __int_as_float((254 - e) << 23);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = unpack16(p.f16, in[i]);
        o[i] = pack2<true>(y.x * f, y.y * f);
      }
      *reinterpret_cast<uint4*>(s_q + r * (D * 2) + ((ch ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
      if (ch == 0) s_qf[r] = __int_as_float(e << 23);
    }
    named_sync(1, NW * 32);
    uint2 qf[NR / 8][kSteps];
#pragma unroll
    for (int h = 0; h < NR / 8; ++h)
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
        qf[h][k] = *reinterpret_cast<const uint2*>(s_q + (8 * h + g) * (D * 2) +
                                                   (((2 * k + (c >> 1)) ^ g) << 4) + (c & 1) * 8);
    int ve[2] = {-1, -1}, pos[2], tok[2];  // (ve: the power of two of a row's outputs, where V rows are far apart)
    float slope[2], in_scale[2];
    float m[2], l[2], o[kAcc][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = min(row_of(r), rows - 1);  // rows past the unit repeat its last
      const int i = w.first + row / p.G, t = w.s.t0 + i, h = w.kvh * p.G + row % p.G;
      tok[r] = t;
      pos[r] = w.s.L + (p.anc ? anc_depth(p.anc + (size_t)t * p.W, p.W) : i);
      slope[r] = (MOD && p.slopes) ? __ldg(p.slopes + h) * kLog2e : 0.0f;
      const bool cap = MOD && p.softcap_log2 > 0.0f;  // (the cap's function scales)
      in_scale[r] = s_qf[row_of(r)] * (cap ? 1.0f : p.scale_log2);
      m[r] = -INFINITY;
      l[r] = 0.0f;
    }
    // The outputs are held as O 2^(kPBias + 127 - vtop), vtop from the scale bytes (-1: no row yet): one above the first
    // tile's largest, for tiles from vtop - kNear + 1 to vtop + 1.  From the first that is not on, they are held over a
    // power of two of each row.
    int vtop = -1;
    bool apart = false;
#pragma unroll
    for (int n = 0; n < kAcc; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    const int all_below = p.anc ? w.s.L : w.s.L + w.first + 1;  // keys below it are visible to every row
    const int all_from = p.window > 0
                             ? (p.anc ? w.s.L + w.s.n : w.s.L + w.first + w.ntok) - p.window : -1;

    for (int t = w.end - 1; t >= w.begin; --t) {  // (last first: see paged_tc_kernel)
      const int j0 = t * kQ8Keys + kWarpKeys * warp;
      if (!warp_wait(&bar_full[st], phase, p.wait_limit)) {
        s_abort = 1;
        break;
      }
      if (j0 < w.hi && j0 + kWarpKeys > w.lo) {
        const uint32_t aK = smem_u32(sK) + st * Lay::kSide, aV = smem_u32(sV) + st * Lay::kSide;
        float s[KB * 8];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const int key0 = kWarpKeys * warp + 16 * kb;
          float s0[4] = {}, s1[4] = {};
          // (matrices: keys 0 .. 7 and 8 .. 15 of 16 dims, then of the next 16)
          const int key = key0 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
          for (int k = 0; k < kSteps / 2; ++k) {
            uint32_t x[4], lo[4], hi[4];
            ldsm4(aK + chunk_at<D>(key, 2 * k + (lane >> 4)), x);
#pragma unroll
            for (int i = 0; i < 4; ++i) halves<E4M3>(x[i], lo[i], hi[i]);
            if (NR == 16) {  // S: [8 keys][row g: two keys, row g + 8: two keys]
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint2 q0 = qf[0][2 * k + i], q1 = qf[NR / 8 - 1][2 * k + i];
                const uint32_t a[4] = {q0.x, q1.x, q0.y, q1.y};
                mma16816<true>(s0, a, lo[2 * i], hi[2 * i]);
                mma16816<true>(s1, a, lo[2 * i + 1], hi[2 * i + 1]);
              }
            } else {  // S^T: [key g: two rows, key g + 8: two rows], even and odd steps apart
              const uint32_t a0[4] = {lo[0], lo[1], hi[0], hi[1]}, a1[4] = {lo[2], lo[3], hi[2], hi[3]};
              mma16816<true>(s0, a0, qf[0][2 * k].x, qf[0][2 * k].y);
              mma16816<true>(s1, a1, qf[0][2 * k + 1].x, qf[0][2 * k + 1].y);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[8 * kb + e] = NR == 16 ? s0[e] : s0[e] + s1[e];
            s[8 * kb + 4 + e] = s1[e];
          }
        }
        const uint32_t bad8 = (s_bad_pages[st] >> (2 * KB * warp)) & ((1u << (2 * KB)) - 1u);
        const bool plain = j0 + kWarpKeys <= all_below && j0 > all_from && j0 >= w.lo && bad8 == 0;
        // the keys' scales: factors of K, bytes of V
        float kf[kAll];
        int vb[kAll];
        unsigned off = 0;  // how far the bytes of V are from what the outputs are held over
        const uint8_t* ks = s_ks + st * kQ8Keys + kWarpKeys * warp;
        const uint8_t* vs = s_vs + st * kQ8Keys + kWarpKeys * warp;
#pragma unroll
        for (int i = 0; i < kAll; ++i) {
          kf[i] = q8::factor(ks[key_of(i)]);
          vb[i] = vs[key_of(i)];
          off = max(off, (unsigned)(vb[i] - (vtop + 1 - q8::kNear)));
        }
        uint32_t hidden = 0;  // bits by s's index
        // scores in the log2 domain, hidden keys at -inf
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < kAll; ++i) s[at(r, i)] *= q8::at_most(in_scale[r] * kf[i], FLT_MAX);
        if (MOD && p.softcap_log2 > 0.0f) {
          float f[KB * 8], top = 0.0f;
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < kAll; ++i) {
              const float x = s[at(r, i)], w2 = x * x;
              const int j = j0 + key_of(i);
              if (plain || (j >= w.lo && j < w.hi)) top = fmaxf(top, w2);
              f[at(r, i)] = x * fmaf(fmaf(fmaf(p.cap_q[3], w2, p.cap_q[2]), w2, p.cap_q[1]), w2, p.cap_q[0]);
            }
          const bool far = __any_sync(0xffffffffu, top > p.cap_top);
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < kAll; ++i)
              s[at(r, i)] = far ? p.softcap_log2 * tanh_any(s[at(r, i)] * cap_in2) : f[at(r, i)];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < kAll; ++i) {
            float& x = s[at(r, i)];
            const int j = j0 + key_of(i);
            int kpos = j;
            if (!plain) {
              // (causal: up to its own position; a tree's: the prefix and its mask)
              bool see = j < (p.anc ? w.s.L : pos[r] + 1);
              if (p.anc && j >= w.s.L && j < w.hi) {
                const int a = j - w.s.L;
                const uint64_t* anc = p.anc + (size_t)tok[r] * p.W;
                see = (__ldg(reinterpret_cast<const unsigned long long*>(anc) + (a >> 6)) >> (a & 63)) & 1;
                if (MOD) kpos = w.s.L + anc_count(anc, p.W, a + 1) - 1;
              }
              if (p.window > 0) see = see && pos[r] - kpos < p.window;
              if ((bad8 >> (key_of(i) >> 3)) & 1) see = false;
              if (MOD) x = fmaf(slope[r], (float)(kpos - pos[r]), x);
              if (!see) {
                x = -INFINITY;
                hidden |= 1u << at(r, i);
              }
            } else if (MOD) {
              x = fmaf(slope[r], (float)(kpos - pos[r]), x);
            }
          }
        // running maximum (lazily moved), probabilities, sums
        float corr[2], before[2];
        bool move = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float mx = s[at(r, 0)];
#pragma unroll
          for (int i = 1; i < kAll; ++i) mx = fmaxf(mx, s[at(r, i)]);
          mx = reduce(mx, [](float a, float b) { return fmaxf(a, b); });
          corr[r] = 1.0f;
          before[r] = m[r];
          if (m[r] == -INFINITY) {
            m[r] = mx;
          } else if (mx > m[r] + kRescaleLog2) {
            corr[r] = ex2(m[r] - mx);
            m[r] = mx;
            move = true;
          }
          const float mm = m[r] == -INFINITY ? 0.0f : m[r];  // 2^(-inf - 0) = 0
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < kAll; ++i) sum += s[at(r, i)] = ex2(s[at(r, i)] - mm);
          l[r] = fmaf(l[r], corr[r], sum);
        }
        if (!apart && __any_sync(0xffffffffu, off > q8::kNear)) {
          // (keys outside of the unit's range hold anything; rows that are no numbers count for none)
          int lo = 255, hi = -1;
#pragma unroll
          for (int i = 0; i < kAll; ++i) {
            const int j = j0 + key_of(i);
            if (vb[i] == q8::kNaN || j < w.lo || j >= w.hi) continue;
            lo = min(lo, vb[i]);
            hi = max(hi, vb[i]);
          }
          hi = __reduce_max_sync(0xffffffffu, hi);
          lo = __reduce_min_sync(0xffffffffu, lo);
          const int top = vtop < 0 ? hi + 1 : vtop;
          if (hi >= 0 && hi <= top + 1 && lo > top - q8::kNear) {
            vtop = top;  // (if these are the first rows, the outputs are 0 so far)
          } else if (hi >= 0) {
            apart = true;
            ve[0] = ve[1] = vtop;
          }
        }
        if (apart) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            int want = q8::kNone;
#pragma unroll
            for (int i = 0; i < kAll; ++i) {
              const float x = s[at(r, i)];
              if (x > 0.0f && vb[i] != q8::kNaN) want = max(want, (__float_as_int(x) >> 23) - 126 + vb[i]);
            }
            want = (int)reduce((float)want, [](float a, float b) { return fmaxf(a, b); });
            const bool fresh = before[r] == -INFINITY;
            const int e = q8::held_over(ve[r], want, m[r] - before[r], fresh);
            move |= e != ve[r];
            // (fresh: outputs of 0)
            corr[r] = fresh || m[r] == before[r] ? q8::exp2_whole(ve[r] - e) : ex2(before[r] - m[r] + (float)(ve[r] - e));
            ve[r] = e;
          }
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int n = 0; n < kAcc; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] *= corr[NR == 16 ? e >> 1 : e & 1];
        }
        if (apart) {
#pragma unroll
          for (int i = 0; i < kAll; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float& x = s[at(r, i)];
              const float y = vb[i] == q8::kNaN ? q8::factor(q8::kNaN) : q8::times_exp2(x, vb[i] - ve[r] + kPBias);
              x = (hidden >> at(r, i)) & 1 ? 0.0f : y;
            }
        } else {
#pragma unroll
          for (int i = 0; i < kAll; ++i) {
            // (of a key that no row sees it may be anything)
            const float f = vb[i] == q8::kNaN ? q8::factor(q8::kNaN) : __int_as_float((vb[i] - vtop + 127 + kPBias) << 23);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float& x = s[at(r, i)];
              x = (hidden >> at(r, i)) & 1 ? 0.0f : x * f;  // (a hidden row's scale may say NaN)
            }
          }
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const int key0 = kWarpKeys * warp + 16 * kb;
          uint32_t vkeep[2] = {0xffffffffu, 0xffffffffu};  // V pairs of keys that some row may see
          if (!plain) {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int j = j0 + 16 * kb + 8 * nt + c2 + e;
                if (j < w.lo || j >= w.hi) vkeep[nt] &= e ? 0x0000ffffu : 0xffff0000u;
              }
          }
          const float* sb = s + 8 * kb;
          uint32_t pf[4] = {pack2<true>(sb[0], sb[1]), pack2<true>(sb[2], sb[3]), 0, 0};
          if (NR == 16) {
            pf[2] = pack2<true>(sb[4], sb[5]);
            pf[3] = pack2<true>(sb[6], sb[7]);
          } else {
            pf[0] = transpose8(pf[0]);
            pf[1] = transpose8(pf[1]);
          }
          const int key = key0 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
          for (int n = 0; n < kSteps / 2; ++n) {
            uint32_t x[4], ev[4], od[4];
            ldsm4_t(aV + chunk_at<D>(key, 2 * n + (lane >> 4)), x);
            if (!plain) {
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] &= vkeep[i & 1];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) halves_t<E4M3>(x[i], ev[i], od[i]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // 16 dims each
              if (NR == 16) {  // O += P V: even dims, odd dims
                mma16816<true>(o[(2 * (2 * n + i)) % kAcc], pf, ev[2 * i], ev[2 * i + 1]);
                mma16816<true>(o[(2 * (2 * n + i) + 1) % kAcc], pf, od[2 * i], od[2 * i + 1]);
              } else {  // O^T += V^T P^T
                const uint32_t a[4] = {ev[2 * i], od[2 * i], ev[2 * i + 1], od[2 * i + 1]};
                mma16816<true>(o[(2 * n + i) % kAcc], a, pf[0], pf[1]);
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_empty[st]);
      next_stage();
    }

    // the warps' rows joined in shared memory, 32 dims at a time
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] = reduce(l[r], [](float a, float b) { return a + b; });
      if (NR == 16 ? (lane & 3) == 0 : lane < 4) s_ml[warp][row_of(r)] = make_float2(m[r], l[r]);
    }
    named_sync(1, NW * 32);
    const bool abort = s_abort;
    float f[2], vf[2];  // (vf: the second of the outputs' own factor's two)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mm = -INFINITY, ll = 0.0f;
#pragma unroll
      for (int x = 0; x < NW; ++x) mm = fmaxf(mm, s_ml[x][row_of(r)].x);
      f[r] = m[r] == -INFINITY ? 0.0f : ex2(m[r] - mm);  // (0: nothing seen by this warp, its sums are 0)
      const int e = (apart ? ve[r] : vtop) - 127 - kPBias;
      f[r] *= q8::exp2_whole(e >> 1);
      vf[r] = q8::exp2_whole(e - (e >> 1));
      // (a whole unit's rows are divided by their sums ahead of vf: their own sums may pass the 32-bit range)
      if (w.slot < 0) {
#pragma unroll
        for (int x = 0; x < NW; ++x) ll = row_sum(s_ml[x][row_of(r)], mm, ll);
        f[r] *= ll == 0.0f ? 0.0f : 1.0f / ll;
      }
    }
    const int row = (tid >> 3) & (NR - 1), od = (tid & 7) * 4;  // this thread's row and dims of a joined piece
    float mm = -INFINITY, ll = 0.0f;
#pragma unroll
    for (int x = 0; x < NW; ++x) mm = fmaxf(mm, s_ml[x][row].x);
#pragma unroll
    for (int x = 0; x < NW; ++x) ll = row_sum(s_ml[x][row], mm, ll);
    const bool mine = tid < 8 * NR && row < rows;
    const int out_tok = w.s.t0 + w.first + row / p.G, h = w.kvh * p.G + row % p.G;
    const size_t oidx = (size_t)out_tok * p.Hq + h;
    auto swz = [](int r) { return NR == 16 ? (r & 1) << 4 : ((r & 6) << 2) | ((r & 1) << 2); };
#pragma unroll
    for (int d = 0; d < D / 32; ++d) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {  // 16 dims each
        if (NR == 16) {
          const float(&ev)[4] = o[(4 * d + 2 * x) % kAcc], (&odd)[4] = o[(4 * d + 2 * x + 1) % kAcc];
#pragma unroll
          for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float4*>(s_acc + (warp * 16 + r * 8 + g) * 32 + ((16 * x + 4 * c) ^ swz(g))) =
                make_float4(ev[2 * r] * f[r] * vf[r], odd[2 * r] * f[r] * vf[r], ev[2 * r + 1] * f[r] * vf[r],
                            odd[2 * r + 1] * f[r] * vf[r]);
        } else {
          const float(&v)[4] = o[(2 * d + x) % kAcc];
#pragma unroll
          for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float2*>(s_acc + (warp * 16 + c2 + r) * 32 + ((16 * x + 2 * g) ^ swz(c2 + r))) =
                make_float2(v[r] * f[r] * vf[r], v[2 + r] * f[r] * vf[r]);
        }
      }
      named_sync(1, NW * 32);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < NW; ++x) {
        const float4 v = *reinterpret_cast<const float4*>(s_acc + (x * 16 + row) * 32 + (od ^ swz(row)));
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
      if (mine) {
        if (w.slot >= 0)
          *reinterpret_cast<float4*>(p.part + ((size_t)w.slot * kUnitRows + row) * D + 32 * d + od) = a;
        else if (TV_CHECK(out_tok < p.T && h < p.Hq))
          *reinterpret_cast<uint2*>(p.out + oidx * D + 32 * d + od) =
              make_uint2(pack16(p.f16, a.x, a.y), pack16(p.f16, a.z, a.w));
      }
      named_sync(1, NW * 32);
    }
    if (mine && (tid & 7) == 0) {
      if (w.slot >= 0) p.part_ml[(size_t)w.slot * kUnitRows + row] = make_float2(mm, ll);
      else if (p.lse) p.lse[oidx] = w.s.bad ? 0.0f : (ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2);
    }
    if (lane == 0) s_ring.done(np);
    if (abort) {
      if (tid == 0) report_late(p, s_cur, b);
      break;
    }
  }
}

template <int D, bool E4M3, bool MOD, int NW, int NR>
cudaError_t launch(int ctas, const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedAttnParams& p,
                   cudaStream_t stream) {
  auto kernel = paged_rows_q8_kernel<D, E4M3, MOD, NW, NR>;
  if (!set_dyn_smem(kernel, RowsQ8Layout<D, NW>::kDyn)) return cudaErrorUnknown;
  return launch_pdl(kernel, dim3(ctas), dim3(32 * (NW + 2)), (size_t)RowsQ8Layout<D, NW>::kDyn, stream, tmK, tmV,
                    p);
}
template <int D, bool E4M3, bool MOD>
cudaError_t launch_kind(const PagedPlan& pl, const CUtensorMap& tmK, const CUtensorMap& tmV,
                        const PagedAttnParams& p, cudaStream_t stream) {
  const bool few = p.tq * p.G <= 8;
  if (pl.whole)
    return few ? launch<D, E4M3, MOD, 8, 8>(device_sm_count(), tmK, tmV, p, stream)
               : launch<D, E4M3, MOD, 8, 16>(device_sm_count(), tmK, tmV, p, stream);
  return few ? launch<D, E4M3, MOD, 4, 8>(pl.ctas, tmK, tmV, p, stream)
             : launch<D, E4M3, MOD, 4, 16>(pl.ctas, tmK, tmV, p, stream);
}
template <bool E4M3>
cudaError_t launch_format(const PagedPlan& pl, int D, bool mod, const CUtensorMap& tmK, const CUtensorMap& tmV,
                          const PagedAttnParams& p, cudaStream_t stream) {
  if (D == 128)
    return mod ? launch_kind<128, E4M3, true>(pl, tmK, tmV, p, stream)
               : launch_kind<128, E4M3, false>(pl, tmK, tmV, p, stream);
  return mod ? launch_kind<64, E4M3, true>(pl, tmK, tmV, p, stream)
             : launch_kind<64, E4M3, false>(pl, tmK, tmV, p, stream);
}

}  // namespace
}  // namespace paged
}  // namespace tv
