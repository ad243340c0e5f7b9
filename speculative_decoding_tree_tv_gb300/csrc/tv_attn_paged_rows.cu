// paged_rows_kernel: units of at most 16 rows.  HBM-bound: per 64-key stage a CTA reads 64 D * 4
// bytes and issues D warp mma (D / 2 with at most 8 rows).  Four consumer warps take 16 keys of
// a stage each and keep a running maximum, sum and output of their own (no barrier
// between them until the unit's end); two more warps issue the TMA loads of K and V, one box
// per lane (64 dims x the rows of a page): a warp issues a box in some 57 cycles, which with pages of 16
// rows and one warp for both held 4 short sequences at 13.5 us, now 11.8.
// A decode of 64 sequences (1.23 GB of cache) takes 186 us, 97 % of what a copy reaches.
#define TV_UNIT 12
#include "tv_warp_mma.cuh"

namespace tv {
namespace paged {
namespace {

constexpr int kUnitRows = 16;  // rows of a slot

// NR: the most rows of a unit.  16: S = Q K^T and O = P V, rows in the mma's 16.  8: S^T = K Q^T and
// O^T = V^T P^T, keys and dims in its 16 and rows in its 8, so half the products and half the
// exponentials (4 short sequences 11.8 -> 10.6 us, a decode of 64 at D 64 107 -> 102 us, capped in
// a window 64 -> 53 us).
// NW consumer warps, 16 keys of a stage each: 4 and two CTAs an SM, which fill it when there is work
// for all, or 8 and one CTA where every unit has an SM to itself (p.whole).
template <int D, int NW>
struct RowsLayout {
  static constexpr int kKeys = 16 * NW;
  static constexpr int kAtoms = D / 64;
  static constexpr int kAtom = kKeys * 128;         // bytes of one 64-dim atom of a stage
  static constexpr int kSide = kAtoms * kAtom;      // K or V of a stage
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kScratch = NW * 16 * 32 * 4;  // [warp][row][32 dims]
  static constexpr int kDyn = 2 * kStages * kSide + kScratch + 1024;
};

// Column order of a row of s_acc: neither the stores (NR 16: 8 rows of 8 floats, NR 8: every other
// row, 8 floats) nor the loads (a row) meet in a bank.
template <int NR>
__device__ __forceinline__ int acc_swizzle(int row) {
  return NR == 16 ? ((row & 3) << 3) | (row & 4) : ((row & 6) << 2) | ((row & 1) << 2);
}
template <int D, bool F16, bool MOD, int NW, int NR>
__global__ void __launch_bounds__(32 * (NW + 2), NW == 4 ? 2 : 1)
paged_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const PagedAttnParams p) {
  using Lay = RowsLayout<D, NW>;
  constexpr int kSteps = D / 16, kRowsWarps = NW, kRowsKeys = 16 * NW, kRowsThreads = 32 * (NW + 2);
  constexpr int kStages = Lay::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sK = smem;
  uint8_t* sV = smem + kStages * Lay::kSide;
  // the unit's Q rows; at its end the warps' outputs (32 dims at a time)
  uint4* s_q = reinterpret_cast<uint4*>(smem + 2 * kStages * Lay::kSide);
  float* s_acc = reinterpret_cast<float*>(s_q);
  __shared__ __align__(8) uint64_t bar_full[kStages], bar_empty[kStages];
  __shared__ uint32_t s_bad_pages[kStages];  // bit g: keys 8 g .. 8 g + 7 have no page
  __shared__ float2 s_ml[kRowsWarps][kUnitRows];
  __shared__ volatile int s_abort;  // a consumer's wait ran out
  __shared__ PartRing s_ring;
  __shared__ Cursor<kRowsKeys> s_cur;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  if (tid == 0) {
    s_abort = 0;
    s_ring.init(kRowsWarps + 1);  // V, consumers
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar_full[s], 2);
      mbar_init(&bar_empty[s], kRowsWarps);
    }
    mbar_fence_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  prefetch_lengths<kRowsThreads>(p);
  pdl_wait();
  find_share<kRowsKeys, kRowsThreads>(p, s_cur);
  uint32_t st = 0, phase = 0, np = 0;  // stage, its ring's phase; parts so far
  auto next_stage = [&]() {
    phase ^= st == kStages - 1;
    st = st == kStages - 1 ? 0 : st + 1;
  };

  if (warp >= kRowsWarps) {
    // ------------------------------------------------- K, V producers
    // (K's also walks the share)
    const bool isV = warp > kRowsWarps;
    const CUtensorMap* map = isV ? &tmV : &tmK;
    uint8_t* ring = isV ? sV : sK;
    Part w;
    Cursor<kRowsKeys> cur = s_cur;
    if (p.merge && !isV && lane == 0) p.desc[share_index()] = make_int4(0, 0, 0, 0);
    PageFeed<kRowsKeys> feed;
    const int rows_page = min(1 << p.page_shift, kRowsKeys);  // rows of one box
    uint32_t issued = 0;
    const int npg = kRowsKeys / rows_page;
    const int pg = lane % npg, atom = lane / npg, row0 = pg * rows_page;
    const bool issues = atom < Lay::kAtoms;
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
        const int row = (t * kRowsKeys + row0) & ((1 << p.page_shift) - 1);
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
          tma_load_rows(ring + st * Lay::kSide + atom * Lay::kAtom + row0 * 128, map, &bar_full[st],
                        atom * 64, row, w.kvh, page, p.row_dim, p.head_dim);
        next_stage();
        ++issued;
      }
      if (!ok) break;
    }
    if (!p.merge && !isV) write_status(p);
    // no copy may be in flight when the CTA leaves (where the other producer gave up, its half of a
    // stage never comes: this one's has landed long before the limit)
    for (uint32_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
      if (!mbar_wait(&bar_full[i % kStages], (i / kStages) & 1)) break;
    return;  // (what a producer that gave up did not load, the consumers wait for in vain, and report)
  }

  // ---------------------------------------------------------------- consumers
  const float cap_in2 = 2.0f * kLog2e * p.cap_in;
  const int g = lane >> 2, c2 = (lane & 3) * 2;  // fragment row and first column of this lane
  // A lane's two rows, and the kKeys keys of 16 that it holds of both
  constexpr int kKeys = NR == 16 ? 4 : 2, kScores = 2 * kKeys;
  constexpr int kQRegs = kSteps * (NR == 16 ? 4 : 2), kAcc = NR == 16 ? D / 8 : D / 16;
  auto row_of = [&](int r) { return NR == 16 ? r * 8 + g : c2 + r; };
  auto key_of = [&](int i) { return NR == 16 ? 8 * (i >> 1) + c2 + (i & 1) : 8 * i + g; };
  auto at = [](int r, int i) { return NR == 16 ? 4 * (i >> 1) + 2 * r + (i & 1) : 2 * i + r; };
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
    named_sync(1, kRowsWarps * 32);
    if (s_abort) {
      if (tid == 0) report_late(p, s_cur, b);
      break;
    }
    const Part w = s_ring.at(np);
    if (w.b < 0) break;
    b = w.b;
    const int rows = w.ntok * p.G;
    // the unit's Q rows to shared memory (rows past the unit repeat its last one); 16-byte
    // chunk c of row r lies at c ^ (r & 7)
    for (int x = tid; x < NR * (D / 8); x += kRowsWarps * 32) {
      const int r = x / (D / 8), c = x % (D / 8), row = min(r, rows - 1);
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (w.s.t0 + w.first + row / p.G) * p.q_token_stride +
          (w.kvh * p.G + row % p.G) * p.q_head_stride);
      s_q[r * (D / 8) + (c ^ (r & 7))] = __ldg(src + c);
    }
    named_sync(1, kRowsWarps * 32);
    uint32_t qf[kQRegs / 4][4];  // (NR 8: two steps' fragments together)
    {
      const int row8 = NR == 16 ? ((lane >> 3) & 1) * 8 : 0, chunk = NR == 16 ? lane >> 4 : lane >> 3;
      const uint32_t base = smem_u32(s_q) + ((lane & 7) + row8) * (D * 2);
#pragma unroll
      for (int k = 0; k < kQRegs / 4; ++k)
        ldsm4(base + (((NR / 8 == 2 ? 2 * k : 4 * k) + chunk) ^ (lane & 7)) * 16, qf[k]);
    }
    int pos[2], tok[2];
    float slope[2];
    float m[2], l[2], o[kAcc][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = min(row_of(r), rows - 1);  // rows past the unit repeat its last
      const int i = w.first + row / p.G, t = w.s.t0 + i, h = w.kvh * p.G + row % p.G;
      tok[r] = t;
      pos[r] = w.s.L + (p.anc ? anc_depth(p.anc + (size_t)t * p.W, p.W) : i);
      slope[r] = (MOD && p.slopes) ? __ldg(p.slopes + h) * kLog2e : 0.0f;
      m[r] = -INFINITY;
      l[r] = 0.0f;
    }
#pragma unroll
    for (int n = 0; n < kAcc; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    const int all_below = p.anc ? w.s.L : w.s.L + w.first + 1;  // keys below it are visible to every row
    const int all_from = p.window > 0
                             ? (p.anc ? w.s.L + w.s.n : w.s.L + w.first + w.ntok) - p.window : -1;

    for (int t = w.end - 1; t >= w.begin; --t) {  // (last first: see paged_tc_kernel)
      const int j0 = t * kRowsKeys + 16 * warp;
      if (!warp_wait(&bar_full[st], phase, p.wait_limit)) {
        s_abort = 1;
        break;
      }
      if (j0 < w.hi && j0 + 16 > w.lo) {
        float s[8] = {};
        if (NR == 16) {  // S: [8 keys][row g: two keys, row g + 8: two keys]
          const int key = 16 * warp + (lane >> 4) * 8 + (lane & 7);
          const uint32_t base = smem_u32(sK) + st * Lay::kSide + key * 128;
          const int kc = (lane >> 3) & 1, sw = key & 7;
          float (&s0)[4] = reinterpret_cast<float (&)[4]>(s[0]), (&s1)[4] = reinterpret_cast<float (&)[4]>(s[4]);
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            uint32_t b[4];
            ldsm4(base + (k >> 2) * Lay::kAtom + ((((k & 3) * 2 + kc) ^ sw) << 4), b);
            mma16816<F16>(s0, qf[NR == 16 ? k : 0], b[0], b[1]);
            mma16816<F16>(s1, qf[NR == 16 ? k : 0], b[2], b[3]);
          }
        } else {  // S^T: [key g: two rows, key g + 8: two rows], even and odd steps apart
          const int key = 16 * warp + ((lane >> 3) & 1) * 8 + (lane & 7);
          const uint32_t base = smem_u32(sK) + st * Lay::kSide + key * 128;
          const int kc = lane >> 4, sw = key & 7;
          float (&s0)[4] = reinterpret_cast<float (&)[4]>(s[0]), (&s1)[4] = reinterpret_cast<float (&)[4]>(s[4]);
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            uint32_t a[4];
            ldsm4(base + (k >> 2) * Lay::kAtom + ((((k & 3) * 2 + kc) ^ sw) << 4), a);
            mma16816<F16>(k & 1 ? s1 : s0, a, qf[k / 2][2 * (k & 1)], qf[k / 2][2 * (k & 1) + 1]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) s[e] += s[4 + e];
        }
        const uint32_t bad8 = (s_bad_pages[st] >> (2 * warp)) & 3u;
        const bool plain = j0 + 16 <= all_below && j0 > all_from && j0 >= w.lo && bad8 == 0;
        uint32_t vkeep[2] = {0xffffffffu, 0xffffffffu};  // V pairs of keys that some row sees
        if (!plain) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int j = j0 + 8 * nt + c2 + e;
              if (j < w.lo || j >= w.hi) vkeep[nt] &= e ? 0x0000ffffu : 0xffff0000u;
            }
        }
        // scores in the log2 domain, hidden keys at -inf
        if (MOD && p.softcap_log2 > 0.0f) {
          float f[kScores], top = 0.0f;
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
              const float x = s[at(r, i)], w2 = x * x;
              const int j = j0 + key_of(i);  // (keys outside of the unit's range hold anything)
              if (plain || (j >= w.lo && j < w.hi)) top = fmaxf(top, w2);
              f[at(r, i)] = x * fmaf(fmaf(fmaf(p.cap_q[3], w2, p.cap_q[2]), w2, p.cap_q[1]), w2, p.cap_q[0]);
            }
          const bool far = __any_sync(0xffffffffu, top > p.cap_top);
#pragma unroll
          for (int e = 0; e < kScores; ++e) s[e] = far ? p.softcap_log2 * tanh_any(s[e] * cap_in2) : f[e];
        } else {
#pragma unroll
          for (int e = 0; e < kScores; ++e) s[e] *= p.scale_log2;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < kKeys; ++i) {
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
              if ((bad8 >> (NR == 16 ? i >> 1 : i)) & 1) see = false;
              if (MOD) x = fmaf(slope[r], (float)(kpos - pos[r]), x);
              if (!see) x = -INFINITY;
            } else if (MOD) {
              x = fmaf(slope[r], (float)(kpos - pos[r]), x);
            }
          }
        // running maximum (lazily moved), probabilities, sums
        float corr[2];
        bool move = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float mx = s[at(r, 0)];
#pragma unroll
          for (int i = 1; i < kKeys; ++i) mx = fmaxf(mx, s[at(r, i)]);
          mx = reduce(mx, [](float a, float b) { return fmaxf(a, b); });
          corr[r] = 1.0f;
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
          for (int i = 0; i < kKeys; ++i) sum += s[at(r, i)] = ex2(s[at(r, i)] - mm);
          l[r] = fmaf(l[r], corr[r], sum);
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int n = 0; n < kAcc; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] *= corr[NR == 16 ? e >> 1 : e & 1];
        }
        // P is rounded to the cache's type for the product (half a step: 2^-8 or 2^-11 of a probability); the
        // sums took it as it was
        if (NR == 16) {  // O += P V
          const uint32_t pf[4] = {pack2<F16>(s[0], s[1]), pack2<F16>(s[2], s[3]), pack2<F16>(s[4], s[5]),
                                  pack2<F16>(s[6], s[7])};
          const int key = 16 * warp + ((lane >> 3) & 1) * 8 + (lane & 7);
          const uint32_t base = smem_u32(sV) + st * Lay::kSide + key * 128;
          const int dc = lane >> 4, sw = key & 7;
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            uint32_t b[4];
            ldsm4_t(base + (n >> 2) * Lay::kAtom + ((((n & 3) * 2 + dc) ^ sw) << 4), b);
            if (!plain) {
#pragma unroll
              for (int q = 0; q < 4; ++q) b[q] &= vkeep[q & 1];
            }
            mma16816<F16>(o[(2 * n) % kAcc], pf, b[0], b[1]);
            mma16816<F16>(o[(2 * n + 1) % kAcc], pf, b[2], b[3]);
          }
        } else {  // O^T += V^T P^T
          const uint32_t p0 = transpose8(pack2<F16>(s[0], s[1])), p1 = transpose8(pack2<F16>(s[2], s[3]));
          const int key = 16 * warp + (lane >> 4) * 8 + (lane & 7);
          const uint32_t base = smem_u32(sV) + st * Lay::kSide + key * 128;
          const int dc = (lane >> 3) & 1, sw = key & 7;
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            uint32_t a[4];
            ldsm4_t(base + (n >> 2) * Lay::kAtom + ((((n & 3) * 2 + dc) ^ sw) << 4), a);
            if (!plain) {
#pragma unroll
              for (int q = 0; q < 4; ++q) a[q] &= vkeep[q >> 1];
            }
            mma16816<F16>(o[n], a, p0, p1);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_empty[st]);
      next_stage();
    }

    // the four warps' rows joined in shared memory, 32 dims at a time
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] = reduce(l[r], [](float a, float b) { return a + b; });
      if (NR == 16 ? (lane & 3) == 0 : lane < 4) s_ml[warp][row_of(r)] = make_float2(m[r], l[r]);
    }
    named_sync(1, kRowsWarps * 32);
    const bool abort = s_abort;
    float f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mm = -INFINITY;
#pragma unroll
      for (int x = 0; x < kRowsWarps; ++x) mm = fmaxf(mm, s_ml[x][row_of(r)].x);
      f[r] = m[r] == -INFINITY ? 0.0f : ex2(m[r] - mm);  // (0: nothing seen by this warp, its sums are 0)
    }
    const int row = (tid >> 3) & (NR - 1), od = (tid & 7) * 4;  // this thread's row and dims of a joined piece
    float mm = -INFINITY, ll = 0.0f;
#pragma unroll
    for (int x = 0; x < kRowsWarps; ++x) mm = fmaxf(mm, s_ml[x][row].x);
#pragma unroll
    for (int x = 0; x < kRowsWarps; ++x) {
      const float2 v = s_ml[x][row];
      ll = fmaf(v.x == -INFINITY ? 0.0f : ex2(v.x - mm), v.y, ll);  // (a NaN stays: maxima leave it out, sums do not)
    }
    const bool mine = tid < 8 * NR && row < rows;
    const int out_tok = w.s.t0 + w.first + row / p.G, h = w.kvh * p.G + row % p.G;
    const size_t oidx = (size_t)out_tok * p.Hq + h;
    const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
#pragma unroll
      for (int x = 0; x < kAcc * 32 / D; ++x) {
        const float(&v)[4] = o[c * (kAcc * 32 / D) + x];
        if (NR == 16) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float2*>(s_acc + (warp * 16 + r * 8 + g) * 32 + ((8 * x + c2) ^ acc_swizzle<NR>(g))) =
                make_float2(v[2 * r] * f[r], v[2 * r + 1] * f[r]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s_acc[(warp * 16 + c2 + (e & 1)) * 32 + ((16 * x + 8 * (e >> 1) + g) ^ acc_swizzle<NR>(c2 + (e & 1)))] =
                v[e] * f[e & 1];
        }
      }
      named_sync(1, kRowsWarps * 32);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kRowsWarps; ++x) {
        const float4 v = *reinterpret_cast<const float4*>(s_acc + (x * 16 + row) * 32 + (od ^ acc_swizzle<NR>(row)));
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
      if (mine) {
        if (w.slot >= 0)
          *reinterpret_cast<float4*>(p.part + ((size_t)w.slot * kUnitRows + row) * D + 32 * c + od) = a;
        else if (TV_CHECK(out_tok < p.T && h < p.Hq))
          *reinterpret_cast<uint2*>(p.out + oidx * D + 32 * c + od) =
              make_uint2(pack2<F16>(a.x * inv, a.y * inv), pack2<F16>(a.z * inv, a.w * inv));
      }
      named_sync(1, kRowsWarps * 32);
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

template <int D, bool F16, bool MOD, int NW, int NR>
cudaError_t launch(int ctas, const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedAttnParams& p,
                   cudaStream_t stream) {
  auto kernel = paged_rows_kernel<D, F16, MOD, NW, NR>;
  if (!set_dyn_smem(kernel, RowsLayout<D, NW>::kDyn)) return cudaErrorUnknown;
  return launch_pdl(kernel, dim3(ctas), dim3(32 * (NW + 2)), (size_t)RowsLayout<D, NW>::kDyn, stream, tmK, tmV, p);
}
template <int D, bool F16, bool MOD>
cudaError_t launch_kind(const PagedPlan& pl, const CUtensorMap& tmK, const CUtensorMap& tmV,
                        const PagedAttnParams& p, cudaStream_t stream) {
  const bool few = p.tq * p.G <= 8;
  if (pl.whole)
    return few ? launch<D, F16, MOD, 8, 8>(device_sm_count(), tmK, tmV, p, stream)
               : launch<D, F16, MOD, 8, 16>(device_sm_count(), tmK, tmV, p, stream);
  return few ? launch<D, F16, MOD, 4, 8>(pl.ctas, tmK, tmV, p, stream)
             : launch<D, F16, MOD, 4, 16>(pl.ctas, tmK, tmV, p, stream);
}

}  // namespace

cudaError_t launch_rows(const PagedPlan& pl, int D, bool f16, bool mod, const CUtensorMap& tmK,
                        const CUtensorMap& tmV, const PagedAttnParams& p, cudaStream_t stream) {
  if (D == 128) {
    if (f16) return mod ? launch_kind<128, true, true>(pl, tmK, tmV, p, stream)
                        : launch_kind<128, true, false>(pl, tmK, tmV, p, stream);
    return mod ? launch_kind<128, false, true>(pl, tmK, tmV, p, stream)
               : launch_kind<128, false, false>(pl, tmK, tmV, p, stream);
  }
  if (f16) return mod ? launch_kind<64, true, true>(pl, tmK, tmV, p, stream)
                      : launch_kind<64, true, false>(pl, tmK, tmV, p, stream);
  return mod ? launch_kind<64, false, true>(pl, tmK, tmV, p, stream)
             : launch_kind<64, false, false>(pl, tmK, tmV, p, stream);
}

}  // namespace paged
}  // namespace tv
