// paged_tc_kernel: units of up to 256 rows (two row blocks of 128 TMEM lanes, each nb =
// floor(128 / G) whole tokens) on the 5th-generation tensor cores.
//
// A CTA (one per SM) walks its share of the units, and a unit's keys from its last tile to
// its first: with a distance bias the scores fall that way, and the running maximum
// stays (the other way it moves with every tile, and O is scaled each time: a chunk of 2048 behind 6,100
// keys with slopes, now 178 us, went from 269 to 209 us by this alone).  Without slopes it takes
// 157 us, 79 % of the measured matrix rate: a tile of 256 rows takes some 2,850 cycles, its products
// 2,550 at that rate, and what a CTA does once (start, changes of unit, joining) some 14 us.
// 16 trees of 64 nodes stream their pages at 6.4 TB/s in the loop (75.6 us in all).  Warp roles:
//   warps 0-3, 4-7  softmax of row block 0, 1: one thread per row (TMEM lane), 128 scores a
//                   tile, online softmax in the log2 domain with lazy rescaling;
//   warp 8, 10      K and V tiles of 128 keys by TMA (a lane per box: 64 dims of the rows of
//                   one page), each into a ring of its own;
//   warp 9          the products: S_r = Q_r K^T and O_r += P_r V (tcgen05.mma, operands in
//                   shared memory but P, which is read from TMEM where it overlays S_r);
//   warp 11         walks the share and publishes its parts; the parts' Q rows.
// The products are issued in the order PV_0(t), S_0(t + 1), PV_1(t), S_1(t + 1): while one row
// block's softmax runs, the tensor core works on the other's.  S_r(t + 1) may
// overwrite P_r(t), as products retire in issue order.  The next unit's first S
// is issued while this one's epilogue still reads O: its first PV needs P, which the same
// threads write after the epilogue.  Every wait is bounded.
#define TV_UNIT 13
#include <climits>

#include "tv_attn_paged.cuh"

namespace tv {
namespace paged {
namespace {

constexpr int kTcThreads = 384;
constexpr int kRB = 128;           // rows of a row block
constexpr int kAtomBytes = 16384;  // 128 rows x 128 bytes
constexpr int kKStages = 2, kVStages = 3;
constexpr int kBadRing = 8;        // page flags outlive their K stage by two tiles at most

template <int D>
struct TcLayout {
  static constexpr int A = D / 64;
  static constexpr int kTile = A * kAtomBytes;  // one K or V tile, one row block of Q
  static constexpr int kK = 2 * kTile;
  static constexpr int kV = kK + kKStages * kTile;
  static constexpr int kDyn = kV + kVStages * kTile + 1024;
};

// kind::f16 with fp32 accumulators: c_format F32, a/b_format F16 (0) or BF16 (1), b_major
constexpr uint32_t idesc(bool f16, int N, int b_mn) {
  return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kRB >> 4) << 24);
}

// 8 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 32 bytes of a row in one store where rows lie on sectors (`whole`), else in two.
__device__ __forceinline__ void store32(uint8_t* at, const uint32_t (&x)[8], int whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(x[0]), "r"(x[1]),
                 "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(at)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<uint4*>(at)[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// What one row sees.
struct Row {
  const uint64_t* anc;  // mask row, or nullptr (causal)
  int limit;            // causal and prefix keys below it are visible ..
  int from;             // .. and at or past this one (the window)
  int pos;
};

// The row's mask for keys j .. j + 31.
__device__ __forceinline__ uint32_t tree32(const PagedAttnParams& p, const Row& r, int j, int L, int hi) {
  const int x = j - L;  // tree index of the first key
  return r.anc && x > -32 && j < hi ? anc_bits32(r.anc, p.W, x) & range_bits(0, hi - j) : 0u;
}

// Visibility of keys j .. j + 31 for a row (the window's reach inside a tree is
// taken in tree_chunk).
__device__ __forceinline__ uint32_t see32(const PagedAttnParams& p, const Row& r, int j, int L, int hi) {
  return range_bits(r.from - j, r.limit - j) | tree32(p, r, j, L, hi);
}

// x, scaled, less slope times distance; b0: the first key's bias.
__device__ __forceinline__ void bias_chunk(float b0, float slope, float in_scale, uint32_t (&x)[32]) {
  const float2 in2 = make_float2(in_scale, in_scale), slope2 = make_float2(slope, slope);
  const float2 b2 = make_float2(b0, b0);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float2 y = ffma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), in2,
                           ffma2(slope2, make_float2((float)e, (float)(e + 1)), b2));
    x[e] = __float_as_uint(y.x);
    x[e + 1] = __float_as_uint(y.y);
  }
}

// 32 keys from j that reach the tree: a node's position is its depth's, which the mask tells (v
// lacks the nodes whose page is none).  Clears v where the window does not reach, and adds the bias.
__device__ __forceinline__ void tree_chunk(const PagedAttnParams& p, const Row& r, int j, int L, int hi,
                                           float in_scale, float slope, uint32_t& v, uint32_t (&x)[32]) {
  const int a = j - L;  // tree index of the first key
  const int before = a > 0 ? anc_count(r.anc, p.W, min(a, 64 * p.W)) : 0;
  const uint32_t tree = tree32(p, r, j, L, hi);
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const int kpos = a + e < 0 ? j + e : L + before + __popc(tree & (0xffffffffu >> (31 - e))) - 1;
    if (p.window > 0 && r.pos - kpos >= p.window) v &= ~(1u << e);
    if (p.slopes)
      x[e] = __float_as_uint(fmaf(slope, (float)(kpos - r.pos), __uint_as_float(x[e]) * in_scale));
  }
}

// CAP: a softcap; BIAS: slopes, or tree distances that the window reaches.  Variants of
// their own, and rolled loops wherever a warp does not wait for them: a loop over the tiles that is
// larger than the instruction cache (some 32 KB) runs at half the speed.
template <int D, bool F16, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kTcThreads, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const PagedAttnParams p, const int nb) {
  using Lay = TcLayout<D>;
  constexpr int A = Lay::A;
  constexpr uint32_t kTmemCols = 512, kOCol = 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + Lay::kK;
  uint8_t* sV = smem + Lay::kV;
  __shared__ __align__(8) uint64_t bar_q_full, bar_q_empty, bar_drain;
  __shared__ __align__(8) uint64_t bar_k_full[kKStages], bar_k_empty[kKStages];
  __shared__ __align__(8) uint64_t bar_v_full[kVStages], bar_v_empty[kVStages];
  // (one per stage: the loads run up to three tiles ahead, and a barrier that is two phases
  // ahead of its reader cannot be told from one that is not ready)
  __shared__ __align__(8) uint64_t bar_v_zero[kVStages];
  __shared__ __align__(8) uint64_t bar_s_full[2], bar_p_full[2][2], bar_o_done[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile uint32_t s_bad_pages[kBadRing];  // bit g: keys 8 g .. 8 g + 7 have no page
  __shared__ volatile int s_abort;
  __shared__ PartRing s_ring;
  __shared__ Cursor<kTcKeys> s_cur;
  __shared__ int s_late;  // the first sequence that a softmax warp gave up in
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  if (tid == 0) {
    mbar_init(&bar_q_full, 1);
    mbar_init(&bar_q_empty, 1);
    mbar_init(&bar_drain, 1);
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&bar_k_full[i], 1);
      mbar_init(&bar_k_empty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&bar_v_full[i], 1);
      mbar_init(&bar_v_empty[i], 1);
      mbar_init(&bar_v_zero[i], 1);
    }
    for (int r = 0; r < 2; ++r) {
      mbar_init(&bar_s_full[r], 1);
      mbar_init(&bar_p_full[r][0], 4);  // one arrival a warp: those of 128 threads queue up
      mbar_init(&bar_p_full[r][1], 4);  // for some 400 cycles
      mbar_init(&bar_o_done[r], 1);
    }
    mbar_fence_init();
    s_abort = 0;
    s_late = INT_MAX;
    s_ring.init(11);  // K, V, products, eight softmax warps
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 0) tmem_alloc(&s_tmem, kTmemCols);
  prefetch_lengths<kTcThreads>(p);
  pdl_wait();
  tc_fence_before();
  find_share<kTcKeys, kTcThreads>(p, s_cur);
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  uint32_t n = 0;  // parts so far
  bool ok = true;
  if (warp == 8 || warp == 10) {
    // ------------------------------------------------------- K, V producers
    const bool isV = warp == 10;
    const CUtensorMap* map = isV ? &tmV : &tmK;
    uint8_t* ring = isV ? sV : sK;
    uint64_t* full = isV ? bar_v_full : bar_k_full;
    uint64_t* empty = isV ? bar_v_empty : bar_k_empty;
    const uint32_t stages = isV ? kVStages : kKStages;
    PageFeed<kTcKeys> feed;
    const int rows_page = min(1 << p.page_shift, kTcKeys), npg = kTcKeys / rows_page;
    const int pg = lane % npg, atom = lane / npg, row0 = pg * rows_page;
    const bool issues = atom < A;
    uint32_t it = 0;
    // Rows of V before lo and from hi on may hold anything (NaN times a probability of 0 is
    // NaN): cleared in the tiles that have them (a unit's first and last at most), once the
    // tile after them is on its way, or a part without tiles comes (the ring of parts moves on only
    // with the softmax warps, which wait for the products of that tile).
    uint32_t z_it = 0;
    int z0 = 0, z1 = kTcKeys;
    auto clear_rows = [&]() {
      if (z0 == 0 && z1 == kTcKeys) return;
      const uint32_t st = z_it % stages;
      ok = warp_wait(&full[st], (z_it / stages) & 1, p.wait_limit);
      for (int zr = lane >> 3; zr < kTcKeys; zr += 4)
        if (zr < z0 || zr >= z1)
#pragma unroll
          for (int a = 0; a < A; ++a)
            *reinterpret_cast<uint4*>(ring + st * Lay::kTile + a * kAtomBytes + zr * 128 +
                                      ((lane & 7) << 4)) = make_uint4(0, 0, 0, 0);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_v_zero[st]);
      z0 = 0;
      z1 = kTcKeys;
    };
    ok = p.wait_limit > 0;
    for (; ok; ++n) {
      ok = __all_sync(0xffffffffu, s_ring.ready(n, p.wait_limit));
      if (!ok) break;
      const Part w = s_ring.at(n);
      if (w.b < 0) break;
      if (isV && w.begin == w.end) clear_rows();
      feed.start(p, w);
      for (int t = w.end - 1; t >= w.begin; --t, ++it) {
        const uint32_t st = it % stages;
        const int key = t * kTcKeys + row0;
        uint32_t bad8;
        const int page = feed.get(p, w, t, pg, bad8);
        ok = warp_wait(&empty[st], ((it / stages) & 1) ^ 1, p.wait_limit) && !s_abort;
        if (!ok) break;
        if (lane == 0) {
          if (!isV) s_bad_pages[it % kBadRing] = bad8;
          mbar_expect_tx(&full[st], Lay::kTile);
        }
        __syncwarp();
        if (issues)
          tma_load_rows(ring + st * Lay::kTile + atom * kAtomBytes + row0 * 128, map, &full[st],
                        atom * 64, key & ((1 << p.page_shift) - 1), w.kvh, page, p.row_dim, p.head_dim);
        if (isV) {
          clear_rows();
          if (!ok) {
            ++it;  // (this tile's copy is on its way)
            break;
          }
          z_it = it;
          z0 = max(0, w.lo - t * kTcKeys);
          z1 = min(kTcKeys, w.hi - t * kTcKeys);
        }
      }
      if (lane == 0) s_ring.done(n);
    }
    if (isV && ok) clear_rows();
    // no copy may be in flight when the CTA leaves
    for (uint32_t i = it > stages ? it - stages : 0; i < it; ++i)
      mbar_wait(&full[i % stages], (i / stages) & 1);
  } else if (warp == 11) {
    // ------------------------------ the share's parts, and their Q rows
    uint32_t parts = 0;
    Part w;
    Cursor<kTcKeys> cur = s_cur;
    if (p.merge && lane == 0) p.desc[share_index()] = make_int4(0, 0, 0, 0);
    for (;; ++n) {
      const bool more = cur.next(p, w);
      ok = s_ring.publish(n, w, p.wait_limit);
      if (!ok || !more) break;
      if (p.merge && w.parts && lane == 0)
        p.desc[share_index()] = make_int4(w.s.t0 + w.first, w.ntok, w.kvh, w.parts);
      if (w.begin == w.end) continue;
      ok = warp_wait(&bar_q_empty, (parts & 1) ^ 1, p.wait_limit) && !s_abort;
      if (!ok) break;
      if (lane == 0) {
        const int nrb = w.ntok > nb ? 2 : 1;
        mbar_expect_tx(&bar_q_full, (uint32_t)(nrb * A * 64 * p.G * nb * 2));
        for (int r = 0; r < nrb; ++r)
#pragma unroll
          for (int a = 0; a < A; ++a)
            tma_load_3d(sQ + (r * A + a) * kAtomBytes, &tmQ, &bar_q_full, a * 64, w.kvh * p.G,
                        w.s.t0 + w.first + r * nb);
      }
      __syncwarp();
      ++parts;
    }
    if (!p.merge) write_status(p);
    if (parts > 0) mbar_wait(&bar_q_full, (parts - 1) & 1);
  } else if (warp == 9) {
    // ------------------------------------------------------------- products
    // One thread waits and issues: what it does between two products is on the critical
    // path of both row blocks (with the whole warp waiting and voting, a barrier that
    // had completed already cost some 150 cycles).
    if (elect_one()) {
      constexpr uint32_t idS = idesc(F16, kTcKeys, 0), idO = idesc(F16, D, 1);
      const uint64_t dQ = sw128_desc(smem_u32(sQ), 16, 1024);
      const uint64_t dK = sw128_desc(smem_u32(sK), 16, 1024);
      const uint64_t dV = sw128_desc(smem_u32(sV), kAtomBytes, 1024);
      uint32_t kst = 0, kph = 0, vst = 0, vph = 0, qph = 0, zph = 0, pph[2] = {0, 0};
      // S_r = Q_r K^T
      auto issue_s = [&](int r) {
        const uint64_t q = dQ + (uint64_t)(r * (Lay::kTile >> 4)), k = dK + (uint64_t)(kst * (Lay::kTile >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = ((kk >> 2) * kAtomBytes + (kk & 3) * 32) >> 4;
          mma_bf16(tmem + 128 * r, q + off, k + off, idS, kk > 0);
        }
        mma_commit(&bar_s_full[r]);
      };
      // O_r (+)= P_r V over the tile's first or last 64 keys
      auto issue_pv = [&](int r, int half, bool first) {
        const uint64_t v = dV + (uint64_t)(vst * (Lay::kTile >> 4) + half * 512);
        const uint32_t tP = tmem + 128 * r + 32 * half;
        mma_bf16_ts(tmem + kOCol + 128 * r, tP, v, idO, !first);
#pragma unroll
        for (int kk = 1; kk < kTcKeys / 32; ++kk)
          mma_bf16_ts(tmem + kOCol + 128 * r, tP + 8 * kk, v + (uint64_t)(kk * 128), idO, 1);
      };
      auto next_k = [&]() {
        kph ^= kst == kKStages - 1;
        kst = kst == kKStages - 1 ? 0 : kst + 1;
      };
      for (; ok; ++n) {
        ok = s_ring.ready(n, p.wait_limit);
        if (!ok) break;
        const Part w = s_ring.at(n);
        s_ring.done(n);
        if (w.b < 0) break;
        const int T = w.end - w.begin, nrb = w.ntok > nb ? 2 : 1;
        if (T == 0) continue;
        ok = wait_within(&bar_q_full, qph, p.wait_limit) && wait_within(&bar_k_full[kst], kph, p.wait_limit);
        if (!ok) break;
        qph ^= 1;
        tc_fence_after();
        for (int r = 0; r < nrb; ++r) issue_s(r);
        mma_commit(&bar_k_empty[kst]);
        next_k();
        if (T == 1) mma_commit(&bar_q_empty);
        for (int t = 0; t < T; ++t) {
          const int j0 = (w.end - 1 - t) * kTcKeys;
          const bool more = t + 1 < T;
          ok = wait_within(&bar_v_full[vst], vph, p.wait_limit);
          if (w.lo > j0 || w.hi < j0 + kTcKeys) {  // the V producer clears rows of this tile
            ok = ok && wait_within(&bar_v_zero[vst], (zph >> vst) & 1, p.wait_limit);
            zph ^= 1u << vst;
          }
          if (more) ok = ok && wait_within(&bar_k_full[kst], kph, p.wait_limit);
          for (int r = 0; ok && r < nrb; ++r) {
            ok = wait_within(&bar_p_full[r][0], pph[r], p.wait_limit);
            if (!ok) break;
            tc_fence_after();
            issue_pv(r, 0, t == 0);
            ok = wait_within(&bar_p_full[r][1], pph[r], p.wait_limit);
            if (!ok) break;
            pph[r] ^= 1;
            tc_fence_after();
            issue_pv(r, 1, false);
            if (more) issue_s(r);
            else mma_commit(&bar_o_done[r]);
          }
          if (!ok) break;
          mma_commit(&bar_v_empty[vst]);
          vph ^= vst == kVStages - 1;
          vst = vst == kVStages - 1 ? 0 : vst + 1;
          if (more) {
            mma_commit(&bar_k_empty[kst]);
            next_k();
          }
          if (t + 2 == T) mma_commit(&bar_q_empty);
        }
      }
      if (!ok) {
        (void)TV_CHECK(false);
        s_abort = 1;
      }
      mma_commit(&bar_drain);  // everything issued retires before TMEM is released
      if (!mbar_wait(&bar_drain, 0)) s_abort = 1;
    }
    ok = __all_sync(0xffffffffu, ok);
  } else {
    // -------------------------------------------------------------- softmax
    const int rb = warp >> 2, row = tid & (kRB - 1);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128 * rb, tO = tmem + kOCol + 128 * rb;
    const int tl = row / p.G, h_in = row % p.G;
    const bool warp_in_block = (warp & 3) * 32 < nb * p.G;
    uint32_t sc = 0, oc = 0, kt = 0;
    // Rows left for an earlier share are announced while the next part's first tile is under way:
    // the fence before the announcement waits for their stores, some 4,000 cycles right behind them.
    int left = -1;
    int b = s_cur.b;
    auto announce = [&]() {
      if (left >= 0) leave_rows(p, left, warp);
      left = -1;
    };
    for (; ok; ++n) {
      ok = __all_sync(0xffffffffu, s_ring.ready(n, p.wait_limit));
      if (!ok) break;
      const Part& w = s_ring.at(n);  // (stays in shared memory: the tiles need the registers)
      if (w.b < 0) break;
      b = w.b;
      const int T = w.end - w.begin;
      const int L = w.s.L, hi = w.hi, j_last = (w.end - 1) * kTcKeys;
      if (T == 0 || rb * nb >= w.ntok || rb * nb + (warp & 3) * 32 / p.G >= w.ntok) announce();  // (no tile of it here)
      if (T == 0) {  // a sequence with a status
        const int tile_tok = rb * nb + tl;
        const bool mine = tl < nb && tile_tok < w.ntok;
        const size_t oidx = (size_t)(w.s.t0 + w.first + tile_tok) * p.Hq + w.kvh * p.G + h_in;
        if (mine && TV_CHECK(oidx < (size_t)p.T * p.Hq)) {
          uint4* orow = reinterpret_cast<uint4*>(p.out + oidx * D);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) orow[c] = make_uint4(0, 0, 0, 0);
          if (p.lse) p.lse[oidx] = 0.0f;
        }
        __syncwarp();
        if (lane == 0) s_ring.done(n);
        continue;
      }
      if (rb * nb >= w.ntok) {  // no second row block
        kt += T;
        __syncwarp();
        if (lane == 0) s_ring.done(n);
        continue;
      }
      // rows past the unit take the last token's mask: computed, never written
      const int i = w.first + min(rb * nb + min(tl, nb - 1), w.ntok - 1);
      const bool warp_works = warp_in_block && rb * nb + (warp & 3) * 32 / p.G < w.ntok;
      Row r;
      r.anc = p.anc ? p.anc + (size_t)(w.s.t0 + i) * p.W : nullptr;
      r.pos = w.s.L + (p.anc ? anc_depth(r.anc, p.W) : i);
      r.limit = p.anc ? w.s.L : w.s.L + i + 1;
      r.from = p.window > 0 ? r.pos - p.window + 1 : 0;
      const float slope = (BIAS && p.slopes) ? __ldg(p.slopes + w.kvh * p.G + h_in) * kLog2e : 0.0f;
      // what turns a score into the log2 domain; capped scores are there already, and with
      // slopes it comes with the bias
      const float in_scale = CAP ? 1.0f : p.scale_log2;
      const float scale = (BIAS && p.slopes) ? 1.0f : in_scale;
      float m_run = -INFINITY, l_run = 0.0f;
      for (int t = 0; t < T; ++t, ++kt, ++sc) {
        const int j0 = j_last - t * kTcKeys;
        uint32_t vis[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (j0 + kTcKeys > r.limit || j0 < r.from) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const uint32_t v = see32(p, r, j0 + 32 * c, L, hi);
            if (c == 0) vis[0] = v;
            if (c == 1) vis[1] = v;
            if (c == 2) vis[2] = v;
            if (c == 3) vis[3] = v;
          }
        }
        ok = warp_wait(&bar_s_full[rb], sc & 1, p.wait_limit);
        if (!ok) break;
        if (!warp_works) {
          if (lane == 0) {
            mbar_arrive(&bar_p_full[rb][0]);
            mbar_arrive(&bar_p_full[rb][1]);
          }
          continue;
        }
        const uint32_t bad = s_bad_pages[kt % kBadRing];
        tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + lane_base + 32 * c, sr[c]);
        tmem_wait_ld();
        if (bad) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int g = 0; g < 4; ++g)
              if ((bad >> (4 * c + g)) & 1u) vis[c] &= ~(0xffu << (8 * g));
        }
        if (CAP) {
          float top = 0.0f;
          const float2 q0 = make_float2(p.cap_q[0], p.cap_q[0]), q1 = make_float2(p.cap_q[1], p.cap_q[1]);
          const float2 q2 = make_float2(p.cap_q[2], p.cap_q[2]), q3 = make_float2(p.cap_q[3], p.cap_q[3]);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 8) {  // four pairs step by step, so that their chains overlap
              float2 s[4], w[4], f[4];
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                s[b] = make_float2(__uint_as_float(sr[c][e + 2 * b]), __uint_as_float(sr[c][e + 2 * b + 1]));
                w[b] = fmul2(s[b], s[b]);
              }
#pragma unroll
              for (int b = 0; b < 4; ++b) f[b] = ffma2(q3, w[b], q2);
#pragma unroll
              for (int b = 0; b < 4; ++b) f[b] = ffma2(f[b], w[b], q1);
#pragma unroll
              for (int b = 0; b < 4; ++b) f[b] = ffma2(f[b], w[b], q0);
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                top = max3(top, w[b].x, w[b].y);
                f[b] = fmul2(s[b], f[b]);
                sr[c][e + 2 * b] = __float_as_uint(f[b].x);
                sr[c][e + 2 * b + 1] = __float_as_uint(f[b].y);
              }
            }
          // a warp with a score past the cubic's range takes all again, through TMEM (which
          // still holds them), to keep the code of this rare way small (rows past the unit and keys outside
          // of its range hold anything, and have no say in it)
          const bool is_row = tl < nb && rb * nb + tl < w.ntok;
          bool far = __any_sync(0xffffffffu, top > p.cap_top && is_row);
          if (far && (j0 < w.lo || j0 + kTcKeys > hi)) {
            top = 0.0f;
#pragma unroll 1
            for (int c = 0; c < 128; c += 8) {
              uint32_t x[8];
              tmem_ld8(tS + lane_base + c, x);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float y = __uint_as_float(x[e]);
                if (j0 + c + e >= w.lo && j0 + c + e < hi) top = fmaxf(top, y * y);
              }
            }
            far = __any_sync(0xffffffffu, top > p.cap_top && is_row);
          }
          if (far) {
            const float in = 2.0f * kLog2e * p.cap_in;
#pragma unroll 1
            for (int c = 0; c < 128; c += 8) {
              uint32_t x[8];
              tmem_ld8(tS + lane_base + c, x);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e)
                x[e] = __float_as_uint(p.softcap_log2 * tanh_any(__uint_as_float(x[e]) * in));
              tmem_st8(tS + lane_base + c, x);
            }
            tmem_wait_st();
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tS + lane_base + 32 * c, sr[c]);
            tmem_wait_ld();
          }
        }
        if (BIAS && r.anc && j0 + kTcKeys > L) {
          // the tile reaches the tree: also through TMEM
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_st32(tS + lane_base + 32 * c, sr[c]);
          tmem_wait_st();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32], v = c == 0 ? vis[0] : c == 1 ? vis[1] : c == 2 ? vis[2] : vis[3];
            tmem_ld32(tS + lane_base + 32 * c, x);
            tmem_wait_ld();
            tree_chunk(p, r, j0 + 32 * c, L, hi, in_scale, slope, v, x);
            tmem_st32(tS + lane_base + 32 * c, x);
            if (c == 0) vis[0] = v;
            if (c == 1) vis[1] = v;
            if (c == 2) vis[2] = v;
            if (c == 3) vis[3] = v;
          }
          tmem_wait_st();
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + lane_base + 32 * c, sr[c]);
          tmem_wait_ld();
        } else if (BIAS && p.slopes) {
          const float b0 = slope * (float)(j0 - r.pos);
#pragma unroll
          for (int c = 0; c < 4; ++c) bias_chunk(fmaf(slope, 32.0f * c, b0), slope, in_scale, sr[c]);
        }
        if ((vis[0] & vis[1] & vis[2] & vis[3]) != 0xffffffffu) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((vis[c] >> e) & 1u)) sr[c][e] = __float_as_uint(-INFINITY);
        }
        __syncwarp();
        // Probabilities of 32 keys against the maximum m: their sums into ps, packed pairs to pw.
        float2 ps[4] = {};
        const float2 sc2 = make_float2(scale, scale);
        auto probs = [&](int c, float m, uint32_t (&pw)[16]) {
          const float2 nm2 = make_float2(-m, -m);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = ffma2(make_float2(__uint_as_float(sr[c][2 * e]),
                                               __uint_as_float(sr[c][2 * e + 1])), sc2, nm2);
            const float2 x = make_float2(ex2(y.x), ex2(y.y));
            ps[e & 3] = fadd2(ps[e & 3], x);
            pw[e] = pack2<F16>(x.x, x.y);
          }
        };
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = __uint_as_float(sr[c][0]);
#pragma unroll
          for (int e = 1; e < 31; e += 2)
            mx[c] = max3(mx[c], __uint_as_float(sr[c][e]), __uint_as_float(sr[c][e + 1]));
          mx[c] = fmaxf(mx[c], __uint_as_float(sr[c][31]));
        }
        const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
        const bool moves = m_run == -INFINITY || tmax > m_run + kRescaleLog2;
        if (__any_sync(0xffffffffu, moves)) {
          const float m_new = moves ? tmax : m_run;
          const float corr = moves && m_run != -INFINITY ? ex2(m_run - m_new) : 1.0f;
          m_run = m_new;
          l_run *= corr;
          if (t > 0) {
            // O holds every tile up to t - 1: S(t) was issued after PV(t - 1) and has completed
#pragma unroll 1
            for (int c = 0; c < D; c += 8) {  // (few at a time: the scores hold the registers)
              uint32_t o[8];
              tmem_ld8(tO + lane_base + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              tmem_st8(tO + lane_base + c, o);
            }
          }
        }
        const float mm = m_run == -INFINITY ? 0.0f : m_run;  // nothing seen yet: 2^-inf = 0
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          // (rounded to the cache's type, the product's operand: half a step, 2^-8 or 2^-11 of a
          // probability; the sums take them as they were)
          uint32_t pw[16];
          probs(c, mm, pw);
          tmem_st16(tS + lane_base + 16 * c, pw);
          if (c & 1) {  // 64 keys are there: their product may start
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_p_full[rb][c >> 1]);
          }
        }
        announce();
        const float2 pa = fadd2(fadd2(ps[0], ps[1]), fadd2(ps[2], ps[3]));
        l_run += pa.x + pa.y;
      }
      if (ok) ok = warp_wait(&bar_o_done[rb], oc & 1, p.wait_limit);
      if (!ok) break;
      ++oc;
      tc_fence_after();
      if (!warp_works) {
        if (lane == 0) s_ring.done(n);
        continue;
      }
      // ------------------------------------------------------- epilogue
      const int tile_tok = rb * nb + tl;
      const bool mine = tl < nb && tile_tok < w.ntok;
      const size_t oidx = (size_t)(w.s.t0 + w.first + tile_tok) * p.Hq + w.kvh * p.G + h_in;
      const int crow = rb * kRB + row;
      const bool leaves = w.slot >= 0 && (p.merge || w.parts == 0);  // rows for another to join
      float4* part = reinterpret_cast<float4*>(p.part) + crow;       // [slot][D / 4][256]
      if (leaves) {
        if (mine) p.part_ml[(size_t)w.slot * 256 + crow] = make_float2(m_run, l_run);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + lane_base + 32 * c, o);
          tmem_wait_ld();
          if (mine)
#pragma unroll
            for (int q = 0; q < 8; ++q)
              part[((size_t)w.slot * (D / 4) + 8 * c + q) * 256] =
                  make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
                              __uint_as_float(o[4 * q + 2]), __uint_as_float(o[4 * q + 3]));
          __syncwarp();
        }
        if (!p.merge) left = w.slot;
      } else {
        // the rows of the shares that went on with the unit, then the output
        const int more = w.slot >= 0 ? w.parts - 1 : 0;
        float m_all = m_run, l_all = l_run;
        for (int k = 1; ok && k <= more; ++k) {
          ok = await_rows(p, w.slot + k, warp);
          const float2 ml = ok && mine ? __ldcg(&p.part_ml[(size_t)(w.slot + k) * 256 + crow])
                                       : make_float2(-INFINITY, 0.0f);
          // (maxima leave a NaN out, sums carry it: 0 times NaN is NaN)
          const float top = fmaxf(m_all, ml.x);
          l_all = fmaf(m_all == -INFINITY ? 0.0f : ex2(m_all - top), l_all,
                       (ml.x == -INFINITY ? 0.0f : ex2(ml.x - top)) * ml.y);
          m_all = top;
        }
        if (!ok) break;
        const float f0 = m_run == -INFINITY ? 0.0f : ex2(m_run - m_all);
        const float inv = l_all == 0.0f ? 0.0f : 1.0f / l_all;
        uint8_t* orow = reinterpret_cast<uint8_t*>(p.out + oidx * D);
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o[2][32];
          tmem_ld32(tO + lane_base + 64 * c, o[0]);
          tmem_ld32(tO + lane_base + 64 * c + 32, o[1]);
          tmem_wait_ld();
          if (more && mine) {
#pragma unroll
            for (int e = 0; e < 64; ++e)
              o[e >> 5][e & 31] = __float_as_uint(__uint_as_float(o[e >> 5][e & 31]) * f0);
#pragma unroll 1
            for (int k = 1; k <= more; ++k) {
              const float m = __ldcg(&p.part_ml[(size_t)(w.slot + k) * 256 + crow].x);
              float4 v[16];
#pragma unroll
              for (int q = 0; q < 16; ++q)
                v[q] = __ldcg(&part[((size_t)(w.slot + k) * (D / 4) + 16 * c + q) * 256]);
              const float f = m == -INFINITY ? 0.0f : ex2(m - m_all);
              if (f == 0.0f) continue;  // (a part whose keys are all hidden: select, do not multiply)
#pragma unroll
              for (int q = 0; q < 16; ++q) {
                uint32_t* x = &o[q >> 3][4 * (q & 7)];
                x[0] = __float_as_uint(fmaf(f, v[q].x, __uint_as_float(x[0])));
                x[1] = __float_as_uint(fmaf(f, v[q].y, __uint_as_float(x[1])));
                x[2] = __float_as_uint(fmaf(f, v[q].z, __uint_as_float(x[2])));
                x[3] = __float_as_uint(fmaf(f, v[q].w, __uint_as_float(x[3])));
              }
            }
          }
          if (mine && TV_CHECK(oidx < (size_t)p.T * p.Hq))
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // 16 columns: 32 bytes, a whole sector at a time
              uint32_t x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                x[e] = pack2<F16>(__uint_as_float(o[q >> 1][16 * (q & 1) + 2 * e]) * inv,
                                  __uint_as_float(o[q >> 1][16 * (q & 1) + 2 * e + 1]) * inv);
              store32(orow + 128 * c + 32 * q, x, p.out_sectors);
            }
          __syncwarp();
        }
        if (mine && p.lse) p.lse[oidx] = l_all == 0.0f ? -INFINITY : (m_all + log2f(l_all)) * kLn2;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) s_ring.done(n);
    }
    announce();
    if (!ok && lane == 0) atomicMin(&s_late, b);  // (what other roles did not do, these warps waited for)
  }
  if (!ok) s_abort = 1;
  tc_fence_before();
  __syncthreads();  // every role is done; TMA and MMA work has retired
  if (tid == 0 && s_late != INT_MAX) report_late(p, s_cur, s_late);
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

template <int D, bool F16, bool CAP, bool BIAS>
cudaError_t launch(const PagedPlan& pl, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                   const CUtensorMap& tmV, const PagedAttnParams& p, cudaStream_t stream) {
  if (!set_dyn_smem(paged_tc_kernel<D, F16, CAP, BIAS>, TcLayout<D>::kDyn)) return cudaErrorUnknown;
  return launch_pdl(paged_tc_kernel<D, F16, CAP, BIAS>, dim3(pl.ctas), dim3(kTcThreads),
                    (size_t)TcLayout<D>::kDyn, stream, tmQ, tmK, tmV, p, pl.nb);
}
template <int D, bool F16>
cudaError_t launch_kind(const PagedPlan& pl, bool bias, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                        const CUtensorMap& tmV, const PagedAttnParams& p, cudaStream_t stream) {
  if (p.softcap_log2 > 0.0f)
    return bias ? launch<D, F16, true, true>(pl, tmQ, tmK, tmV, p, stream)
                : launch<D, F16, true, false>(pl, tmQ, tmK, tmV, p, stream);
  return bias ? launch<D, F16, false, true>(pl, tmQ, tmK, tmV, p, stream)
              : launch<D, F16, false, false>(pl, tmQ, tmK, tmV, p, stream);
}

}  // namespace

cudaError_t launch_tc(const PagedPlan& pl, int D, bool f16, bool bias, const CUtensorMap& tmQ,
                      const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedAttnParams& p,
                      cudaStream_t stream) {
  if (D == 128)
    return f16 ? launch_kind<128, true>(pl, bias, tmQ, tmK, tmV, p, stream)
               : launch_kind<128, false>(pl, bias, tmQ, tmK, tmV, p, stream);
  return f16 ? launch_kind<64, true>(pl, bias, tmQ, tmK, tmV, p, stream)
             : launch_kind<64, false>(pl, bias, tmQ, tmK, tmV, p, stream);
}

}  // namespace paged
}  // namespace tv
