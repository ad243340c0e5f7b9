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
//   warp 11         walks the share and publishes its parts; the parts' Q rows;
//   warps 12-19     over an 8-bit cache: tiles of codes, which land in the second half of their
//                   stage, become fp16 tiles in place (warps 8 and 10 look at their scales ahead of that).
// 8-bit tiles take 4,400 cycles (the section on them tells why): 16 trees of 64 nodes 103 us with e4m3 and 104 with int8, a
// chunk of 2,048 behind 6,100 keys 236 and 242 us, where a 16-bit cache takes 76 and 157.
// The products are issued in the order PV_0(t), S_0(t + 1), PV_1(t), S_1(t + 1): while one row
// block's softmax runs, the tensor core works on the other's.  S_r(t + 1) may
// overwrite P_r(t), as products retire in issue order.  The next unit's first S
// is issued while this one's epilogue still reads O: its first PV needs P, which the same
// threads write after the epilogue.  Every wait is bounded.
#pragma once

#include <cfloat>
#include <climits>

#include "tv_attn_paged.cuh"
#include "tv_quant.cuh"

namespace tv {
namespace paged {
namespace {

constexpr int kTcThreads = 384, kConvertThreads = 256;  // (those: over an 8-bit cache)
constexpr int kRB = 128;           // rows of a row block
constexpr int kAtomBytes = 16384;  // 128 rows x 128 bytes
constexpr int kKStages = 2, kVStages = 3;
constexpr int kBadRing = 8;        // page flags outlive their K stage by two tiles at most
constexpr int kExpRing = 4;        // and what an 8-bit tile's K and V are held over, V's stage by none

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

// Row of token i (of the sequence) of a part; `shared`: of a prefix, whose rows are several sequences', behind all keys.
__device__ __forceinline__ Row row_of(const PagedAttnParams& p, const Part& w, int i, bool shared) {
  Row r;
  r.anc = p.anc && !shared ? p.anc + (size_t)(w.s.t0 + i) * p.W : nullptr;
  r.pos = shared ? prefix_pos(p, w.b, w.s.t0 + i, w.s.L) : w.s.L + (p.anc ? anc_depth(r.anc, p.W) : i);
  r.limit = shared || p.anc ? w.s.L : w.s.L + i + 1;
  r.from = p.window > 0 ? r.pos - p.window + 1 : 0;
  return r;
}

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

// Where the kernel that joins rows finds those of a unit (its first part's warp).
__device__ __forceinline__ void note_unit(const PagedAttnParams& p, const Part& w) {
  int4* src = p.src + (w.s.shared ? 0 : (size_t)p.T * p.Hkv);
  for (int i = threadIdx.x & 31; i < w.ntok; i += 32) {
    const int t = w.s.t0 + w.first + i;
    if (TV_IN(t, p.T))
      src[(size_t)t * p.Hkv + w.kvh] =
          make_int4(w.slot, w.parts, w.s.t0 + w.first, w.s.shared ? w.b : w.b - p.groups);
  }
}

// ------------------------------------------------------------- 8-bit tiles
// A raw tile of 128 rows of D codes lands in the second half of its stage, and the 16-bit tile is written over the
// whole stage, in the layout that TMA gives a 16-bit cache's: 64 rows a pass, whose place holds no codes but their own
// and ones that have been taken.  256 threads take a pass's codes into registers, and then write them; a thread has the
// 16 codes of chunk ctid % (D / 16) of rows unit_row + i kRowStep, whose places differ by a multiple of the swizzle's
// period.  What bounds it is the SM's instruction cache: the roles' code does not fit (92 to 95 % of the fetches hit,
// 98 % without this role), every warp waits for instructions, and a tile of 256 rows takes 4,400 cycles instead of
// 2,850.  So K and V share their code, and a pass is half a tile.  16 trees of 64 at 4 warps 174 us, at 8 146, with K
// in fp16 like V 108, with the scales looked at by the warps that load 105, two passes 103 (a chunk of 2,048 behind
// 6,100: 458, 323, 247, 226, 226).  Four warps a side, codes in places of their own with one tile ahead, or a pass of a
// whole tile twice unrolled: 128, 121, 109 us.
constexpr int kPasses = 2;
template <int D>
constexpr int kUnits = kTcKeys / kPasses * (D / 16) / kConvertThreads;
template <int D>
constexpr int kRowStep = kConvertThreads / (D / 16);
constexpr int kTcPBias = 6;

// Registers of the threads of a warpgroup (Q8 kernels alone).
template <bool MORE, int N, bool Q8>
__device__ __forceinline__ void set_registers() {
  if (Q8 && MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  if (Q8 && !MORE) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// A thread's row of a step of rows: the two 64-dim atoms of a row lie in the same banks, so of eight threads with
// a row's chunks the four of the second atom take its neighbour.
template <int D>
__device__ __forceinline__ int unit_row(int ctid) {
  const int c = ctid % (D / 16);
  return (ctid / (D / 16)) ^ (c >> 2);
}
template <int D>
__device__ __forceinline__ void load_raw(const uint8_t* tile, int ctid, int row0, uint4 (&x)[kUnits<D>]) {
  const uint4* raw = reinterpret_cast<const uint4*>(tile + TcLayout<D>::kTile / 2) +
                     (row0 + unit_row<D>(ctid)) * (D / 16) +
                     ctid % (D / 16);
#pragma unroll
  for (int i = 0; i < kUnits<D>; ++i) x[i] = raw[i * kConvertThreads];
}
// Whether a predicate holds in all threads of a named barrier, which they all come to.
template <int ID, int THREADS>
__device__ __forceinline__ bool all_threads(bool good) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(all)
      : "r"((uint32_t)good), "n"(ID), "n"(THREADS)
      : "memory");
  return all != 0;
}
// The largest and the smallest scale byte of rows z0 .. z1 - 1 that are numbers (0 and 255 if none is), and which of a
// lane's four rows (bytes 0xff) are not (by a whole warp).
__device__ __forceinline__ int2 scale_range(const uint8_t* scale, int z0, int z1, uint32_t& nan4) {
  const int r = (threadIdx.x & 31) * 4;
  const uint32_t s4 = *reinterpret_cast<const uint32_t*>(scale + r);
  uint32_t out4 = 0;
  if (z0 > 0 || z1 < kTcKeys)
    out4 = (r >= z0 && r < z1 ? 0u : 0xffu) | (r + 1 >= z0 && r + 1 < z1 ? 0u : 0xff00u) |
           (r + 2 >= z0 && r + 2 < z1 ? 0u : 0xff0000u) | (r + 3 >= z0 && r + 3 < z1 ? 0u : 0xff000000u);
  nan4 = __vcmpeq4(s4, 0xffffffffu) & ~out4;
  out4 |= nan4;
  const uint32_t hi = __vmaxu4(s4 & ~out4, (s4 & ~out4) >> 16), lo = __vminu4(s4 | out4, (s4 | out4) >> 16);
  return make_int2(__reduce_max_sync(0xffffffffu, max(hi & 255u, (hi >> 8) & 255u)),
                   __reduce_min_sync(0xffffffffu, min(lo & 255u, (lo >> 8) & 255u)));
}
// What a tile is held over: a scale byte, ref, the largest of the part's first tile, for rows up to kUp above it, and
// below it for K rows as far as they lose no bit in fp16 (15; kUp: int8's -1152 f has to be a half), for V rows as far as
// a unit's rows share a power of two.  Or the tile is apart: codes go on as they are, and a row of the unit takes their powers
// of two itself (apart_tile): where K rows are further apart or one is no number, and where V rows are, then to the part's
// end.  kHasNaN: V rows of the tile are no numbers, which are noted and taken for the zeros that their codes are.
constexpr int kUp = 4;
constexpr int kHasNaN = 1 << 16, kApart = 1 << 17, kExpMask = 0xffff;
constexpr int kNoRef = -1, kFarRef = -2;  // no row yet; apart to the part's end
// What a tile is held over, and ref from then on (by a whole warp).
__device__ __forceinline__ int2 held_at(uint8_t* scale, int z0, int z1, bool v, int ref, volatile uint32_t* words) {
  uint32_t nan4;
  const int2 range = scale_range(scale, z0, z1, nan4);  // (0, 255): no row is a number
  const int to = ref == kNoRef ? max(range.x, 1) : ref;
  int over = kApart | 1;
  if (ref != kFarRef && range.x <= to + kUp && range.y >= to - (v ? q8::kNear - kUp : 15)) {
    over = to;
    if (range.y < q8::kNaN) ref = to;
  } else if (v) {
    ref = kFarRef;
  }
  if (__any_sync(0xffffffffu, nan4 != 0)) {
    if (!v) return make_int2(kApart | 1, ref);
    const int lane = threadIdx.x & 31;
    const uint32_t bits = (nan4 & 1) | (nan4 >> 7 & 2) | (nan4 >> 14 & 4) | (nan4 >> 21 & 8);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t word = __reduce_or_sync(0xffffffffu, lane / 8 == w ? bits << (4 * (lane & 7)) : 0u);
      if (lane == 0) words[w] = word;
    }
    uint32_t* s4 = reinterpret_cast<uint32_t*>(scale + 4 * lane);
    *s4 = (*s4 & ~nan4) | (nan4 & (uint32_t)(over & 255) * 0x01010101u);
    over |= kHasNaN;
  }
  return make_int2(over, ref);
}
// Pairs of fp16 values of four codes, times a pair of equal factors f; g = -1152 f.
template <bool E4M3>
__device__ __forceinline__ void widen4(uint32_t x, __half2 f, __half2 g, uint32_t& lo, uint32_t& hi) {
  uint32_t a, b;
  __half2 v0, v1;
  if (E4M3) {
    asm("{.reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(a), "=r"(b)
        : "r"(x));
    v0 = __hmul2(*reinterpret_cast<const __half2*>(&a), f);
    v1 = __hmul2(*reinterpret_cast<const __half2*>(&b), f);
  } else {  // 1024 + (code + 128), less 1152 (exact ahead of the sum's one rounding)
    const uint32_t u = x ^ 0x80808080u;
    a = __byte_perm(u, 0x64646464u, 0x4140);
    b = __byte_perm(u, 0x64646464u, 0x4342);
    v0 = __hfma2(*reinterpret_cast<const __half2*>(&a), f, g);
    v1 = __hfma2(*reinterpret_cast<const __half2*>(&b), f, g);
  }
  lo = *reinterpret_cast<const uint32_t*>(&v0);
  hi = *reinterpret_cast<const uint32_t*>(&v1);
}
template <int D, bool E4M3>
__device__ __forceinline__ void convert_rows(uint8_t* tile, const int (&e)[kUnits<D>], int ctid, int row0,
                                             const uint4 (&x)[kUnits<D>]) {
  const int c = ctid % (D / 16), r0 = unit_row<D>(ctid), ch = 2 * (c & 3), sw = r0 & 7;
  uint8_t* row = tile + (c >> 2) * kAtomBytes + (row0 + r0) * 128;
  uint8_t *first = row + ((ch ^ sw) << 4), *second = row + (((ch + 1) ^ sw) << 4);
#pragma unroll
  for (int i = 0; i < kUnits<D>; ++i) {
    const float f32 = __int_as_float(e[i] << 23);
    const __half2 f = __floats2half2_rn(f32, f32);
    const __half2 g = E4M3 ? f : __hmul2(f, __half2half2(__ushort_as_half(0xe480)));  // (-1152)
    uint32_t o[8];
    widen4<E4M3>(x[i].x, f, g, o[0], o[1]);
    widen4<E4M3>(x[i].y, f, g, o[2], o[3]);
    widen4<E4M3>(x[i].z, f, g, o[4], o[5]);
    widen4<E4M3>(x[i].w, f, g, o[6], o[7]);
    *reinterpret_cast<uint4*>(first + i * kRowStep<D> * 128) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(second + i * kRowStep<D> * 128) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}
// V rows outside of [z0, z1), whose codes and scales may be anything, become zeros (by the threads that wrote them).
template <int D>
__device__ __forceinline__ void clear_outside(uint8_t* tile, int ctid, int z0, int z1) {
  const int c = ctid % (D / 16);
#pragma unroll 1
  for (int i = 0; i < 2 * kPasses * kUnits<D>; ++i) {
    const int r = unit_row<D>(ctid) + (i >> 1) * kRowStep<D>;
    if (r < z0 || r >= z1)
      *reinterpret_cast<uint4*>(tile + (c >> 2) * kAtomBytes + r * 128 + (((2 * (c & 3) + (i & 1)) ^ (r & 7)) << 4)) =
          make_uint4(0, 0, 0, 0);
  }
}

// A row of bf16 queries in shared memory becomes fp16, over the power of two of its largest; returns that.
// Elements below 2^-14 of the largest lose bits (to 2^-25 of it), the others none.
template <int D>
__device__ __forceinline__ float as_halves(uint8_t* block, int row) {
  uint8_t* at = block + row * 128;
  const int sw = row & 7;
  uint32_t top = 0;
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    const uint4 v = *reinterpret_cast<const uint4*>(at + (c >> 3) * kAtomBytes + (((c & 7) ^ sw) << 4));
    const uint32_t m = 0x7fff7fffu;
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m)));
  }
  const int e = min(max((int)(max(top & 0xffffu, top >> 16) >> 7), 1), 253);
  const float f = __int_as_float((254 - e) << 23);
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    uint4* p = reinterpret_cast<uint4*>(at + (c >> 3) * kAtomBytes + (((c & 7) ^ sw) << 4));
    const uint4 v = *p;
    const float2 a = q8::unpack<false>(v.x), b = q8::unpack<false>(v.y);
    const float2 d = q8::unpack<false>(v.z), g = q8::unpack<false>(v.w);
    *p = make_uint4(pack2<true>(a.x * f, a.y * f), pack2<true>(b.x * f, b.y * f), pack2<true>(d.x * f, d.y * f),
                    pack2<true>(g.x * f, g.y * f));
  }
  return __int_as_float(e << 23);
}

// What an 8-bit cache's tiles are held over, and their scales (K's outlive their stage).
template <bool Q8>
struct Held {
  __align__(16) uint8_t kscale[Q8 ? kExpRing : 1][kTcKeys];
  uint8_t vscale[Q8 ? kVStages : 1][kTcKeys];
  uint8_t flat[Q8 ? kTcKeys : 1];                                 // of tiles whose codes go on as they are
  volatile int kexp[Q8 ? kExpRing : 1], vexp[Q8 ? kExpRing : 1];  // a scale byte, kHasNaN, kApart
  volatile uint32_t vnan[Q8 ? kExpRing : 1][4];                   // keys whose V row is no number, where vexp says so
};

// A row's tile of an 8-bit cache whose K or V rows are far apart: a key's power of two goes on its score, a V row's on its
// probability, and O is held over the row's largest p_j 2^t_j.  Otherwise as the loop of paged_tc_kernel, bit for bit
// where sums and maxima are concerned.  By a whole warp, 32 keys at a time through TMEM.  A function, and called from a loop
// of its own behind that one: in it the tiles that need none of this pay for it (16 trees of 64 104 us, 106 to 109 with the
// call there, 119 with its code there; 103 without any).
struct ApartRow {
  float m_run, l_run;
  int vexp, vnan;
};
template <int D, bool CAP, bool BIAS>
__device__ __noinline__ ApartRow apart_tile(const PagedAttnParams& p, const Part& w, const Held<true>& held,
                                            uint64_t* p_full, int nb, int t, uint32_t kt, uint32_t bad, uint32_t tmem,
                                            float qf, ApartRow a) {
  const int rb = threadIdx.x >> 7, row = threadIdx.x & (kRB - 1), tl = row / p.G;
  const uint32_t lane_base = (uint32_t)(((threadIdx.x >> 5) & 3) * 32) << 16;
  const uint32_t tS = tmem + 128 * rb + lane_base, tO = tmem + 256 + 128 * rb + lane_base;
  const int j0 = (w.end - 1 - t) * kTcKeys, L = w.s.L, lo = w.lo, hi = w.hi;
  const Row r = row_of(p, w, w.first + min(rb * nb + min(tl, nb - 1), w.ntok - 1), false);
  const float slope = (BIAS && p.slopes) ? __ldg(p.slopes + w.kvh * p.G + row % p.G) * kLog2e : 0.0f;
  tc_fence_after();
  const int k_held = held.kexp[kt % kExpRing], v_held = held.vexp[kt % kExpRing];
  const uint8_t *ks = held.kscale[kt % kExpRing], *vs = held.vscale[kt % kVStages];
  const bool k_apart = k_held & kApart, v_apart = v_held & kApart;
  const float kf = fminf(qf * __int_as_float((k_held & kExpMask) << 23), FLT_MAX);  // (0 where K is apart)
  auto key_factor = [&](int j) { return k_apart ? q8::at_most(qf * q8::factor(ks[j]), FLT_MAX) : kf; };
  const float in_scale = CAP ? 1.0f : k_apart ? p.scale_log2 : fminf(fmaxf(p.scale_log2 * kf, FLT_MIN), FLT_MAX);
  const float scale = (BIAS && p.slopes) ? 1.0f : in_scale;
  uint32_t x[32];
  bool far = false;
  if (CAP) {
    float top = 0.0f;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      tmem_ld32(tS + 32 * c, x);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int j = 32 * c + e;
        const float y = __uint_as_float(x[e]) * key_factor(j);
        if (j0 + j >= lo && j0 + j < hi) top = fmaxf(top, y * y);
      }
    }
    far = __any_sync(0xffffffffu, top > p.cap_top && tl < nb && rb * nb + tl < w.ntok);
  }
  float tmax = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    const int j = j0 + 32 * c;
    uint32_t v = see32(p, r, j, L, hi);
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if ((bad >> (4 * c + g)) & 1u) v &= ~(0xffu << (8 * g));
    tmem_ld32(tS + 32 * c, x);
    tmem_wait_ld();
    if (CAP || k_apart) {
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        float s = __uint_as_float(x[e]) * key_factor(32 * c + e);
        if (CAP && far) s = p.softcap_log2 * tanh_any(s * (2.0f * kLog2e * p.cap_in));
        else if (CAP) {
          const float y = s * s;
          s *= fmaf(fmaf(fmaf(p.cap_q[3], y, p.cap_q[2]), y, p.cap_q[1]), y, p.cap_q[0]);
        }
        x[e] = __float_as_uint(s);
      }
    }
    if (BIAS && r.anc && j0 + kTcKeys > L)
      tree_chunk(p, r, j, L, hi, in_scale, slope, v, x);
    else if (BIAS && p.slopes)
      bias_chunk(fmaf(slope, 32.0f * c, slope * (float)(j0 - r.pos)), slope, in_scale, x);
    if ((v_held & kHasNaN) && (v & held.vnan[kt % kExpRing][c])) a.vnan = 1;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      if (!((v >> e) & 1u)) x[e] = __float_as_uint(-INFINITY);
      tmax = fmaxf(tmax, __uint_as_float(x[e]));
    }
    tmem_st32(tS + 32 * c, x);
  }
  tmem_wait_st();
  tmax *= scale;
  // (scores so large that a rounding of the maximum is a power of two or more: see paged_tc_kernel)
  const bool big = !CAP && __any_sync(0xffffffffu, fabsf(tmax) > 0x1p22f && fabsf(tmax) < INFINITY);
  auto score = [&](uint32_t y) { return big ? __fmul_rn(__uint_as_float(y), scale) : __uint_as_float(y); };
  const float sc = big ? 1.0f : scale;
  const bool moves = a.m_run == -INFINITY || tmax > a.m_run + kRescaleLog2, fresh = a.m_run == -INFINITY;
  const float m_new = moves ? tmax : a.m_run, nm = m_new == -INFINITY ? 0.0f : -m_new;
  int vexp = v_held & kExpMask;
  if (v_apart) {
    float top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      tmem_ld32(tS + 32 * c, x);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) top = fmaxf(top, fmaf(score(x[e]), sc, nm) + (float)vs[32 * c + e]);
    }
    vexp = q8::held_over(a.vexp, top > -INFINITY ? (int)ceilf(fminf(fmaxf(top, -1e4f), 1e4f)) : q8::kNone,
                         m_new - a.m_run, fresh);
  }
  const float corr = moves && !fresh ? ex2(a.m_run - m_new) : 1.0f;
  a.l_run *= corr;
  if (t > 0 && __any_sync(0xffffffffu, moves || vexp != a.vexp)) {
    // (the two powers of two may each be past the 32-bit range; O of a fresh row is 0)
    const float o_corr = moves && !fresh ? ex2(a.m_run - m_new + (float)(a.vexp - vexp)) : q8::exp2_whole(a.vexp - vexp);
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      tmem_ld32(tO + c, x);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * o_corr);
      tmem_st32(tO + c, x);
    }
  }
  a.m_run = m_new;
  a.vexp = vexp;
  const float mm = (m_new == -INFINITY ? 0.0f : m_new) - (float)kTcPBias;
  const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-mm, -mm);
  float2 ps[4] = {};
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    tmem_ld32(tS + 32 * c, x);
    tmem_wait_ld();
    uint32_t pw[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 y = ffma2(make_float2(score(x[2 * e]), score(x[2 * e + 1])), sc2, nm2);
      const float2 f = make_float2(ex2(y.x), ex2(y.y));
      ps[e & 3] = fadd2(ps[e & 3], f);
      const int j = 32 * c + 2 * e;
      pw[e] = pack2<true>(v_apart ? q8::times_exp2(f.x, vs[j] - vexp) : f.x,
                          v_apart ? q8::times_exp2(f.y, vs[j + 1] - vexp) : f.y);
    }
    tmem_st16(tS + 16 * c, pw);
    if (c & 1) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&p_full[c >> 1]);
    }
  }
  const float2 pa = fadd2(fadd2(ps[0], ps[1]), fadd2(ps[2], ps[3]));
  a.l_run += pa.x + pa.y;
  return a;
}

// CAP: a softcap; BIAS: slopes, or tree distances that the window reaches.  Variants of
// their own, and rolled loops wherever a warp does not wait for them: a loop over the tiles that is
// larger than the instruction cache (some 32 KB) runs at half the speed.
// PRE: of a call with shared prefixes: a part may be a prefix's, and rows are left as they are.
// Q8: over an 8-bit cache: warps 12-19 convert tiles (convert_rows) to fp16, over a power of two of the part's K or V rows
// (held_at); from a tile on whose rows are too far apart for one, apart_tile takes the softmax.  bf16 queries become fp16
// over a power of two of their row (as_halves).  Scores take the powers of two of q and K with their scale, O's is V's, and P
// is fp16 with six more bits of range below.
template <int D, bool F16, bool CAP, bool BIAS, bool PRE, bool Q8>
__global__ void __launch_bounds__(Q8 ? kTcThreads + kConvertThreads : kTcThreads, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedAttnParams p, const int nb) {
  using Lay = TcLayout<D>;
  constexpr int A = Lay::A;
  constexpr uint32_t kTmemCols = 512, kOCol = 256;
  constexpr int kThreads = Q8 ? kTcThreads + kConvertThreads : kTcThreads;
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
  // (8-bit cache) raw tiles have landed; their scales have been looked at
  __shared__ __align__(8) uint64_t bar_q_raw;  // (bf16 queries, ahead of as_halves)
  __shared__ __align__(8) uint64_t bar_k_raw[Q8 ? kKStages : 1], bar_v_raw[Q8 ? kVStages : 1];
  __shared__ __align__(8) uint64_t bar_k_scale[Q8 ? kKStages : 1], bar_v_scale[Q8 ? kVStages : 1];
  __shared__ Held<Q8> s_held;
  auto& s_kscale = s_held.kscale;
  auto& s_vscale = s_held.vscale;
  auto& s_vnan = s_held.vnan;
  volatile int *s_kexp = s_held.kexp, *s_vexp = s_held.vexp;
  __shared__ PartRing s_ring;
  __shared__ Cursor<kTcKeys, PRE> s_cur;
  __shared__ int s_late;  // the first sequence that a softmax warp gave up in
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  if (tid == 0) {
    mbar_init(&bar_q_full, Q8 && !F16 ? 8 : 1);
    mbar_init(&bar_q_raw, 1);
    mbar_init(&bar_q_empty, 1);
    mbar_init(&bar_drain, 1);
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&bar_k_full[i], Q8 ? kConvertThreads / 32 : 1);
      mbar_init(&bar_k_empty[i], 1);
      if (Q8) mbar_init(&bar_k_raw[Q8 ? i : 0], 1 + 32);
      if (Q8) mbar_init(&bar_k_scale[Q8 ? i : 0], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&bar_v_full[i], Q8 ? kConvertThreads / 32 : 1);
      if (Q8) mbar_init(&bar_v_raw[Q8 ? i : 0], 1 + 32);
      if (Q8) mbar_init(&bar_v_scale[Q8 ? i : 0], 1);
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
    s_ring.init(Q8 ? 11 + kConvertThreads / 32 : 11);  // K, V, products, eight softmax warps (, those that convert)
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (Q8 && tid < kTcKeys) s_held.flat[Q8 ? tid : 0] = 1;
  if (warp == 0) tmem_alloc(&s_tmem, kTmemCols);
  prefetch_lengths<kThreads, PRE>(p);
  pdl_wait();
  tc_fence_before();
  const int good = find_share<kTcKeys, kThreads>(p, s_cur);
  if (PRE && blockIdx.x == 0 && tid == 0) p.desc[0] = make_int4(good, 0, 0, 0);
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  uint32_t n = 0;  // parts so far
  bool ok = true;
  // (8-bit cache) the launch's 96 registers a thread are shared out: 168 to a softmax thread, 48 to the others
  if (Q8 && warp >= 12) {
    // ------------------------------------------- raw tiles to 16-bit operands
    set_registers<false, 48, Q8>();
    const int ctid = tid - kTcThreads;
    uint32_t it = 0, kst = 0, kph = 0, vst = 0, vph = 0;  // tiles so far
    for (; ok; ++n) {
      ok = all_threads<2, kConvertThreads>(__all_sync(0xffffffffu, s_ring.ready(n, p.wait_limit)));
      if (!ok) break;
      const Part& w = s_ring.at(n);
      if (w.b < 0) break;
      const int lo = w.lo, hi = w.hi, begin = w.begin;
      for (int t = w.end - 1; ok && t >= begin; --t, ++it) {
        const int z0 = lo - t * kTcKeys, z1 = hi - t * kTcKeys;
#pragma unroll 1
        for (int side = 0; ok && side < 2; ++side) {
          const uint32_t st = side ? vst : kst, ph = side ? vph : kph;
          bool landed = warp_wait((side ? bar_v_scale : bar_k_scale) + (Q8 ? st : 0), ph, p.wait_limit);
          landed = warp_wait((side ? bar_v_raw : bar_k_raw) + (Q8 ? st : 0), ph, p.wait_limit) && landed;  // (it has)
          uint8_t* tile = (side ? sV : sK) + st * Lay::kTile;
          const int held = (side ? s_vexp : s_kexp)[Q8 ? it % kExpRing : 0], over = held & kExpMask;
          const uint8_t* scale = held & kApart ? s_held.flat : side ? s_vscale[Q8 ? st : 0] : s_kscale[Q8 ? it % kExpRing : 0];
#pragma unroll 1
          for (int pass = 0; ok && pass < kPasses; ++pass) {
            const int row0 = pass * (kTcKeys / kPasses);
            uint4 x[kUnits<D>];
            load_raw<D>(tile, ctid, row0, x);
            int e[kUnits<D>];  // exponents of the rows' factors, as floats have them (outside of the unit's range: anything)
#pragma unroll
            for (int i = 0; i < kUnits<D>; ++i) e[i] = scale[row0 + unit_row<D>(ctid) + i * kRowStep<D>] + 127 - over;
            // (the pass's codes are in registers before their place is written; a warp that gave up joins the others here)
            ok = all_threads<2, kConvertThreads>(landed);
            if (!ok) break;
            if (p.e4m3) convert_rows<D, true>(tile, e, ctid, row0, x);
            else convert_rows<D, false>(tile, e, ctid, row0, x);
          }
          if (!ok) break;
          if (side && (z0 > 0 || z1 < kTcKeys)) clear_outside<D>(tile, ctid, z0, z1);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive((side ? bar_v_full : bar_k_full) + st);
        }
        kph ^= kst == kKStages - 1;
        kst = kst == kKStages - 1 ? 0 : kst + 1;
        vph ^= vst == kVStages - 1;
        vst = vst == kVStages - 1 ? 0 : vst + 1;
      }
      if (lane == 0) s_ring.done(n);
    }
  } else if (warp >= 8) {
  set_registers<false, 48, Q8>();
  if (warp == 8 || warp == 10) {
    // ------------------------------------------------------- K, V producers
    const bool isV = warp == 10;
    const CUtensorMap* map = isV ? &tmV : &tmK;
    uint8_t* ring = isV ? sV : sK;
    uint64_t* full = Q8 ? (isV ? bar_v_raw : bar_k_raw) : isV ? bar_v_full : bar_k_full;
    uint64_t* empty = isV ? bar_v_empty : bar_k_empty;
    const uint32_t stages = isV ? kVStages : kKStages;
    PageFeed<kTcKeys, PRE> feed;
    const int rows_page = min(1 << p.page_shift, kTcKeys), npg = kTcKeys / rows_page;
    // (8-bit cache: lane l < 16 has the keys 8 l .. 8 l + 7, their scales and, if they are its first, their page's box)
    const int pg = Q8 ? (lane & 15) * 8 / rows_page : lane % npg, atom = lane / npg;
    const int row0 = Q8 ? (lane & 15) * 8 : pg * rows_page;
    const bool issues = Q8 ? lane < 16 && (lane * 8) % rows_page == 0 : atom < A;
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
    // (8-bit cache) The scales of tile j, once it has landed: what its K or V is held over.
    int ref = kNoRef;
    auto look_at_scales = [&](uint32_t j, int z0, int z1, bool first) {
      const uint32_t st = isV ? j % kVStages : j % kKStages, ph = (isV ? j / kVStages : j / kKStages) & 1;
      if (!warp_wait(&full[st], ph, p.wait_limit)) return false;
      uint8_t* scale = isV ? s_vscale[Q8 ? st : 0] : s_kscale[Q8 ? j % kExpRing : 0];
      const int2 at = held_at(scale, z0, z1, isV, first ? kNoRef : ref, s_vnan[Q8 ? j % kExpRing : 0]);
      ref = at.y;
      if (lane == 0) (isV ? s_vexp : s_kexp)[Q8 ? j % kExpRing : 0] = at.x;
      __syncwarp();
      if (lane == 0) mbar_arrive((isV ? bar_v_scale : bar_k_scale) + st);
      return true;
    };
    ok = p.wait_limit > 0;
    for (; ok; ++n) {
      ok = __all_sync(0xffffffffu, s_ring.ready(n, p.wait_limit));
      if (!ok) break;
      const Part w = s_ring.at(n);
      if (w.b < 0) break;
      if (!Q8 && isV && w.begin == w.end) clear_rows();
      feed.start(p, w);
      if (Q8) {
        // Loads go first, as far as there is room; else the scales of the next tile that lands are looked at.
        const uint32_t it0 = it, it1 = it + (w.end - w.begin);
        for (uint32_t seen = it; seen < it1;) {
          const uint32_t st = isV ? it % kVStages : it % kKStages, ph = ((isV ? it / kVStages : it / kKStages) & 1) ^ 1;
          if (it < it1 && (seen == it || __all_sync(0xffffffffu, mbar_test(&empty[st], ph)))) {
            const int t = w.end - 1 - (int)(it - it0), row = (t * kTcKeys + row0) & ((1 << p.page_shift) - 1);
            uint32_t bad8;
            const int page = feed.get(p, w, t, pg, bad8);
            ok = warp_wait(&empty[st], ph, p.wait_limit) && !s_abort;
            if (!ok) break;
            if (lane == 0) {
              if (!isV) s_bad_pages[it % kBadRing] = bad8;
              mbar_expect_tx(&full[st], Lay::kTile / 2);
            }
            __syncwarp();
            if (issues)
              tma_load_rows(ring + st * Lay::kTile + Lay::kTile / 2 + row0 * D, map, &full[st], 0, row, w.kvh, page,
                            p.row_dim, p.head_dim);
            if (lane < 16)
              load_scales(p, (isV ? s_vscale[Q8 ? st : 0] : s_kscale[Q8 ? it % kExpRing : 0]) + row0, isV ? p.v_scale : p.k_scale,
                          page, w.kvh, row);
            cp_arrive(&full[st]);
            ++it;
          } else {
            const int j0 = (w.end - 1 - (int)(seen - it0)) * kTcKeys;
            ok = look_at_scales(seen, w.lo - j0, w.hi - j0, seen == it0);
            if (!ok) break;
            ++seen;
          }
        }
        if (lane == 0) s_ring.done(n);
        continue;
      }
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
    if (!Q8 && isV && ok) clear_rows();
    if (Q8) asm volatile("cp.async.wait_all;" ::: "memory");
    // no copy may be in flight when the CTA leaves
    for (uint32_t i = it > stages ? it - stages : 0; i < it; ++i)
      mbar_wait(&full[i % stages], (i / stages) & 1);
  } else if (warp == 11) {
    // ------------------------------ the share's parts, and their Q rows
    uint32_t parts = 0;
    Part w;
    Cursor<kTcKeys, PRE> cur = s_cur;
    if (!PRE && p.merge && lane == 0) p.desc[share_index()] = make_int4(0, 0, 0, 0);
    uint64_t& bar_q_land = Q8 && !F16 ? bar_q_raw : bar_q_full;
    // One thread: a part's Q rows, as boxes of nb tokens.
    auto load_q = [&](const Part& w) {
      if (lane == 0) {
        const int nrb = w.ntok > nb ? 2 : 1;
        mbar_expect_tx(&bar_q_land, (uint32_t)(nrb * A * 64 * p.G * nb * 2));
        for (int r = 0; r < nrb; ++r)
#pragma unroll
          for (int a = 0; a < A; ++a)
            tma_load_3d(sQ + (r * A + a) * kAtomBytes, &tmQ, &bar_q_land, a * 64, w.kvh * p.G,
                        w.s.t0 + w.first + r * nb);
      }
      __syncwarp();
      ++parts;
    };
    if (PRE) {
      // Many small units: parts are published ahead of the Q rows that they wait for, so that their K and V
      // are on their way.
      uint32_t nq = 0;  // parts whose Q rows are asked for
      bool more = true;
      for (;;) {
        const bool behind = nq < n, full = n - nq == kPartRing - 1;
        const bool free = behind && __all_sync(0xffffffffu, mbar_test(&bar_q_empty, (parts & 1) ^ 1));
        if (behind && (full || !more || free)) {
          const Part& q = s_ring.at(nq);
          if (q.begin != q.end) {
            ok = warp_wait(&bar_q_empty, (parts & 1) ^ 1, p.wait_limit) && !s_abort;
            if (!ok) break;
            load_q(q);
          }
          ++nq;
        } else if (more) {
          more = cur.next(p, w);
          ok = s_ring.publish(n, w, p.wait_limit);
          if (!ok) break;
          if (more) {
            ++n;
            if (w.parts || w.slot < 0) note_unit(p, w);
          }
        } else {
          break;
        }
      }
    } else {
      for (;; ++n) {
        const bool more = cur.next(p, w);
        ok = s_ring.publish(n, w, p.wait_limit);
        if (!ok || !more) break;
        if (p.merge && w.parts && lane == 0)
          p.desc[share_index()] = make_int4(w.s.t0 + w.first, w.ntok, w.kvh, w.parts);
        if (w.begin == w.end) continue;
        ok = warp_wait(&bar_q_empty, (parts & 1) ^ 1, p.wait_limit) && !s_abort;
        if (!ok) break;
        load_q(w);
      }
    }
    if (!p.merge) write_status(p);
    if (parts > 0) mbar_wait(&bar_q_land, (parts - 1) & 1);
  } else if (warp == 9) {
    // ------------------------------------------------------------- products
    // One thread waits and issues: what it does between two products is on the critical
    // path of both row blocks (with the whole warp waiting and voting, a barrier that
    // had completed already cost some 150 cycles).
    if (elect_one()) {
      constexpr uint32_t idS = idesc(F16 || Q8, kTcKeys, 0), idO = idesc(F16 || Q8, D, 1);
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
          if (!Q8 && (w.lo > j0 || w.hi < j0 + kTcKeys)) {  // the V producer clears rows of this tile
            ok = ok && wait_within(&bar_v_zero[vst], (zph >> vst) & 1, p.wait_limit);
            zph ^= 1u << vst;
          }
          // (the next K, of an 8-bit cache, is waited for where it is needed: it is converted meanwhile)
          if (!Q8 && more) ok = ok && wait_within(&bar_k_full[kst], kph, p.wait_limit);
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
            if (Q8 && more && r == 0) {
              ok = wait_within(&bar_k_full[kst], kph, p.wait_limit);
              if (!ok) break;
              tc_fence_after();
            }
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
  }
  } else {
    // -------------------------------------------------------------- softmax
    set_registers<true, 168, Q8>();
    const int rb = warp >> 2, row = tid & (kRB - 1);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128 * rb, tO = tmem + kOCol + 128 * rb;
    const int tl = row / p.G, h_in = row % p.G;
    const bool warp_in_block = (warp & 3) * 32 < nb * p.G;
    uint32_t sc = 0, oc = 0, kt = 0, qn = 0;
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
        if (PRE) {  // (or a prefix without rows)
          if (mine && TV_CHECK(oidx < (size_t)p.T * p.Hq))
            p.raw_ml[oidx + (w.s.shared ? 0 : (size_t)p.T * p.Hq)] = make_float2(-INFINITY, 0.0f);
        } else if (mine && TV_CHECK(oidx < (size_t)p.T * p.Hq)) {
          uint4* orow = reinterpret_cast<uint4*>(p.out + oidx * D);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) orow[c] = make_uint4(0, 0, 0, 0);
          if (p.lse) p.lse[oidx] = 0.0f;
        }
        __syncwarp();
        if (lane == 0) s_ring.done(n);
        continue;
      }
      float qf = 1.0f;  // (8-bit cache, bf16) what the row of q is held over
      if (Q8 && !F16) {
        ok = warp_wait(&bar_q_raw, qn++ & 1, p.wait_limit);
        if (!ok) break;
        if (rb * nb < w.ntok) qf = as_halves<D>(sQ + rb * Lay::kTile, row);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_q_full);
      }
      if (rb * nb >= w.ntok) {  // no second row block
        kt += T;
        __syncwarp();
        if (lane == 0) s_ring.done(n);
        continue;
      }
      if (Q8 && (tl >= nb || rb * nb + tl >= w.ntok)) qf = FLT_MIN;  // (its scores are not to be large ones, see below)
      // rows past the unit take the last token's mask: computed, never written
      const int i = w.first + min(rb * nb + min(tl, nb - 1), w.ntok - 1);
      const bool warp_works = warp_in_block && rb * nb + (warp & 3) * 32 / p.G < w.ntok;
      const bool shared = PRE && w.s.shared;
      const Row r = row_of(p, w, i, shared);
      const float slope = (BIAS && p.slopes) ? __ldg(p.slopes + w.kvh * p.G + h_in) * kLog2e : 0.0f;
      // what turns a score into the log2 domain; capped scores are there already, and with
      // slopes it comes with the bias
      const float in_scale0 = CAP ? 1.0f : p.scale_log2;
      float m_run = -INFINITY, l_run = 0.0f;
      int vexp = -1;  // (8-bit cache) O is held over 2^(vexp - 127); no row yet: -1
      bool vnan = false;  // (8-bit cache) it sees a V row that is no number
      int t = 0;
      for (; t < T; ++t, ++kt, ++sc) {
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
        // (8-bit cache) what the tile's scores are held over, as a 32-bit number: a row of zeros over a tile of tiny
        // keys would make it 0, and hidden keys are at -inf ahead of it; nor is 0 times it to be anything else
        const float kf = Q8 ? fminf(qf * __int_as_float((s_kexp[Q8 ? kt % kExpRing : 0] & kExpMask) << 23), FLT_MAX) : 1.0f;
        const float in_scale = CAP ? 1.0f : Q8 ? fminf(fmaxf(in_scale0 * kf, FLT_MIN), FLT_MAX) : in_scale0;
        const float scale = (BIAS && p.slopes) ? 1.0f : in_scale;
        tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + lane_base + 32 * c, sr[c]);
        tmem_wait_ld();
        int v_held = 0;
        if (Q8) {  // (V's scales are known long before, as a rule)
          ok = warp_wait(&bar_v_scale[Q8 ? kt % kVStages : 0], (kt / kVStages) & 1, p.wait_limit);
          if (!ok) break;
          v_held = s_vexp[Q8 ? kt % kExpRing : 0];
          if ((v_held | s_kexp[Q8 ? kt % kExpRing : 0]) & kApart) break;
        }
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
                if (Q8) s[b] = fmul2(s[b], make_float2(kf, kf));
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
                const float y = __uint_as_float(x[e]) * kf;
                if (j0 + c + e >= w.lo && j0 + c + e < hi) top = fmaxf(top, y * y);
              }
            }
            far = __any_sync(0xffffffffu, top > p.cap_top && is_row);
          }
          if (far) {
            const float in = 2.0f * kLog2e * p.cap_in * kf;
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
        float2 sc2 = make_float2(scale, scale);
        auto probs = [&](int c, float m, uint32_t (&pw)[16]) {
          const float2 nm2 = make_float2(-m, -m);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = ffma2(make_float2(__uint_as_float(sr[c][2 * e]),
                                               __uint_as_float(sr[c][2 * e + 1])), sc2, nm2);
            const float2 x = make_float2(ex2(y.x), ex2(y.y));
            ps[e & 3] = fadd2(ps[e & 3], x);
            pw[e] = pack2<F16 || Q8>(x.x, x.y);
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
        const float tmag = fabsf(tmax);
        if ((Q8 || PRE) && !CAP &&
            __any_sync(0xffffffffu, tmag > 0x1p22f && tmag < INFINITY && (Q8 || (tl < nb && rb * nb + tl < w.ntok)))) {
          // Scores so large that a rounding of the maximum is a power of two or more: the products are rounded
          // like it, ahead of the difference (fused, the largest could end far above 0).  (Of an 8-bit cache
          // apart_tile does, while TMEM still has them as they were.)
          if (Q8 && !BIAS) break;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) sr[c][e] = __float_as_uint(__uint_as_float(sr[c][e]) * scale);
          sc2 = make_float2(1.0f, 1.0f);
        }
        const bool moves = m_run == -INFINITY || tmax > m_run + kRescaleLog2;
        bool vmoves = false;
        float vcorr = 1.0f;
        if (Q8) {
          const int v = v_held & ~kHasNaN;
          if (v_held & kHasNaN) {
#pragma unroll
            for (int c = 0; c < 4; ++c) vnan |= (vis[c] & s_vnan[Q8 ? kt % kExpRing : 0][c]) != 0;
          }
          vmoves = vexp >= 0 && v != vexp;
          if (vmoves) vcorr = q8::exp2_whole(vexp - v);
          vexp = v;
        }
        if (__any_sync(0xffffffffu, moves) || vmoves) {
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
              for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * (Q8 ? corr * vcorr : corr));
              tmem_st8(tO + lane_base + c, o);
            }
          }
        }
        // (nothing seen yet: 2^-inf = 0; an fp16 P reaches up to 2^14 and six bits further down)
        const float mm = (m_run == -INFINITY ? 0.0f : m_run) - (Q8 ? (float)kTcPBias : 0.0f);
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
      if constexpr (Q8) {  // from the first tile of K or V rows far apart on
        for (; ok && t < T; ++t, ++kt, ++sc) {
          ok = warp_wait(&bar_s_full[rb], sc & 1, p.wait_limit) &&
               warp_wait(&bar_v_scale[kt % kVStages], (kt / kVStages) & 1, p.wait_limit);
          if (!ok) break;
          tc_fence_after();
          const ApartRow a = apart_tile<D, CAP, BIAS>(p, w, s_held, bar_p_full[rb], nb, t, kt, s_bad_pages[kt % kBadRing],
                                                      tmem, qf, {m_run, l_run, vexp, vnan});
          m_run = a.m_run;
          l_run = a.l_run;
          vexp = a.vexp;
          vnan = a.vnan;
          announce();
        }
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
      // (8-bit cache) O's own power of two less the bias, which the sums have too, as two factors: O times one
      // of them may leave the 32-bit range where the result does not
      const int ve = vexp - 127 - kTcPBias;
      const float v1 = Q8 && vnan ? __int_as_float(0x7fffffff) : q8::exp2_whole(ve >> 1), v2 = q8::exp2_whole(ve - (ve >> 1));
      if (Q8) l_run *= q8::exp2_whole(-kTcPBias);
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
                  Q8 ? make_float4(__uint_as_float(o[4 * q]) * v1 * v2, __uint_as_float(o[4 * q + 1]) * v1 * v2,
                                   __uint_as_float(o[4 * q + 2]) * v1 * v2, __uint_as_float(o[4 * q + 3]) * v1 * v2)
                     : make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
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
        const float f0 = (m_run == -INFINITY ? 0.0f : ex2(m_run - m_all)) * (Q8 ? v2 : 1.0f);
        const float by_sum = l_all == 0.0f ? 0.0f : 1.0f / l_all;
        // (8-bit cache: rows that are joined take v2 with f0, others the sum first)
        const float first = more ? v1 : v1 * by_sum, inv = Q8 && !more ? v2 : by_sum;
        uint8_t* orow = reinterpret_cast<uint8_t*>(p.out + oidx * D);
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o[2][32];
          tmem_ld32(tO + lane_base + 64 * c, o[0]);
          tmem_ld32(tO + lane_base + 64 * c + 32, o[1]);
          tmem_wait_ld();
          if (Q8 && mine) {
#pragma unroll
            for (int e = 0; e < 64; ++e) o[e >> 5][e & 31] = __float_as_uint(__uint_as_float(o[e >> 5][e & 31]) * first);
          }
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
              // (a part whose keys are all hidden: select, do not multiply)
              if (f == 0.0f && (!Q8 || m == -INFINITY)) continue;
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
          if (PRE) {
            if (mine && TV_CHECK(oidx < (size_t)p.T * p.Hq))
#pragma unroll
              for (int q = 0; q < 8; ++q)  // 8 columns: a sector
                store32(reinterpret_cast<uint8_t*>(p.raw + (oidx + (shared ? 0 : (size_t)p.T * p.Hq)) * D + 64 * c + 8 * q),
                        *reinterpret_cast<const uint32_t(*)[8]>(&o[q >> 2][8 * (q & 3)]), true);
          } else if (mine && TV_CHECK(oidx < (size_t)p.T * p.Hq))
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
        if (PRE && mine) p.raw_ml[oidx + (shared ? 0 : (size_t)p.T * p.Hq)] = make_float2(m_all, l_all);
        else if (mine && p.lse) p.lse[oidx] = l_all == 0.0f ? -INFINITY : (m_all + log2f(l_all)) * kLn2;
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

template <int D, bool F16, bool CAP, bool BIAS, bool PRE, bool Q8>
cudaError_t launch(const PagedPlan& pl, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                   const CUtensorMap& tmV, const PagedAttnParams& p, cudaStream_t stream) {
  if (!set_dyn_smem(paged_tc_kernel<D, F16, CAP, BIAS, PRE, Q8>, TcLayout<D>::kDyn)) return cudaErrorUnknown;
  return launch_pdl(paged_tc_kernel<D, F16, CAP, BIAS, PRE, Q8>, dim3(pl.ctas),
                    dim3(Q8 ? kTcThreads + kConvertThreads : kTcThreads),
                    (size_t)TcLayout<D>::kDyn, stream, tmQ, tmK, tmV, p, pl.nb);
}
template <int D, bool F16, bool PRE, bool Q8>
cudaError_t launch_kind(const PagedPlan& pl, bool bias, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                        const CUtensorMap& tmV, const PagedAttnParams& p, cudaStream_t stream) {
  if (p.softcap_log2 > 0.0f)
    return bias ? launch<D, F16, true, true, PRE, Q8>(pl, tmQ, tmK, tmV, p, stream)
                : launch<D, F16, true, false, PRE, Q8>(pl, tmQ, tmK, tmV, p, stream);
  return bias ? launch<D, F16, false, true, PRE, Q8>(pl, tmQ, tmK, tmV, p, stream)
              : launch<D, F16, false, false, PRE, Q8>(pl, tmQ, tmK, tmV, p, stream);
}
template <bool PRE, bool Q8>
cudaError_t launch_any(const PagedPlan& pl, int D, bool f16, bool bias, const CUtensorMap& tmQ,
                       const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedAttnParams& p,
                       cudaStream_t stream) {
  if (D == 128)
    return f16 ? launch_kind<128, true, PRE, Q8>(pl, bias, tmQ, tmK, tmV, p, stream)
               : launch_kind<128, false, PRE, Q8>(pl, bias, tmQ, tmK, tmV, p, stream);
  return f16 ? launch_kind<64, true, PRE, Q8>(pl, bias, tmQ, tmK, tmV, p, stream)
             : launch_kind<64, false, PRE, Q8>(pl, bias, tmQ, tmK, tmV, p, stream);
}

}  // namespace
}  // namespace paged
}  // namespace tv
