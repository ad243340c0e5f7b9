// The 8-bit paged cache as the kernels see it: a row's codes and its scale byte, and the host
// checks that its entry points share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tv_paged.cuh"

namespace tv {

struct Q8Cache : PagedCache {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ks;
  uint8_t* vs;
  int Hkv;

  __device__ __forceinline__ long long code_at(long long page, int h, int row) const {
    return page * page_stride + h * head_stride + row * row_stride;
  }
  __device__ __forceinline__ long long scale_at(long long page, int h, int row) const {
    return ((page * Hkv + h) << page_shift) + row;
  }
};

// Checks a cache descriptor; fills `out`.
inline tv_status check_q8_cache(const tv_q8_cache* c, Q8Cache* out) {
  if (!c) return TV_ERR_INVALID_ARG;
  if (c->format != TV_E4M3 && c->format != TV_INT8) return TV_ERR_UNSUPPORTED;
  tv_paged_cache rows{c->k,         c->v,   c->page_stride, c->head_stride, c->row_stride, c->num_pages,
                      c->page_size, c->Hkv, c->D,           c->dtype};
  const tv_status st = check_cache(&rows, out);
  if (st != TV_OK) return st;
  if (c->D % 16 != 0 || c->D > 1024) return TV_ERR_UNSUPPORTED;
  if (!c->k_scale || !c->v_scale) return TV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) & 7)
    return TV_ERR_INVALID_ARG;
  if ((out->row_stride | out->head_stride | out->page_stride) & 15) {
    // (a stride of 8, which check_cache gives a dimension of extent one, is never used)
    if ((out->row_stride & 15) || (c->Hkv > 1 && (out->head_stride & 15)) ||
        (c->num_pages > 1 && (out->page_stride & 15)))
      return TV_ERR_INVALID_ARG;
  }
  out->k = static_cast<uint8_t*>(c->k);
  out->v = static_cast<uint8_t*>(c->v);
  out->ks = c->k_scale;
  out->vs = c->v_scale;
  out->Hkv = c->Hkv;
  return TV_OK;
}

namespace q8 {

constexpr int kNaN = 255;  // the scale byte of a row that holds an infinity or a NaN

// The factor of a scale byte: a power of two, so that a product with a code is exact.
__device__ __forceinline__ float factor(int s) {
  return __int_as_float(s == kNaN ? 0x7fffffff : s == 0 ? 0x00400000 : s << 23);  // (0: 2^-127)
}

// 2^e of a whole number, as far as normal 32-bit floats reach.
__device__ __forceinline__ float exp2_whole(int e) { return __int_as_float(min(max(e + 127, 1), 254) << 23); }
// x 2^e, where 2^e alone may be past that.
__device__ __forceinline__ float times_exp2(float x, int e) { return x * exp2_whole(e >> 1) * exp2_whole(e - (e >> 1)); }

// The smaller of two numbers, NaN if x is (a row that is no number has that factor; 0 times a factor past the 32-bit
// range is 0 all the same).
__device__ __forceinline__ float at_most(float x, float top) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(top));
  return y;
}

// While the scale bytes t_j of the V rows that a part has met lie within this of one another, all rows of the unit
// hold their outputs over one power of two.  Beyond it each row has its own, that of its largest p_j 2^t_j so far, so
// that V rows that it does not see, or hardly, cost it no bits.  Either way
// p_j 2^t_j, rounded to fp16 times 2^6, is off by 2^-21 of the row's largest p_j |v_j| at most where it is too small for
// half a step of its own.
constexpr int kNear = 9;
// A row's power of two, as a scale byte's: `e` so far, `want` that of the largest p_j 2^t_j at hand (kNone: it sees none),
// after its maximum went up by `up` (in the log2 domain); `fresh`: it saw nothing before.
constexpr int kNone = -(1 << 20);
__device__ __forceinline__ int held_over(int e, int want, float up, bool fresh) {
  if (!fresh) e -= (int)ceilf(fminf(up, 1e4f));
  return want > kNone && (fresh || want > e + 8) ? want : e;
}

// The scale byte of a row whose largest magnitude is `top` (>= 0): the least e >= -126 with
// top <= M 2^e, M = 448 = 1.75 * 2^8 or 127 = 1.984375 * 2^6, plus 127.
template <bool E4M3>
__device__ __forceinline__ int scale_of(float top) {
  const int bits = __float_as_int(top);
  if (bits >= 0x7f800000) return kNaN;
  const int e = (bits >> 23) - (E4M3 ? 8 : 6) + ((bits & 0x7fffff) > (E4M3 ? 0x600000 : 0x7e0000));
  return max(e, 1);
}

// Two 16-bit values of a word as floats.
template <bool F16>
__device__ __forceinline__ float2 unpack(uint32_t x) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&x));
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// Codes of four values that are scaled already (|y| <= M), nearest, ties to even.
template <bool E4M3>
__device__ __forceinline__ uint32_t encode4(float2 a, float2 b) {
  if (E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
    return (uint32_t)lo | (uint32_t)hi << 16;
  }
  // (behind 1.5 * 2^23 the sum's last byte is the nearest whole number)
  const float big = 12582912.0f;
  const uint32_t x = __byte_perm(__float_as_uint(a.x + big), __float_as_uint(a.y + big), 0x0040);
  const uint32_t y = __byte_perm(__float_as_uint(b.x + big), __float_as_uint(b.y + big), 0x0040);
  return __byte_perm(x, y, 0x5410);
}

// The values of four codes.
template <bool E4M3>
__device__ __forceinline__ void decode4(uint32_t c, float2& a, float2& b) {
  if (E4M3) {
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)c));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(c >> 16)));
    a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  } else {
    const uint32_t u = c ^ 0x80808080u;  // codes + 128, as last bytes of floats of 2^23 and more
    const float off = 8388608.0f + 128.0f;
    a = make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)) - off,
                    __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441)) - off);
    b = make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)) - off,
                    __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443)) - off);
  }
}

}  // namespace q8
}  // namespace tv
