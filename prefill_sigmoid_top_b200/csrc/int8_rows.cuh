// The codes of a symmetric 8-bit row (the activation and weight form of the int8 products).
//   a = max |v| of the row;  scale = a / 127 (fp32);  code = rint(127 v / a), ties to even;  a = 0: scale 0, codes 0.
// A row that holds an infinity or a NaN gets the scale NaN and codes 0: its products are NaN.
//
// The codes are those of exact arithmetic without a division per element.  v and a are bf16: 8 significant bits,
// v = m 2^i, a = n 2^j (m, n in [128, 255]).  127 v / a is a tie only if 254 v = (2k + 1) a.  Unless the prime 127
// divides n (n = 254), the odd part of n then divides that of m and 2k + 1 is a multiple of 127 up to 253: 127, so
// v = +-a/2 (63.5, to the even 64).  A quotient that is no tie is at least 1.5e-5 (relative) away from one.  So for a row with n != 254 one multiply-add is exact:
//   code = low byte of fma(v, c, 1.5 * 2^23), c = 127 / a rounded up (within 2^-22): adding 1.5 * 2^23 rounds to an
//   integer once, and v = +-a/2 falls just beyond 63.5, on 64.
// Rows with n = 254, and rows so large or small that c leaves fp32's range, take the remainder: t = 127 v is exact
// (15 bits), q = rint(t / a) is right or, on a tie, a neighbour; r = t - q a is exact (at most 17 bits), 2 |r| = a
// says tie, and an odd q moves to the even one.
#pragma once

#include "common.cuh"

namespace moe {

// Power of two that brings a row's largest magnitude into a range where 127 v stays finite and 1 / a normal.
__device__ __forceinline__ float prescale(float a) { return a > 0x1p100f ? 0x1p-32f : (a < 0x1p-60f ? 0x1p64f : 1.0f); }

struct RowScale {
  float a, inv, pre;  // largest magnitude times pre; its reciprocal (0: all codes are 0)
  float c;            // 127 / a rounded up, or 0: the remainder decides
};

__device__ __forceinline__ RowScale row_scale_of(uint32_t top) {
  const float amax = __uint_as_float(top << 16);
  RowScale s;
  s.pre = prescale(amax);
  s.a = amax * s.pre;
  s.inv = top != 0 && top < 0x7f80u ? __frcp_rn(s.a) : 0.0f;
  const bool plain = s.inv != 0.0f && s.pre == 1.0f && (top & 0x7fu) != 0x7eu;
  s.c = plain ? __fdiv_ru(127.0f, amax) : 0.0f;
  return s;
}

__device__ __forceinline__ float scale_value(uint32_t top) {
  return top < 0x7f80u ? __fdiv_rn(__uint_as_float(top << 16), 127.0f) : __uint_as_float(0x7fffffffu);
}

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer, ties to even

// The code of v, as the low byte of the result, by the remainder.
__device__ __forceinline__ uint32_t code_of(float v, const RowScale& s) {
  v *= s.pre;
  const float t = 127.0f * v;
  const float y = fmaf(t, s.inv, kMagic);
  const float r = fmaf(-(y - kMagic), s.a, t);
  uint32_t q = __float_as_uint(y);
  if (fabsf(r) * 2.0f == s.a && (q & 1u)) q += r > 0.0f ? 1 : -1;
  return q;
}

// |v| as bf16 bits is ordered like the magnitudes: infinity is 0x7f80, NaN above.
__device__ __forceinline__ uint32_t max_bits(uint32_t top, uint32_t pair) {
  return max(top, max(pair & 0x7fffu, (pair >> 16) & 0x7fffu));
}

// The value of an integer sum: (sx sw) sum in fp32, three roundings, as long as the scales' product is a normal number.
// Where it is not (rows or channels near the ends of fp32's range), the result may be one all the same, or 0 where
// infinity times 0 would be NaN: there the product is taken in fp64, whose range holds it, and rounded once.  Which of
// the two depends on the two scales alone, so a row's results are the same bits in every kernel and batch.
static __device__ __noinline__ float int8_value_fp64(float sx, float sw, int sum) {
  return static_cast<float>(static_cast<double>(sx) * static_cast<double>(sw) * static_cast<double>(sum));
}
__device__ __forceinline__ float int8_value(float sx, float sw, int sum) {
  const float p = sx * sw;
  if (fabsf(p) >= 0x1p-126f && fabsf(p) < INFINITY) return p * static_cast<float>(sum);
  return int8_value_fp64(sx, sw, sum);
}
// Two scales for which this holds have a normal product, or one of 0: (sx sw) sum is int8_value without its test.
__device__ __forceinline__ bool int8_near_scale(float s) {
  return s == 0.0f || (fabsf(s) >= 0x1p-60f && fabsf(s) <= 0x1p60f);
}

// Eight bf16 values (a 16-byte vector) as eight codes; kPlain: the row has s.c.
template <bool kPlain>
__device__ __forceinline__ uint2 codes_of_8(const uint4& v, const RowScale& s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint32_t q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float x = (u & 1) ? bf16_hi(w[2 * p + u / 2]) : bf16_lo(w[2 * p + u / 2]);
      q[u] = kPlain ? __float_as_uint(fmaf(x, s.c, kMagic)) : code_of(x, s);
    }
    o[p] = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
  }
  // a row with no scale (inv 0) has codes 0 whatever its values
  return kPlain || s.inv != 0.0f ? make_uint2(o[0], o[1]) : make_uint2(0, 0);
}

// One value's code.
__device__ __forceinline__ int8_t code_of_1(uint16_t bits, const RowScale& s) {
  const float v = __uint_as_float(static_cast<uint32_t>(bits) << 16);
  const uint32_t q = s.c != 0.0f ? __float_as_uint(fmaf(v, s.c, kMagic)) : code_of(v, s);
  return s.inv != 0.0f ? static_cast<int8_t>(q & 0xffu) : static_cast<int8_t>(0);
}

}  // namespace moe
