// Symmetric 8-bit rows: the activation and weight form of the int8 projections.
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
//
// Bound: memory.  A row is read once into registers (16-byte loads, 8 in flight per thread), reduced and written as
// codes; rows of up to 2048 columns take a warp, up to 8192 four warps, longer or unaligned ones a loop that reads
// twice.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kQThreads = 128;
constexpr int kVecs = 8;  // 16-byte vectors per thread

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

template <bool kPlain, int kRowThreads>
__device__ __forceinline__ void write_codes(const uint4 (&v)[kVecs], const RowScale& s, uint2* dst, int nvec, int tid) {
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = tid + kRowThreads * i;
    if (c >= nvec) break;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
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
    dst[c] = kPlain || s.inv != 0.0f ? make_uint2(o[0], o[1]) : make_uint2(0, 0);
  }
}

// kRowThreads threads per row (32 or 128), kVecs vectors of 8 columns each at most.
template <int kRowThreads>
__global__ void __launch_bounds__(kQThreads) quantize_rows_kernel(Int8RowsArgs a) {
  __shared__ uint32_t part[kQThreads / 32];
  grid_launch_dependents();  // the product that follows sets itself up and loads weights meanwhile
  const int tid = threadIdx.x % kRowThreads;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (kQThreads / kRowThreads) + threadIdx.x / kRowThreads;
  bool live = r < a.rows;
  if (live && a.sorted_ids != nullptr) {
    live = r < *a.ntpp;
    if (live) {
      const int id = a.sorted_ids[r];
      live = id >= 0 && id < a.nslots;  // not padding
    }
  }
  const uint4* src = reinterpret_cast<const uint4*>(a.src + (live ? r : 0) * a.ld);
  const int nvec = live ? a.cols / 8 : 0;
  uint4 v[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = tid + kRowThreads * i;
    v[i] = c < nvec ? src[c] : make_uint4(0, 0, 0, 0);
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) top = max_bits(max_bits(max_bits(max_bits(top, v[i].x), v[i].y), v[i].z), v[i].w);
  top = __reduce_max_sync(0xffffffffu, top);
  if (kRowThreads > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kQThreads / 32; ++q) top = max(top, part[q]);
  }
  if (!live) return;
  if (tid == 0) a.scales[r] = scale_value(top);
  const RowScale s = row_scale_of(top);
  uint2* dst = reinterpret_cast<uint2*>(a.codes + r * a.pitch);
  if (s.c != 0.0f)
    write_codes<true, kRowThreads>(v, s, dst, nvec, tid);
  else
    write_codes<false, kRowThreads>(v, s, dst, nvec, tid);
}

// Any alignment and length: one CTA per row, two passes over it.
__global__ void __launch_bounds__(kQThreads) quantize_any_kernel(Int8RowsArgs a) {
  __shared__ uint32_t part[kQThreads / 32];
  grid_launch_dependents();
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  if (a.sorted_ids != nullptr) {
    if (r >= *a.ntpp) return;
    const int id = a.sorted_ids[r];
    if (id < 0 || id >= a.nslots) return;
  }
  const uint16_t* src = a.src + r * a.ld;
  uint32_t top = 0;
  for (int c = tid; c < a.cols; c += kQThreads) top = max(top, static_cast<uint32_t>(src[c] & 0x7fffu));
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) part[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kQThreads / 32; ++q) top = max(top, part[q]);
  if (tid == 0) a.scales[r] = scale_value(top);
  const RowScale s = row_scale_of(top);
  int8_t* dst = a.codes + r * a.pitch;
  for (int c = tid; c < a.cols; c += kQThreads) {
    const float v = __uint_as_float(static_cast<uint32_t>(src[c]) << 16);
    const uint32_t q = s.c != 0.0f ? __float_as_uint(fmaf(v, s.c, kMagic)) : code_of(v, s);
    dst[c] = s.inv != 0.0f ? static_cast<int8_t>(q & 0xffu) : 0;
  }
}

}  // namespace

cudaError_t launch_quantize_int8(const Int8RowsArgs& a, cudaStream_t stream) {
  const bool vectors = a.cols % 8 == 0 && a.ld % 8 == 0 && a.pitch % 8 == 0 &&
                       (reinterpret_cast<uintptr_t>(a.src) & 15u) == 0 &&
                       (reinterpret_cast<uintptr_t>(a.codes) & 7u) == 0;
  if (vectors && a.cols <= 32 * 8 * kVecs) {
    const int64_t per = kQThreads / 32;
    quantize_rows_kernel<32><<<static_cast<unsigned>((a.rows + per - 1) / per), kQThreads, 0, stream>>>(a);
  } else if (vectors && a.cols <= kQThreads * 8 * kVecs) {
    quantize_rows_kernel<kQThreads><<<static_cast<unsigned>(a.rows), kQThreads, 0, stream>>>(a);
  } else {
    quantize_any_kernel<<<static_cast<unsigned>(a.rows), kQThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace moe
