// bf16 rows to 8-bit codes and scales (int8_rows.cuh has the arithmetic).
//
// Bound: memory.  A row is read once into registers (16-byte loads, 8 in flight per thread), reduced and written as
// codes; rows of up to 2048 columns take a warp, up to 8192 four warps; unaligned or longer ones go by elements.
// Measured: 8192 x 7168 (117 MB in, 59 MB out) 26 us, 6.8 TB/s.
#include "int8_rows.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kQThreads = 128;
constexpr int kVecs = 8;  // 16-byte vectors per thread

template <bool kPlain, int kRowThreads>
__device__ __forceinline__ void write_codes(const uint4 (&v)[kVecs], const RowScale& s, uint2* dst, int nvec, int tid) {
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = tid + kRowThreads * i;
    if (c >= nvec) break;
    dst[c] = codes_of_8<kPlain>(v[i], s);
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

// Any alignment: one CTA per row, element loads, up to kElems per thread in flight and kept in registers; longer rows
// (kKeep false) are read twice.
constexpr int kElems = 16;

template <int kThreads, bool kKeep>
__global__ void __launch_bounds__(kThreads) quantize_any_kernel(Int8RowsArgs a) {
  __shared__ uint32_t part[kThreads / 32];
  grid_launch_dependents();
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  if (a.sorted_ids != nullptr) {
    if (r >= *a.ntpp) return;
    const int id = a.sorted_ids[r];
    if (id < 0 || id >= a.nslots) return;
  }
  const uint16_t* src = a.src + r * a.ld;
  uint16_t v[kElems];
  uint32_t top = 0;
  for (int c0 = tid; c0 < a.cols; c0 += kThreads * kElems) {  // once if kKeep
#pragma unroll
    for (int i = 0; i < kElems; ++i) v[i] = c0 + kThreads * i < a.cols ? src[c0 + kThreads * i] : 0;
#pragma unroll
    for (int i = 0; i < kElems; ++i) top = max(top, static_cast<uint32_t>(v[i] & 0x7fffu));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) part[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kThreads / 32; ++q) top = max(top, part[q]);
  if (tid == 0) a.scales[r] = scale_value(top);
  const RowScale s = row_scale_of(top);
  int8_t* dst = a.codes + r * a.pitch;
  for (int c0 = tid; c0 < a.cols; c0 += kThreads * kElems) {
    if (!kKeep) {
#pragma unroll
      for (int i = 0; i < kElems; ++i) v[i] = c0 + kThreads * i < a.cols ? src[c0 + kThreads * i] : 0;
    }
#pragma unroll
    for (int i = 0; i < kElems; ++i)
      if (c0 + kThreads * i < a.cols) dst[c0 + kThreads * i] = code_of_1(v[i], s);
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
    const unsigned rows = static_cast<unsigned>(a.rows);
    if (a.cols <= 128 * kElems)
      quantize_any_kernel<128, true><<<rows, 128, 0, stream>>>(a);
    else if (a.cols <= 512 * kElems)
      quantize_any_kernel<512, true><<<rows, 512, 0, stream>>>(a);
    else
      quantize_any_kernel<512, false><<<rows, 512, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace moe
