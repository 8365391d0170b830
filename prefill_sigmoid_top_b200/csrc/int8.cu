// Symmetric 8-bit rows: the activation and weight form of the int8 projections.
//   a = max |v| of the row;  scale = a / 127 (fp32);  code = rint(127 v / a), ties to even;  a = 0: scale 0, codes 0.
// The codes are those of exact arithmetic: v and a are bf16, so 127 v (15 significant bits) is exact in fp32, and a
// quotient that is not a tie is at least 1.5e-5 (relative) away from one, far more than the rounding of the
// division.  A row that holds an infinity or a NaN gets the scale NaN and codes 0: its products are NaN.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kQThreads = 128;  // one CTA per row

// |v| as bf16 bits: ordered like the magnitudes, infinity 0x7f80, NaN above.
__global__ void __launch_bounds__(kQThreads) quantize_int8_kernel(Int8RowsArgs a) {
  __shared__ uint32_t part[kQThreads / 32];
  const int tid = threadIdx.x;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    int64_t src_row = r;
    if (a.sorted_ids != nullptr) {
      if (r >= *a.ntpp) return;
      const int id = a.sorted_ids[r];
      if (id < 0 || id >= a.nslots) continue;  // padding
    }
    const uint16_t* src = a.src + src_row * a.ld;
    uint32_t top = 0;
    for (int c = tid; c < a.cols; c += kQThreads) top = max(top, static_cast<uint32_t>(src[c] & 0x7fffu));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) part[tid >> 5] = top;
    __syncthreads();
    top = 0;
#pragma unroll
    for (int q = 0; q < kQThreads / 32; ++q) top = max(top, part[q]);
    __syncthreads();
    const float amax = __uint_as_float(top << 16);
    const bool fin = top < 0x7f80u;
    if (tid == 0) a.scales[r] = fin ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7fffffffu);
    // rows above 2^100 are divided by 2^32 first, so that 127 v stays finite (what drops below the range is code 0)
    const float pre = amax > 0x1p100f ? 0x1p-32f : 1.0f;
    int8_t* dst = a.codes + r * a.pitch;
    for (int c = tid; c < a.cols; c += kQThreads) {
      const float v = __uint_as_float(static_cast<uint32_t>(src[c]) << 16) * pre;
      const float q = fin && top != 0 ? rintf(__fdiv_rn(127.0f * v, amax * pre)) : 0.0f;
      dst[c] = static_cast<int8_t>(static_cast<int>(q));
    }
  }
}

}  // namespace

cudaError_t launch_quantize_int8(const Int8RowsArgs& a, cudaStream_t stream) {
  const int64_t grid = a.rows < (1 << 20) ? a.rows : (1 << 20);
  quantize_int8_kernel<<<static_cast<unsigned>(grid), kQThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
