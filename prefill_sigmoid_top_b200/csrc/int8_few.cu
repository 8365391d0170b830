// The dense int8 product for a few tokens in ONE launch, without the tensor cores: a decode step's projection reads
// little but its weights (2048 x 7168: 2.2 us at HBM speed), so what counts is the chain from launch to result.  A
// quantiser of its own, TMA rings, tensor memory and a split over a cluster make that chain 8.7 us (two launches);
// this kernel takes the weights straight into registers and multiplies with dp4a.
//
// One CTA of 32 warps per SM.  It issues its first weight loads, quantises the token rows for itself into shared
// memory (each thread one 16-byte vector of each row; 14 KB read per row of 7168, from L2), then its warps take output
// channels: kWays warps on one channel, each lane 16 codes at a time against every token's codes (dp4a: four exact
// products added to an int32 sum).  Codes, scales and sums are those of the other forms, so the results are the same
// bits.
//
// Bound: the chain; then HBM, and with more tokens the shared-memory reads of their codes beside it.  Measured, replayed
// with the weights in L2, this form / two launches (us): 2048 x 7168, 1 token 5.1 / 8.7, 2 tokens 6.2 / 10, 4 tokens
// 8.4 / 9.4, 8 tokens 13.6 / 9.6; 7168 x 7168, 4 tokens 16.3 / 12.5.  With other weights each time, as in a model's step:
// 2048 x 7168, 1 token 6.5, 2 tokens 7.4, 4 tokens 9.3 (8 in two launches 9.8); 7168 x 7168, 1 token 12.9, 2 tokens 14.6
// (4 in two launches 14.9); 40000 x 7168, 1 token 46 (6.2 TB/s).  So it is taken for one or two tokens, and for up to
// four where the weights are at most 16 MB (int8_few_takes).
//
// The last weight row may end at its K codes: where K is no multiple of 16 its last chunk is taken code by code (a form
// of its own, since the check and its code cost 0.1 to 0.4 us).
#include <algorithm>
#include <type_traits>

#include "int8_rows.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kWarps = 32;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxWays = 8;
constexpr int kMaxRowBytes = 64 * 1024;  // codes of all rows in shared memory

__device__ __forceinline__ uint4 load_weights(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int c) {
  c = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), c);
  c = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), c);
  c = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), c);
  return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), c);
}

// kRows: tokens, rounded up to a power of two (the codes of absent ones are 0).  kRagged: K is no multiple of 16.
template <int kRows, bool kRagged>
__global__ void __launch_bounds__(kThreads, 1) int8_few_kernel(const uint16_t* __restrict__ x, int64_t ldx, bool vectors,
                                                               const int8_t* __restrict__ w, int64_t ldw, int ways,
                                                               const Int8GemmArgs args) {
  extern __shared__ __align__(16) uint8_t codes[];  // [kRows][chunks * 16]
  __shared__ uint32_t top[kRows][kWarps];
  __shared__ RowScale row_scale[kRows];
  __shared__ float scale[kRows];
  __shared__ int part[kWarps][kRows];
  constexpr int kAhead = 8;  // 16-byte weight loads in flight per lane
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int M = args.M, N = args.rows_per_expert, K = args.kdim;
  const int chunks = (K + 15) / 16;  // of 16 codes
  const int pitch = chunks * 16;
  const int at_once = kWarps / ways;  // channels of the CTA
  const int way = warp % ways, mine = warp / ways;
  const int first = lane + 32 * way, step = 32 * ways;  // this lane's chunks

  // the first weights: they wait for nothing (a channel past the last reads the last one's and stores nothing).  The
  // last row may end at its K codes: of a chunk that it does not fill nothing is loaded here
  uint4 a[kAhead];
  auto fetch = [&](int group, int c0) {
    const int n = min(group * at_once + mine, N - 1);
    const int8_t* row = w + static_cast<int64_t>(n) * ldw;
    const int whole = kRagged && n == N - 1 ? K / 16 : chunks;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int c = c0 + step * i;
      a[i] = c < whole ? load_weights(row + 16 * static_cast<int64_t>(c)) : make_uint4(0, 0, 0, 0);
    }
  };
  const int groups = (N + at_once - 1) / at_once;
  int group = blockIdx.x;
  fetch(group, first);

  // ---- token rows -> codes
  const bool keep = vectors && K <= 8 * kThreads;  // a vector of each row per thread, read once
  uint4 v[kRows];
  if (keep) {
#pragma unroll
    for (int m = 0; m < kRows; ++m)
      v[m] = m < M && tid < K / 8 ? reinterpret_cast<const uint4*>(x + m * ldx)[tid] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int m = 0; m < kRows; ++m) {
    uint32_t t = 0;
    if (keep) {
      t = max_bits(max_bits(max_bits(max_bits(0, v[m].x), v[m].y), v[m].z), v[m].w);
    } else if (m < M && vectors) {
      const uint4* src = reinterpret_cast<const uint4*>(x + m * ldx);
      for (int c = tid; c < K / 8; c += kThreads) {
        const uint4 q = src[c];
        t = max_bits(max_bits(max_bits(max_bits(t, q.x), q.y), q.z), q.w);
      }
    } else if (m < M) {
#pragma unroll 4
      for (int c = tid; c < K; c += kThreads) t = max(t, static_cast<uint32_t>(x[m * ldx + c] & 0x7fffu));
    }
    t = __reduce_max_sync(0xffffffffu, t);
    if (lane == 0) top[m][warp] = t;
  }
  __syncthreads();
  if (warp < kRows) {
    const uint32_t t = __reduce_max_sync(0xffffffffu, top[warp][lane]);
    if (lane == 0) {
      row_scale[warp] = row_scale_of(t);
      scale[warp] = scale_value(t);
    }
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < kRows; ++m) {
    uint8_t* dst = codes + m * pitch;
    const RowScale s = row_scale[m];
    if (vectors) {
      const uint4* src = reinterpret_cast<const uint4*>(x + m * ldx);
      for (int c = tid; c < pitch / 8; c += kThreads) {
        uint2 o = make_uint2(0, 0);
        if (m < M && c < K / 8) {
          const uint4 q = keep ? v[m] : src[c];
          o = s.c != 0.0f ? codes_of_8<true>(q, s) : codes_of_8<false>(q, s);
        }
        reinterpret_cast<uint2*>(dst)[c] = o;
      }
    } else {
#pragma unroll 4
      for (int c = tid; c < pitch; c += kThreads)
        dst[c] = m < M && c < K ? static_cast<uint8_t>(code_of_1(x[m * ldx + c], s)) : 0;
    }
  }
  __syncthreads();

  // ---- channels
  for (; group < groups; group += gridDim.x) {
    const int n = group * at_once + mine;
    int acc[kRows];
#pragma unroll
    for (int m = 0; m < kRows; ++m) acc[m] = 0;
    for (int c0 = first; c0 < chunks; c0 += step * kAhead) {
      if (c0 != first) fetch(group, c0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int c = c0 + step * i;
        if (c < chunks) {
#pragma unroll
          for (int m = 0; m < kRows; ++m)
            acc[m] = dot16(a[i], *reinterpret_cast<const uint4*>(codes + m * pitch + 16 * c), acc[m]);
        }
      }
    }
    if (group + static_cast<int>(gridDim.x) < groups) fetch(group + gridDim.x, first);
#pragma unroll
    for (int m = 0; m < kRows; ++m) acc[m] = __reduce_add_sync(0xffffffffu, acc[m]);
    if (ways > 1) {
      if (lane == 0) {
#pragma unroll
        for (int m = 0; m < kRows; ++m) part[warp][m] = acc[m];
      }
      __syncthreads();
    }
    if (way == 0 && lane < M && n < N) {
      int sum = 0;
      if (ways > 1) {
        for (int q = 0; q < ways; ++q) sum += part[warp + q][lane];
      } else {
#pragma unroll
        for (int m = 0; m < kRows; ++m) sum = lane == m ? acc[m] : sum;
      }
      if (kRagged && n == N - 1)  // the rest of the last row
        for (int k = K / 16 * 16; k < K; ++k)
          sum += w[static_cast<int64_t>(n) * ldw + k] * static_cast<int8_t>(codes[lane * pitch + k]);
      const float r = int8_value(scale[lane], args.ch_scale0[n], sum);
      const size_t at = static_cast<size_t>(lane) * args.out_ld + n;
      if (args.out_f32)
        static_cast<float*>(args.out)[at] = r;
      else
        static_cast<__nv_bfloat16*>(args.out)[at] = __float2bfloat16_rn(r);
    }
    if (ways > 1) __syncthreads();  // the partial sums are read
  }
}

template <int kRows, bool kRagged>
cudaError_t launch_rows(const uint16_t* x, int64_t ldx, const int8_t* w, int64_t ldw, const Int8GemmArgs& args,
                        int num_sms, cudaStream_t stream) {
  auto kern = int8_few_kernel<kRows, kRagged>;
  int dev = 0;
  cudaError_t st = cudaGetDevice(&dev);
  if (st != cudaSuccess) return st;
  static bool done[64] = {};
  if (dev >= 64 || !done[dev]) {
    st = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRowBytes);
    if (st != cudaSuccess) return st;
    if (dev < 64) done[dev] = true;
  }
  const int N = args.rows_per_expert, K = args.kdim;
  // few channels: several warps on one, as long as there are warps for all of them and each has a load for every lane
  int ways = 1;
  while (ways < kMaxWays && static_cast<long long>(N) * 2 * ways <= static_cast<long long>(kWarps) * num_sms &&
         2 * 32 * 16 * ways <= K)
    ways *= 2;
  const int groups = (N + kWarps / ways - 1) / (kWarps / ways);
  const bool vectors = K % 8 == 0 && ldx % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0;
  const size_t smem = static_cast<size_t>(kRows) * ((K + 15) / 16 * 16);
  kern<<<std::min(groups, num_sms), kThreads, smem, stream>>>(x, ldx, vectors, w, ldw, ways, args);
  return cudaGetLastError();
}

}  // namespace

bool int8_few_takes(int64_t M, int64_t N, int64_t K) {
  if (M > 4 || (M > 2 && N * K > (16ll << 20))) return false;
  const int64_t rows = M <= 2 ? M : 4;
  return rows * ((K + 15) / 16 * 16) <= kMaxRowBytes;
}

cudaError_t launch_int8_few(const uint16_t* x, int64_t ldx, const int8_t* w, int64_t ldw, const Int8GemmArgs& args,
                            int num_sms, cudaStream_t stream) {
  auto rows = [&](auto ragged) {
    constexpr bool kRagged = decltype(ragged)::value;
    if (args.M <= 1) return launch_rows<1, kRagged>(x, ldx, w, ldw, args, num_sms, stream);
    if (args.M <= 2) return launch_rows<2, kRagged>(x, ldx, w, ldw, args, num_sms, stream);
    return launch_rows<4, kRagged>(x, ldx, w, ldw, args, num_sms, stream);
  };
  return args.kdim % 16 != 0 ? rows(std::true_type{}) : rows(std::false_type{});
}

}  // namespace moe
