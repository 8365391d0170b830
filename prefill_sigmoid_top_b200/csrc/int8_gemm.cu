// Products of 8-bit integer rows on the 5th-generation tensor cores (tcgen05 kind::i8, int32 accumulators in
// tensor memory), fed by TMA: the expert projections of the plan with per-channel weight scales and per-token
// activation scales, and the dense product.
//
//   acc[n, j] = sum_k xq[n, k] wq[j, k]       exact: |codes| <= 127, so k <= 131072 terms stay below 2^31
//   value     = (sx[n] * sw[j]) * acc          fp32 (acc rounded once to 24 bits)
//   up:    h[row, j]  = bf16(silu(gate) * up)      down: y[slot, j] = bf16(value)      dense: y[n, j]
//
// As in the bf16 kernels the weight rows are the M side of the MMA (128 per CTA) and the tokens its N side, one
// 128-byte swizzled row (128 codes, 4 MMAs of K = 32) per stage.  One CTA computes one tile of 128 channels x up to
// kNmax tokens.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kBM = 128;          // weight rows per CTA
constexpr int kBK = 128;          // codes per stage
constexpr int kATile = kBM * kBK;

enum Mode { kUp = 0, kDown = 1, kDense = 2 };

constexpr int pow2_at_least(int v) {
  int p = 32;
  while (p < v) p <<= 1;
  return p;
}

template <int kMode, int kNmax, int kStages>
struct TCfg {
  static constexpr int kPanels = kMode == kUp ? 2 : 1;
  static constexpr int kBTile = kNmax * kBK;
  static constexpr int kStageBytes = kPanels * kATile + kBTile;
  static constexpr int kTmemCols = pow2_at_least(kPanels * kNmax);
  static constexpr int kMisc = (256 + 12 * kNmax + 1023) / 1024 * 1024;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kMisc;
  static_assert(kBTile % 1024 == 0, "1024-byte alignment of the token tile");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kStages * kStageBytes >= 4096, "expert counts are staged in the ring before it is used");
  // No more tensor memory than the CTA's share of shared memory, so that CTAs that fit on an SM never wait for
  // each other's columns.
  static_assert(kTmemCols * 454 <= kSmem, "tensor memory share (512 columns per 227 KB)");
};

template <int kMode, int kNmax, int kStages>
__global__ void __launch_bounds__(128, 1)
    int8_tile_kernel(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_a1,
                     const __grid_constant__ CUtensorMap tm_b, const Int8GemmArgs args) {
  using C = TCfg<kMode, kNmax, kStages>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* misc = stages + kStages * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc);
  uint64_t* empty = full + kStages;
  uint64_t* accf = empty + kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accf + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* info = const_cast<int*>(abort_flag + 1);  // expert, token tile, weight tile
  int* src = reinterpret_cast<int*>(misc + 256); // [kNmax] up: token of the row
  int* dst = src + kNmax;                        // [kNmax] output row, -1: none
  float* scale = reinterpret_cast<float*>(dst + kNmax);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int W = (args.rows_per_expert + kBM - 1) / kBM;

  // ---- the tile of this CTA: experts in order, then weight tile, then token tile (fastest), so that the tiles
  // that read one weight panel start together
  if (tid == 0) {
    *abort_flag = 0;
    info[0] = -1;
    info[1] = info[2] = 0;
  }
  int count_e, off_e;
  if (kMode == kDense) {
    const int ntiles = (args.M + kNmax - 1) / kNmax;
    __syncthreads();
    if (tid == 0) {
      info[0] = 0;
      info[1] = static_cast<int>(blockIdx.x) % ntiles;
      info[2] = static_cast<int>(blockIdx.x) / ntiles;
    }
    __syncthreads();
    count_e = args.M;
    off_e = 0;
  } else {
    int* cnt = reinterpret_cast<int*>(stages);
    for (int e = tid; e < args.E; e += 128) cnt[e] = args.counts[e];
    __syncthreads();
    if (warp == 0) {
      const int linear = blockIdx.x;
      const int per = (args.E + 31) / 32;
      const int lo = min(args.E, lane * per), hi = min(args.E, lo + per);
      int sum = 0;
      for (int e = lo; e < hi; ++e) sum += W * ((cnt[e] + kNmax - 1) / kNmax);
      int incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      int t = incl - sum;
      if (linear >= t && linear < incl) {
        for (int e = lo; e < hi; ++e) {
          const int ntiles = (cnt[e] + kNmax - 1) / kNmax;
          if (linear < t + W * ntiles) {
            info[0] = e;
            info[1] = (linear - t) % ntiles;
            info[2] = (linear - t) / ntiles;
            break;
          }
          t += W * ntiles;
        }
      }
    }
    __syncthreads();
    if (info[0] < 0) return;  // past the last tile
    count_e = cnt[info[0]];
    off_e = args.offsets[info[0]];
  }
  const int e = info[0], local = info[1], wt = info[2];
  const int nrows = min(kNmax, count_e - local * kNmax);
  const int N = (nrows + 15) & ~15;
  const int row0 = off_e + local * kNmax;
  const int nslots = args.M * args.top_k;
  for (int n = tid; n < N; n += 128) {
    int s = 0, d = -1;
    float f = 0.0f;
    if (n < nrows) {
      if (kMode == kDense) {
        d = row0 + n;
        f = args.row_scale[d];
      } else {
        const int id = args.sorted_ids[row0 + n];
        if (id >= 0 && id < nslots) {
          s = id / args.top_k;
          d = kMode == kUp ? row0 + n : id;
          f = args.row_scale[kMode == kUp ? s : row0 + n];
        } else {
          set_error(args.err, kErrInvalidInput);
        }
      }
    }
    src[n] = s;
    dst[n] = d;
    scale[n] = f;
  }
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(accf, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();  // also ends the use of the ring as scratch
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int nk = (args.kdim + kBK - 1) / kBK;
  const int a_row = e * args.rows_per_expert + wt * kBM;

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    if (lane == 0) {
      prefetch_tensor_map(&tm_a0);
      if (kMode == kUp) prefetch_tensor_map(&tm_a1);
      prefetch_tensor_map(&tm_b);
    }
    // a panel that one token tile reads is streamed; others come from L2 the next time
    const uint64_t pol = count_e <= kNmax ? l2_policy_evict_first() : l2_policy_evict_normal();
    int issued = 0;
    for (int k = 0; k < nk; ++k) {
      const int s = k % kStages;
      bool ok = true;
      if (lane == 0) ok = mbar_wait_bounded(&empty[s], ((k / kStages) & 1) ^ 1, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        if (lane == 0) {
          *abort_flag = 1;
          set_error(args.err, kErrTimeout);
        }
        break;
      }
      uint8_t* st = stages + s * C::kStageBytes;
      uint8_t* bt = st + C::kPanels * kATile;
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[s], C::kPanels * kATile + N * kBK);
        tma_load_2d_hint(&tm_a0, &full[s], st, k * kBK, a_row, pol);
        if (kMode == kUp) tma_load_2d_hint(&tm_a1, &full[s], st + kATile, k * kBK, a_row, pol);
      }
      __syncwarp();
      if (kMode == kUp) {
        for (int i = lane; i < N / 4; i += 32)
          tma_gather4(&tm_b, &full[s], bt + i * 4 * kBK, k * kBK, src[4 * i], src[4 * i + 1], src[4 * i + 2],
                      src[4 * i + 3]);
      } else {
        for (int i = lane; i < N / 16; i += 32)
          tma_load_2d(&tm_b, &full[s], bt + i * 16 * kBK, k * kBK, row0 + 16 * i);
      }
      issued = k + 1;
    }
    // no exit while copies of this CTA may still land
    if (lane == 0) {
      for (int k = max(0, issued - kStages); k < issued; ++k)
        if (!mbar_wait_bounded(&full[k % kStages], (k / kStages) & 1, nullptr)) {
          set_error(args.err, kErrTimeout);
          break;
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idesc = umma_idesc_s8(kBM, N);
      for (int k = 0; k < nk; ++k) {
        const int s = k % kStages;
        if (!mbar_wait_bounded(&full[s], (k / kStages) & 1, abort_flag)) {
          *abort_flag = 1;
          set_error(args.err, kErrTimeout);
          break;
        }
        tc_fence_after_sync();
        uint8_t* st = stages + s * C::kStageBytes;
        const uint64_t da0 = umma_desc_sw128(st), da1 = umma_desc_sw128(st + kATile);
        const uint64_t db = umma_desc_sw128(st + C::kPanels * kATile);
#pragma unroll
        for (int kk = 0; kk < kBK / 32; ++kk) {
          const uint32_t acc = (k | kk) != 0 ? 1u : 0u;
          umma_s8_ss(tmem, da0 + 2 * kk, db + 2 * kk, idesc, acc);
          if (kMode == kUp) umma_s8_ss(tmem + kNmax, da1 + 2 * kk, db + 2 * kk, idesc, acc);
        }
        umma_commit(&empty[s]);
      }
      umma_commit(accf);  // also after an abort, so that the epilogue is not left waiting
    }
    __syncwarp();
  }

  // ---------------------------------------------------- epilogue: warp w owns channels 32 w .. 32 w + 31
  bool ok = true;
  if (lane == 0) ok = mbar_wait_bounded(accf, 0, nullptr);
  ok = __shfl_sync(0xffffffffu, ok, 0);
  tc_fence_after_sync();
  if (!ok && lane == 0) set_error(args.err, kErrTimeout);
  const bool go = __shfl_sync(0xffffffffu, ok && !*abort_flag, 0);
  const int j = wt * kBM + warp * 32 + lane;
  const bool col_ok = j < args.rows_per_expert;
  if (go) {
    const size_t ch = static_cast<size_t>(e) * args.rows_per_expert + j;
    const float s0 = col_ok ? args.ch_scale0[ch] : 0.0f;
    const float s1 = kMode == kUp && col_ok ? args.ch_scale1[ch] : 0.0f;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    for (int c = 0; c < N; c += 16) {
      uint32_t d0[16], d1[16];
      tmem_load_16(lane_base + c, d0);
      if (kMode == kUp) tmem_load_16(lane_base + kNmax + c, d1);
      tmem_load_wait();
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int n = c + q;
        const int row = n < nrows ? dst[n] : -1;
        if (row < 0 || !col_ok) continue;
        const float sx = scale[n];
        const size_t at = static_cast<size_t>(row) * args.out_ld + j;
        float v = (sx * s0) * static_cast<float>(static_cast<int>(d0[q]));
        if (kMode == kUp) v = silu_mul(v, (sx * s1) * static_cast<float>(static_cast<int>(d1[q])));
        if (kMode == kDense && args.out_f32)
          static_cast<float*>(args.out)[at] = v;
        else
          static_cast<__nv_bfloat16*>(args.out)[at] = __float2bfloat16_rn(v);
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

template <int kMode, int kNmax, int kStages>
cudaError_t launch_tiles(const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b, const Int8GemmArgs& args,
                         cudaStream_t stream) {
  using C = TCfg<kMode, kNmax, kStages>;
  auto kern = int8_tile_kernel<kMode, kNmax, kStages>;
  int dev = 0;
  cudaError_t st = cudaGetDevice(&dev);
  if (st != cudaSuccess) return st;
  static bool done[64] = {};
  if (dev >= 64 || !done[dev]) {
    st = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (st != cudaSuccess) return st;
    if (dev < 64) done[dev] = true;
  }
  const long long W = (args.rows_per_expert + kBM - 1) / kBM;
  long long tiles;  // of tokens: an upper bound that needs no look at the plan
  if (kMode == kDense) {
    tiles = (args.M + kNmax - 1) / kNmax;
  } else {
    const long long mk = static_cast<long long>(args.M) * args.top_k;
    tiles = mk / kNmax + (mk < args.E ? mk : args.E);
  }
  if (W * tiles >= (1ll << 31)) return cudaErrorInvalidValue;
  kern<<<static_cast<unsigned>(W * tiles), 128, C::kSmem, stream>>>(a0, a1, b, args);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_int8_up(const CUtensorMap& w_gate, const CUtensorMap& w_up, const CUtensorMap& x_rows,
                           const Int8GemmArgs& args, int nmax, cudaStream_t stream) {
  if (nmax <= 32) return launch_tiles<kUp, 32, 3>(w_gate, w_up, x_rows, args, stream);
  return launch_tiles<kUp, 128, 4>(w_gate, w_up, x_rows, args, stream);
}

cudaError_t launch_int8_down(const CUtensorMap& w_down, const CUtensorMap& h_rows, const Int8GemmArgs& args, int nmax,
                             cudaStream_t stream) {
  if (nmax <= 32) return launch_tiles<kDown, 32, 5>(w_down, w_down, h_rows, args, stream);
  return launch_tiles<kDown, 128, 3>(w_down, w_down, h_rows, args, stream);
}

cudaError_t launch_int8_dense(const CUtensorMap& w, const CUtensorMap& x_rows, const Int8GemmArgs& args, int nmax,
                              cudaStream_t stream) {
  if (nmax <= 32) return launch_tiles<kDense, 32, 5>(w, w, x_rows, args, stream);
  return launch_tiles<kDense, 128, 3>(w, w, x_rows, args, stream);
}

}  // namespace moe
