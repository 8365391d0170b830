// Products of 8-bit integer rows on the 5th-generation tensor cores (tcgen05 kind::i8, int32 accumulators in
// tensor memory), fed by TMA: the expert projections of the plan with per-channel weight scales and per-token
// activation scales, and the dense product.
//
//   acc[n, j] = sum_k xq[n, k] wq[j, k]       exact: |codes| <= 127, so k <= 131072 terms stay below 2^31
//   value     = (sx[n] * sw[j]) * acc          fp32 (acc rounded once to 24 bits; int8_value has the range's ends)
//   up:    h[row, j]  = bf16(silu(gate) * up)      down: y[slot, j] = bf16(value)      dense: y[n, j]
//
// As in the bf16 kernels the weight rows are the M side of the MMA (128 per CTA) and the tokens its N side, one
// 128-byte swizzled row (128 codes, 4 MMAs of K = 32) per stage.  This file has the kernels for few tokens, where the
// product is a stream of weights (bound: HBM); int8_pair.cu those for many.
//
// Two ways to use the SMs:
//  * more tiles than SMs: one CTA per SM takes tiles in turn (static list); the producer runs ahead over tile
//    boundaries through a ring of about 200 KB, so the weight stream never stops, and the epilogue of a tile (other
//    accumulator) runs under the next one's loads;
//  * fewer (a dense layer for one token has N / 128 tiles): a cluster of S <= 8 CTAs takes a tile, each a share of K,
//    and adds up the int32 partial sums through distributed shared memory: exact, in any order, no workspace.
// Measured: 8 tokens x 16 of 256 experts, up (7168 -> 2048) 449 us at 6.75 TB/s; one token, 16 experts, down 49 us
// (235 MB: 35 us at that rate; 3 us before the stream runs, 5 us of a last round in which 8 of 148 SMs have a tile, the
// quantiser's launch).  One CTA per tile with two per SM measured within 5% either way, dp4a without the tensor cores
// 56 us.
//
// Both overlap the quantiser before them (programmatic dependent launch): barriers, tensor memory, the tile list and
// the first weight panels do not depend on it; token rows and scales are read after it has ended.
#include <algorithm>

#include "common.cuh"
#include "int8_plan.cuh"
#include "int8_rows.cuh"
#include "kernels.h"
#include "pair_ptx.cuh"
#include "tile_list.cuh"

namespace moe {
namespace {

constexpr int kBM = 128;          // weight rows per CTA
constexpr int kBK = 128;          // codes per stage
constexpr int kATile = kBM * kBK;
// Warps 0..3 = TMA producers (k-steps in turn: one producer thread issues a 16 KB copy every 0.48 us at best, which
// is 5.0 TB/s over all SMs), 4..7 = epilogue, 8 = MMA issuer.
constexpr int kProducerWarps = 4;
constexpr int kMmaWarp = 8;
constexpr int kThreads = 32 * (kMmaWarp + 1);

enum Mode { kUp = 0, kDown = 1, kDense = 2 };

constexpr int pow2_at_least(int v) {
  int p = 32;
  while (p < v) p <<= 1;
  return p;
}

template <int kMode, int kNmax, int kStages, int kBufs>
struct TCfg {
  static constexpr int kPanels = kMode == kUp ? 2 : 1;
  // Producer warps in use, a power of two.  A producer that has seen step i - kProducers freed knows that step
  // i - kProducers - kStages is consumed; its wait for step i tells phases apart only if that covers step
  // i - 2 kStages, so there are no more of them than stages.
  static constexpr int kProducers = kStages >= 4 ? 4 : (kStages >= 2 ? 2 : 1);
  static_assert(kProducers <= kProducerWarps && kProducers <= kStages, "a producer is at most one phase behind");
  static constexpr int kBTile = kNmax * kBK;
  static constexpr int kStageBytes = kPanels * kATile + kBTile;
  static constexpr int kTmemCols = pow2_at_least(kBufs * kPanels * kNmax);
  static constexpr int kMisc = kMode == kDense ? 1024 : 10240;  // barriers, flags, counts and tile prefix (E <= 1024)
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kMisc;
  static_assert(kBTile % 1024 == 0, "1024-byte alignment of the token tile");
  static_assert(kNmax % 32 == 0 && kNmax <= 128, "token widths; one gathering lane per four rows");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kStages * kStageBytes >= kPanels * kNmax * kBM * 4, "partial sums fit in the ring");
  // No more tensor memory than the CTA's share of shared memory, so that CTAs that fit on an SM never wait for
  // each other's columns.
  static_assert(kTmemCols * 454 <= kSmem, "tensor memory share (512 columns per 227 KB)");
};

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// gridDim.x / args.split clusters of args.split CTAs (no cluster when 1).  split > 1: at most one tile per cluster.
template <int kMode, int kNmax, int kStages, int kBufs>
__global__ void __launch_bounds__(kThreads, 1)
    int8_tile_kernel(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_a1,
                     const __grid_constant__ CUtensorMap tm_b, const Int8GemmArgs args) {
  using C = TCfg<kMode, kNmax, kStages, kBufs>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* misc = stages + kStages * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;      // [kBufs]
  uint64_t* acc_empty = acc_full + kBufs;    // [kBufs]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + kBufs);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* cnt = const_cast<int*>(abort_flag + 1);  // [E]
  int* prefix = cnt + 1024;                     // [E + 1]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int W = (args.rows_per_expert + kBM - 1) / kBM;
  const int split = args.split;
  const int rank = split > 1 ? static_cast<int>(cta_rank_in_cluster()) : 0;
  const int first = static_cast<int>(blockIdx.x) / split, step = static_cast<int>(gridDim.x) / split;
  const int dense_tiles = (args.M + kNmax - 1) / kNmax;

  // the counts' loads are under way while barriers and tensor memory are set up
  if (kMode != kDense && warp != kMmaWarp)
    for (int e = tid; e < args.E; e += 32 * kMmaWarp) cnt[e] = plan_count(args, e);
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    fence_mbar_init();
  }
  tc_fence_before_sync();
  __syncthreads();
  if (kMode != kDense) {
    if (warp == 0) build_tile_prefix<kNmax>(cnt, prefix, args.E, W, lane);
    __syncthreads();
  }
  const int total = kMode == kDense ? W * dense_tiles : prefix[args.E];
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  if (first >= total) {  // the whole cluster leaves
    if (total == 0) grid_dependency_wait();  // someone has to wait: the launch must not end before the quantiser
    if (warp == kMmaWarp) tmem_dealloc(tmem, C::kTmemCols);
    return;
  }
  const int nk_all = (args.kdim + kBK - 1) / kBK;
  const int k_lo = nk_all * rank / split, k_hi = nk_all * (rank + 1) / split;  // split <= nk_all

  struct Tile {
    int e, w, row0, nrows, N, count;
  };
  auto tile_at = [&](int idx) {
    Tile t;
    if (kMode == kDense) {
      t.e = 0;
      t.w = idx / dense_tiles;
      t.row0 = (idx % dense_tiles) * kNmax;
      t.count = args.M;
      t.nrows = min(kNmax, args.M - t.row0);
    } else {
      const TileCoord c = decode_tile<kNmax>(prefix, cnt, args.E, idx);
      t.e = c.e;
      t.w = c.w;
      t.count = cnt[c.e];
      t.nrows = min(kNmax, t.count - c.t * kNmax);
      t.row0 = args.offsets[c.e] + c.t * kNmax;
    }
    t.N = (t.nrows + 15) & ~15;
    return t;
  };
  // Scale and output row (-1: none) of row n of a tile.
  auto token_at = [&](const Tile& t, int n, float& scale, int& row) {
    scale = 0.0f;
    row = -1;
    if (n >= t.nrows) return;
    const int r = t.row0 + n;
    if (kMode == kDense) {
      scale = args.row_scale[r];
      row = r;
    } else {
      const int id = plan_slot(args, r);
      if (id >= 0) {
        scale = args.row_scale[kMode == kUp ? id / args.top_k : r];
        row = kMode == kUp ? r : id;
      } else {
        set_error(args.err, kErrInvalidInput);
      }
    }
  };
  auto store = [&](int row, int ch, float s0, float s1, float sx, int a0, int a1) {
    float v = int8_value(sx, s0, a0);
    if (kMode == kUp) v = silu_mul(v, int8_value(sx, s1, a1));
    const size_t at = static_cast<size_t>(row) * args.out_ld + ch;
    if (kMode == kDense && args.out_f32)
      static_cast<float*>(args.out)[at] = v;
    else
      static_cast<__nv_bfloat16*>(args.out)[at] = __float2bfloat16_rn(v);
  };

  constexpr int kProducers = C::kProducers;
  if (warp < kProducers) {
    // ------------------------------------------------ TMA producers: warp w loads every kProducers-th k-step
    if (warp == 0 && lane == 0) {
      prefetch_tensor_map(&tm_a0);
      if (kMode == kUp) prefetch_tensor_map(&tm_a1);
      prefetch_tensor_map(&tm_b);
    }
    const int nk = k_hi - k_lo;
    int it0 = 0, issued = 0;  // k-steps before this tile; behind the last one that this warp issued
    bool alive = true;
    // the weight panels of the first ring of k-steps, before the wait for the quantiser
    const int ahead = min(nk, kStages);
    {
      const Tile c = tile_at(first);
      const int a_row = c.e * args.rows_per_expert + c.w * kBM;
      const uint64_t pol = c.count <= kNmax ? l2_policy_evict_first() : l2_policy_evict_normal();
      if (lane == 0)
        for (int i = warp; i < ahead; i += kProducers) {
          uint8_t* st = stages + i * C::kStageBytes;
          mbar_arrive_expect_tx(&full[i], C::kPanels * kATile + c.N * kBK);
          tma_load_2d_hint(&tm_a0, &full[i], st, (k_lo + i) * kBK, a_row, pol);
          if (kMode == kUp) tma_load_2d_hint(&tm_a1, &full[i], st + kATile, (k_lo + i) * kBK, a_row, pol);
        }
      __syncwarp();
    }
    grid_dependency_wait();
    for (int tile = first; tile < total && alive; tile += step, it0 += nk) {
      const Tile c = tile_at(tile);
      const int a_row = c.e * args.rows_per_expert + c.w * kBM;
      // a panel that one token tile reads is streamed; others come from L2 the next time
      const uint64_t pol = c.count <= kNmax ? l2_policy_evict_first() : l2_policy_evict_normal();
      int tok[4] = {0, 0, 0, 0};  // gathered rows 4 lane .. 4 lane + 3 (past the tile's last: token 0, never stored)
      if (kMode == kUp) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (4 * lane + u < c.nrows) {
            const int id = plan_slot(args, c.row0 + 4 * lane + u);
            tok[u] = id >= 0 ? id / args.top_k : 0;
          }
      }
      for (int i = (warp - it0) & (kProducers - 1); i < nk; i += kProducers) {
        const int it = it0 + i, s = it % kStages, k = k_lo + i;
        uint8_t* st = stages + s * C::kStageBytes;
        uint8_t* bt = st + C::kPanels * kATile;
        const bool panels = it >= ahead;  // else they are on their way
        bool ok = true;
        if (panels && lane == 0) ok = mbar_wait_bounded(&empty[s], ((it / kStages) & 1) ^ 1, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          if (lane == 0) {
            *abort_flag = 1;
            set_error(args.err, kErrTimeout);
          }
          alive = false;
          break;
        }
        if (panels && lane == 0) {
          mbar_arrive_expect_tx(&full[s], C::kPanels * kATile + c.N * kBK);
          tma_load_2d_hint(&tm_a0, &full[s], st, k * kBK, a_row, pol);
          if (kMode == kUp) tma_load_2d_hint(&tm_a1, &full[s], st + kATile, k * kBK, a_row, pol);
        }
        __syncwarp();
        if (kMode == kUp) {
          if (4 * lane < c.N)
            tma_gather4(&tm_b, &full[s], bt + lane * 4 * kBK, k * kBK, tok[0], tok[1], tok[2], tok[3]);
        } else if (16 * lane < c.N) {
          tma_load_2d(&tm_b, &full[s], bt + lane * 16 * kBK, k * kBK, c.row0 + 16 * lane);
        }
        issued = it + 1;
      }
    }
    // no exit while copies of this CTA may still land
    if (lane == 0) {
      const int lo = max(0, (alive ? it0 : issued) - kStages);  // each slot's last use
      for (int k = lo + ((warp - lo) & (kProducers - 1)); k < issued; k += kProducers)
        if (!mbar_wait_bounded(&full[k % kStages], (k / kStages) & 1, nullptr)) {
          set_error(args.err, kErrTimeout);
          break;
        }
    }
    __syncwarp();
  } else if (warp < kProducerWarps) {
    // idle
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0) {
      int it = 0, j = 0, committed = 0;  // tiles
      bool alive = true;
      for (int tile = first; tile < total && alive; tile += step, ++j) {
        const uint32_t idesc = umma_idesc_s8(kBM, tile_at(tile).N);
        const int buf = j % kBufs;
        if (!mbar_wait_bounded(&acc_empty[buf], ((j / kBufs) & 1) ^ 1, abort_flag)) {
          *abort_flag = 1;
          set_error(args.err, kErrTimeout);
          break;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem + buf * C::kPanels * kNmax;
        for (int k = k_lo; k < k_hi; ++k, ++it) {
          const int s = it % kStages;
          if (!mbar_wait_bounded(&full[s], (it / kStages) & 1, abort_flag)) {
            *abort_flag = 1;
            set_error(args.err, kErrTimeout);
            alive = false;
            break;
          }
          tc_fence_after_sync();
          uint8_t* st = stages + s * C::kStageBytes;
          const uint64_t da0 = umma_desc_sw128(st), da1 = umma_desc_sw128(st + kATile);
          const uint64_t db = umma_desc_sw128(st + C::kPanels * kATile);
#pragma unroll
          for (int kk = 0; kk < kBK / 32; ++kk) {
            const uint32_t acc = (k > k_lo || kk > 0) ? 1u : 0u;
            umma_s8_ss(d, da0 + 2 * kk, db + 2 * kk, idesc, acc);
            if (kMode == kUp) umma_s8_ss(d + kNmax, da1 + 2 * kk, db + 2 * kk, idesc, acc);
          }
          umma_commit(&empty[s]);
        }
        umma_commit(&acc_full[buf]);  // also after an abort, so that the epilogue is not left waiting
        committed = j + 1;
      }
      // after an abort nobody else waits for the products under way, which still read the ring
      if (*abort_flag && committed > 0)
        mbar_wait_bounded(&acc_full[(committed - 1) % kBufs], ((committed - 1) / kBufs) & 1, nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue: a warp reads the tensor-memory lanes of its quarter
    grid_dependency_wait();
    const int q = warp & 3;
    int j = 0;
    for (int tile = first; tile < total; tile += step, ++j) {
      const Tile c = tile_at(tile);
      const int buf = j % kBufs;
      const int ch = c.w * kBM + q * 32 + lane;
      const bool col_ok = ch < args.rows_per_expert;
      const size_t ch_at = static_cast<size_t>(c.e) * args.rows_per_expert + ch;
      const float s0 = col_ok ? args.ch_scale0[ch_at] : 0.0f;
      const float s1 = kMode == kUp && col_ok ? args.ch_scale1[ch_at] : 0.0f;
      float tok_s;
      int tok_row;
      token_at(c, lane, tok_s, tok_row);  // of row `lane` of the 32-row chunk
      bool ok = true;
      if (lane == 0) ok = mbar_wait_bounded(&acc_full[buf], (j / kBufs) & 1, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      tc_fence_after_sync();
      const bool go = __shfl_sync(0xffffffffu, ok && !*abort_flag, 0);
      if (!go) {
        if (lane == 0 && !ok) set_error(args.err, kErrTimeout);
        break;
      }
      const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * C::kPanels * kNmax;
      int* red = reinterpret_cast<int*>(stages) + q * 32 + lane;  // split: [panel][row][128] partial sums
      for (int n0 = 0; n0 < c.N; n0 += 16) {
        if (n0 > 0 && (n0 & 31) == 0) token_at(c, n0 + lane, tok_s, tok_row);
        uint32_t d0[16], d1[16];
        tmem_load_16(lane_base + n0, d0);
        if (kMode == kUp) tmem_load_16(lane_base + kNmax + n0, d1);
        tmem_load_wait();
        if (split > 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (n0 + i >= c.nrows) break;
            red[(n0 + i) * kBM] = static_cast<int>(d0[i]);
            if (kMode == kUp) red[(kNmax + n0 + i) * kBM] = static_cast<int>(d1[i]);
          }
          continue;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (n0 + i >= c.nrows) break;
          const int row = __shfl_sync(0xffffffffu, tok_row, (n0 + i) & 31);
          const float sx = __shfl_sync(0xffffffffu, tok_s, (n0 + i) & 31);
          if (row >= 0 && col_ok)
            store(row, ch, s0, s1, sx, static_cast<int>(d0[i]), kMode == kUp ? static_cast<int>(d1[i]) : 0);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_one(&acc_empty[buf]);
    }
  }
  if (split > 1) {
    // every CTA of the cluster takes a share of the tile's rows and adds the others' partial sums to its own
    cluster_sync_all();
    const Tile c = tile_at(first);
    if (warp >= kProducerWarps && warp < kMmaWarp && !*abort_flag) {
      const int q = warp & 3;
      const int ch = c.w * kBM + q * 32 + lane;
      const bool col_ok = ch < args.rows_per_expert;
      const size_t ch_at = static_cast<size_t>(c.e) * args.rows_per_expert + ch;
      const float s0 = col_ok ? args.ch_scale0[ch_at] : 0.0f;
      const float s1 = kMode == kUp && col_ok ? args.ch_scale1[ch_at] : 0.0f;
      const int* mine = reinterpret_cast<const int*>(stages) + q * 32 + lane;
      for (int n = c.nrows * rank / split; n < c.nrows * (rank + 1) / split; ++n) {
        float sx;
        int row;
        token_at(c, n, sx, row);
        int a0 = 0, a1 = 0;
        for (int r = 0; r < split; ++r) {
          a0 += ld_cluster_s32(cluster_addr(mine + n * kBM, r));
          if (kMode == kUp) a1 += ld_cluster_s32(cluster_addr(mine + (kNmax + n) * kBM, r));
        }
        if (row >= 0 && col_ok) store(row, ch, s0, s1, sx, a0, a1);
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while another reads its sums
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, C::kTmemCols);
}

template <int kMode, int kNmax, int kStages, int kBufs>
cudaError_t launch_tiles(const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b, const Int8GemmArgs& args,
                         unsigned grid, cudaStream_t stream) {
  using C = TCfg<kMode, kNmax, kStages, kBufs>;
  auto kern = int8_tile_kernel<kMode, kNmax, kStages, kBufs>;
  int dev = 0;
  cudaError_t st = cudaGetDevice(&dev);
  if (st != cudaSuccess) return st;
  static bool done[64] = {};
  if (dev >= 64 || !done[dev]) {
    st = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (st != cudaSuccess) return st;
    if (dev < 64) done[dev] = true;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(args.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = args.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a0, a1, b, args);
}

// kDeep: ring stages of the persistent form (one CTA per SM); kShallow: of the split form (two per SM).
template <int kMode, int kNmax, int kDeep, int kShallow, int kBufs>
cudaError_t launch_form(const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b, Int8GemmArgs args,
                        int num_sms, cudaStream_t stream) {
  const long long W = (args.rows_per_expert + kBM - 1) / kBM;
  long long tiles;  // of the plan: an upper bound that needs no look at it
  if (kMode == kDense) {
    tiles = (args.M + kNmax - 1) / kNmax;
  } else {
    const long long mk = static_cast<long long>(args.M) * args.top_k;
    tiles = mk / kNmax + (mk < args.E ? mk : args.E);
  }
  tiles *= W;
  if (tiles >= (1ll << 31)) return cudaErrorInvalidValue;
  const int nk = (args.kdim + kBK - 1) / kBK;
  args.split = int8_tile_split(tiles, nk, num_sms);
  if (args.split > 1)
    return launch_tiles<kMode, kNmax, kShallow, 1>(a0, a1, b, args, static_cast<unsigned>(tiles * args.split), stream);
  return launch_tiles<kMode, kNmax, kDeep, kBufs>(a0, a1, b, args,
                                                  static_cast<unsigned>(std::min<long long>(tiles, num_sms)), stream);
}

}  // namespace

int int8_tile_split(long long tiles, int nk, int num_sms) {
  int split = 1;
  while (split < 8 && 4 * split <= nk && split * tiles <= num_sms) split *= 2;
  return split;
}

cudaError_t launch_int8_up(const CUtensorMap& w_gate, const CUtensorMap& w_up, const CUtensorMap& x_rows,
                           const Int8GemmArgs& args, int num_sms, cudaStream_t stream) {
  return launch_form<kUp, 32, 5, 2, 2>(w_gate, w_up, x_rows, args, num_sms, stream);
}

cudaError_t launch_int8_down(const CUtensorMap& w_down, const CUtensorMap& h_rows, const Int8GemmArgs& args,
                             int num_sms, cudaStream_t stream) {
  return launch_form<kDown, 32, 10, 4, 2>(w_down, w_down, h_rows, args, num_sms, stream);
}

cudaError_t launch_int8_dense(const CUtensorMap& w, const CUtensorMap& x_rows, const Int8GemmArgs& args, int nmax,
                              int num_sms, cudaStream_t stream) {
  if (nmax <= 32) return launch_form<kDense, 32, 10, 5, 2>(w, w, x_rows, args, num_sms, stream);
  return launch_form<kDense, 128, 6, 3, 2>(w, w, x_rows, args, num_sms, stream);
}

}  // namespace moe
