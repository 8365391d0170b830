// Products of 8-bit rows on 2-SM pairs (tcgen05 kind::i8 with cta_group::2) for many tokens: the plan's expert
// projections and the dense product, the int8 form of the bf16 pair kernels (same pair protocol and warp roles).
//
// Why pairs: a single SM that computes 128 channels x 128 tokens reads 32 KB of shared-memory operands for every
// 262 clocks of int8 MMA, twice what L2 delivers to it.  A pair computes 512 channels x 256 tokens: each CTA reads
// its own 2 x 128 channels and half of the tokens, 48 KB for 1024 clocks.
//
// Tile: a weight block w of one expert x up to kNmax tokens; CTA r of the pair holds two boxes of 128 weight rows:
//   up:          rows 256 w + 128 r.. of W_gate and of W_up (the two accumulators of silu(gate) * up);
//   down, dense: rows 512 w + 128 r.. and 512 w + 256 + 128 r.. (two accumulators of M = 256 each);
//   dense with one box: rows 256 w + 128 r.. (one accumulator of M = 256, so two sets of 256 tokens; smaller tiles fill
//                the pairs better, 2048 x 2048 x 7168 44 -> 36 us; the down projection with it: 812 -> 882 us);
// and token rows [r N/2, (r + 1) N/2) of the tile's N (its tokens rounded up to 32, the width step of this MMA).
// Channels past the expert's last row are computed and not stored.
//
// Warps (640 threads): 0..2 = producers, 3 = MMA issuer (leader), 4..19 = epilogue.  A stage holds the weight boxes
// and the token rows of one k-step; the producer warps take stages in turn.  One producer thread per operand, as the
// bf16 pair kernels have, needs about 0.7 us for a stage however wide its tokens (the wake-up of its wait and the issue
// of its copies in series); with three: 8192 x 7168 x 7168 314 -> 299 us, prefill up 1467 -> 1403 us, batch up 1128 ->
// 1102 us.
//
// Measured, replayed alone / as calls in a row, which run under the power cap, with their quantisers: 8192 x 7168 x 7168
// 301 / 365 us (2.8 / 2.3 Pop/s), batch up (512 tokens, 256 experts) 1.12 / 1.21 ms (6.8 / 6.3 TB/s), skewed prefill
// (2048 tokens) up 1.41 / 1.70 ms, down 0.80 / 0.96 ms.  Bound: HBM for the experts with few tokens, power and the
// operand feed for the busy ones (tensor pipe 67% active at 4096 x 7168 x 7168).
//
// The launch overlaps the kernel before it (programmatic dependent launch): set-up and the first weight boxes come
// before the wait for it.  Every mbarrier wait is bounded; a timeout sets the error word and unwinds, and both CTAs
// still meet at the last cluster barrier.
#include "common.cuh"
#include "int8_plan.cuh"
#include "int8_rows.cuh"
#include "kernels.h"
#include "pair_ptx.cuh"
#include "tile_list.cuh"

namespace moe {
namespace {

constexpr int kBM = 128;              // weight rows per box
constexpr int kBK = 128;              // codes per stage
constexpr int kBoxBytes = kBM * kBK;  // 16 KB
constexpr int kBRows = 32;            // rows per token box
constexpr int kProducers = 3;
constexpr int kMmaWarp = 3;
constexpr int kFirstEpi = 4;
constexpr int kEpiWarps = 16;
constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
constexpr uint64_t kDrainNs = 10ull * 1000ull * 1000ull;  // after an abort

enum Mode { kUp = 0, kDown = 1, kDense = 2 };

template <int kNmax, int kStages, int kBoxes>
struct PCfg {
  static constexpr int kHalf = kNmax / 2;
  static constexpr int kABytes = kBoxes * kBoxBytes;
  static constexpr int kStage = kABytes + kHalf * kBK;
  static constexpr int kAccCols = kBoxes * kNmax;
  static constexpr int kAccBufs = 512 / kAccCols;
  static_assert(kAccBufs == 1 || kAccBufs == 2, "barriers for two accumulator sets");
  static constexpr int kMisc = 10240;  // barriers, flags, counts and tile prefix over the experts (E <= 1024)
  static constexpr int kSmem = 1024 + kStages * kStage + kMisc;
  static_assert(kNmax == 128 || kNmax == 256, "token-tile widths");
  // A producer that has seen step i - kProducers freed knows that step i - kProducers - kStages is consumed; its wait
  // for step i tells phases apart only if that covers step i - 2 kStages.
  static_assert(kStages >= kProducers, "a producer is at most one phase behind");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kSmem > 116 * 1024, "one CTA per SM: it owns all 512 tensor-memory columns");
};

// Up gathers its token rows from the codes of x by token id (tile::gather4); down and dense read consecutive rows.  With
// the copies spread over three producer warps the gather costs no more than a copy of the codes in plan order made
// before (prefill, 256-row tiles: 1434 us against 1454 with that pass; batch, 128-row tiles: 1099 against 1176).
template <int kMode, int kNmax, int kStages, int kBoxes>
__global__ void __launch_bounds__(kThreads, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_a1,
                     const __grid_constant__ CUtensorMap tm_b, const Int8GemmArgs args) {
  using C = PCfg<kNmax, kStages, kBoxes>;
  static_assert(kBoxes == 2 || (kBoxes == 1 && kMode == kDense), "weight boxes per CTA");
  constexpr bool kGather = kMode == kUp;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* misc = ring + kStages * C::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;    // [2] (the leader's counts both CTAs' epilogue warps)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* cnt = const_cast<int*>(abort_flag + 1);  // [E]
  int* prefix = cnt + 1024;                     // [E + 1]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cta_rank_in_cluster();
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x) >> 1;
  const int npairs = static_cast<int>(gridDim.x) >> 1;
  const int E = args.E;
  constexpr int kBlock = kMode == kUp ? 2 * kBM : 2 * kBoxes * kBM;  // channels of a weight block
  const int W = (args.rows_per_expert + kBlock - 1) / kBlock;
  const int tw = kMode == kDense ? args.tile_n : kNmax;     // tokens per tile
  const int dense_tiles = (args.M + tw - 1) / tw;

  if (kMode != kDense)
    for (int e = tid; e < E; e += kThreads) cnt[e] = plan_count(args, e);
  if (tid == 0) *abort_flag = 0;
  __syncthreads();
  if (kMode != kDense && warp == 0) build_tile_prefix<kNmax>(cnt, prefix, E, W, lane);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  const int total = kMode == kDense ? W * dense_tiles : prefix[E];
  if (pair >= total) {  // both CTAs of a pair see the same count
    if (total == 0) grid_dependency_wait();  // someone has to wait: the launch must not end before the quantiser
    return;
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  cluster_sync_all();  // the peer's barriers are initialised and both CTAs hold tensor memory
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int nk = (args.kdim + kBK - 1) / kBK;

  struct Tile {
    int e, w, row0, nrows, N, count;
  };
  auto tile_at = [&](int idx) {
    Tile t;
    if (kMode == kDense) {
      t.e = 0;
      t.w = idx / dense_tiles;
      t.row0 = (idx % dense_tiles) * tw;
      t.count = args.M;
      t.nrows = min(tw, args.M - t.row0);
    } else {
      const TileCoord c = decode_tile<kNmax>(prefix, cnt, E, idx);
      t.e = c.e;
      t.w = c.w;
      t.count = cnt[c.e];
      t.nrows = min(kNmax, t.count - c.t * kNmax);
      t.row0 = args.offsets[c.e] + c.t * kNmax;
    }
    t.N = (t.nrows + 31) & ~31;
    return t;
  };
  // Scale and output row (-1: none) of row n of a tile.
  auto token_at = [&](const Tile& t, int n, float& scale, int& to) {
    scale = 0.0f;
    to = -1;
    if (n >= t.nrows) return;
    const int row = t.row0 + n;
    if (kMode == kDense) {
      scale = args.row_scale[row];
      to = row;
    } else {
      const int id = plan_slot(args, row);
      if (id >= 0) {
        scale = args.row_scale[kMode == kUp ? id / args.top_k : row];
        to = kMode == kUp ? row : id;
      } else {
        set_error(args.err, kErrInvalidInput);
      }
    }
  };

  if (warp < kProducers) {
    // ------------------------------------------------ producers (both CTAs): warp w loads every third k-step
    if (warp == 0 && lane == 0) {
      prefetch_tensor_map(&tm_a0);
      if (kMode == kUp) prefetch_tensor_map(&tm_a1);
      prefetch_tensor_map(&tm_b);
    }
    const uint64_t pol_b = l2_policy_evict_normal();
    int it0 = 0;  // k-steps before this tile
    bool alive = true;
    // the weight boxes of the first ring of k-steps, before the wait for the kernel that writes the token rows
    const int ahead = min(nk, kStages);
    {
      const Tile c = tile_at(pair);
      const uint64_t pol = c.count <= tw ? l2_policy_evict_first() : l2_policy_evict_normal();
      const int row_a0 = c.e * args.rows_per_expert + c.w * kBlock + static_cast<int>(rank) * kBM;
      const int row_a1 = kMode == kUp ? row_a0 : row_a0 + 2 * kBM;
      const int half = c.N / 2, nbox = (half + kBRows - 1) / kBRows;
      for (int k = warp; k < ahead; k += kProducers) {
        if (leader && lane == 0)
          mbar_arrive_expect_tx(&full[k], 2u * (C::kABytes + (kGather ? half : nbox * kBRows) * kBK));
        __syncwarp();
        if (lane < kBoxes)
          tma_load_2d_pair(kMode == kUp && lane == 1 ? &tm_a1 : &tm_a0, cluster_addr(&full[k], 0),
                           ring + k * C::kStage + lane * kBoxBytes, k * kBK, lane == 0 ? row_a0 : row_a1, pol);
      }
    }
    grid_dependency_wait();
    for (int tile = pair; tile < total && alive; tile += npairs, it0 += nk) {
      const Tile c = tile_at(tile);
      const uint64_t pol = c.count <= tw ? l2_policy_evict_first() : l2_policy_evict_normal();
      const int row_a0 = c.e * args.rows_per_expert + c.w * kBlock + static_cast<int>(rank) * kBM;
      const int row_a1 = kMode == kUp ? row_a0 : row_a0 + 2 * kBM;
      const int half = c.N / 2;
      const int row0 = c.row0 + static_cast<int>(rank) * half;
      const int nbox = (half + kBRows - 1) / kBRows;
      // gathered: lane i copies rows 4 i .. 4 i + 3 of this CTA's half (rows past the tile's last take token 0;
      // their columns are never stored)
      int tok[4] = {0, 0, 0, 0};
      if (kGather) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = 4 * lane + u;
          if (r < half && static_cast<int>(rank) * half + r < c.nrows) {
            const int id = plan_slot(args, row0 + r);
            tok[u] = id >= 0 ? id / args.top_k : 0;
          }
        }
      }
      const uint32_t bytes = 2u * (C::kABytes + (kGather ? half : nbox * kBRows) * kBK);  // of both CTAs
      for (int k = (warp + kProducers - it0 % kProducers) % kProducers; k < nk; k += kProducers) {
        const int it = it0 + k, s = it % kStages;
        const bool boxes = it >= ahead;  // else they are on their way
        bool ok = true;
        if (boxes && lane == 0) {
          ok = mbar_wait_bounded(&empty[s], ((it / kStages) & 1) ^ 1, abort_flag);
          if (ok && leader) mbar_arrive_expect_tx(&full[s], bytes);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          if (lane == 0) {
            *abort_flag = 1;
            set_error(args.err, kErrTimeout);
          }
          alive = false;
          break;
        }
        uint8_t* st = ring + s * C::kStage;
        const uint32_t bar = cluster_addr(&full[s], 0);
        if (boxes && lane < kBoxes)
          tma_load_2d_pair(kMode == kUp && lane == 1 ? &tm_a1 : &tm_a0, bar, st + lane * kBoxBytes, k * kBK,
                           lane == 0 ? row_a0 : row_a1, pol);
        if (kGather) {
          if (4 * lane < half)
            tma_gather4_pair(&tm_b, bar, st + C::kABytes + lane * 4 * kBK, k * kBK, tok[0], tok[1], tok[2], tok[3],
                             pol_b);
        } else if (lane < nbox) {
          tma_load_2d_pair(&tm_b, bar, st + C::kABytes + lane * kBRows * kBK, k * kBK, row0 + lane * kBRows, pol_b);
        }
      }
    }
    // After an abort nobody waits for the copies under way, and the leader's barriers count both CTAs' copies, of which
    // the other may have issued fewer.  So they get time to land: a ring of 192 KB needs some microseconds.
    if ((!alive || *abort_flag) && lane == 0)
      for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < kDrainNs;) {
      }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------ MMA issuer (leader only)
    if (leader && lane == 0) {
      int it = 0, j = 0, committed = 0;  // tiles
      bool alive = true;
      for (int tile = pair; tile < total && alive; tile += npairs, ++j) {
        const uint32_t idesc = umma_idesc_s8(2 * kBM, tile_at(tile).N);
        const int buf = j % C::kAccBufs;
        if (!mbar_wait_bounded(&acc_empty[buf], ((j / C::kAccBufs) & 1) ^ 1, abort_flag)) {
          *abort_flag = 1;
          set_error(args.err, kErrTimeout);
          break;
        }
        tc_fence_after_sync();
        const uint32_t d0 = tmem + buf * C::kAccCols;
        const uint32_t d1 = d0 + kNmax;
        for (int k = 0; k < nk; ++k, ++it) {
          const int s = it % kStages;
          if (!mbar_wait_bounded(&full[s], (it / kStages) & 1, abort_flag)) {
            *abort_flag = 1;
            set_error(args.err, kErrTimeout);
            alive = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t da0 = umma_desc_sw128(ring + s * C::kStage);
          const uint64_t da1 = umma_desc_sw128(ring + s * C::kStage + kBoxBytes);
          const uint64_t db = umma_desc_sw128(ring + s * C::kStage + C::kABytes);
#pragma unroll
          for (int kk = 0; kk < kBK / 32; ++kk) {
            const uint32_t acc = (k | kk) != 0 ? 1u : 0u;
            umma_s8_pair(d0, da0 + 2 * kk, db + 2 * kk, idesc, acc);
            if (kBoxes == 2) umma_s8_pair(d1, da1 + 2 * kk, db + 2 * kk, idesc, acc);
          }
          umma_commit_pair(&empty[s]);
        }
        umma_commit_pair(&acc_full[buf]);  // also on an abort, so neither epilogue is left waiting
        committed = j + 1;
      }
      // after an abort nobody else waits for the products under way, which still read both rings
      if (*abort_flag && committed > 0)
        mbar_wait_bounded(&acc_full[(committed - 1) % C::kAccBufs], ((committed - 1) / C::kAccBufs) & 1, nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue (both CTAs: their own 2 x 128 channels)
    grid_dependency_wait();
    const int q = warp & 3;
    const int part_c = (warp - kFirstEpi) >> 2;  // which of the four 16-column chunks of every 64 this warp drains
    constexpr int kChunks = kNmax / 64;
    const int g8 = lane >> 3, b8 = lane & 7;
    int j = 0;
    for (int tile = pair; tile < total; tile += npairs, ++j) {
      const Tile c = tile_at(tile);
      const int buf = j % C::kAccBufs;
      const int colbase = c.w * kBlock + static_cast<int>(rank) * kBM + q * 32;  // this warp's first channel
      // what the scaling needs, loaded while the tile is still being computed: the lane's channel scales, and in
      // lane i < 16 the scale and output row of the chunk's token i
      const int ch0 = colbase + lane, ch1 = kMode == kUp ? ch0 : ch0 + 2 * kBM;  // one box: there is no ch1
      const size_t ch_at = static_cast<size_t>(c.e) * args.rows_per_expert;
      const float s0 = ch0 < args.rows_per_expert ? args.ch_scale0[ch_at + ch0] : 0.0f;
      const float s1 = kBoxes == 2 && ch1 < args.rows_per_expert ? (kMode == kUp ? args.ch_scale1 : args.ch_scale0)[ch_at + ch1] : 0.0f;
      float tok_s[kChunks];
      int tok_row[kChunks];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) token_at(c, 16 * part_c + 64 * i + (lane & 15), tok_s[i], tok_row[i]);
      // no scale of the warp's is near the ends of fp32's range: then their products need no look at each
      bool near = int8_near_scale(s0) && int8_near_scale(s1);
#pragma unroll
      for (int i = 0; i < kChunks; ++i) near = near && int8_near_scale(tok_s[i]);
      near = __all_sync(0xffffffffu, near);
      bool ok = true;
      if (lane == 0) ok = mbar_wait_bounded(&acc_full[buf], (j / C::kAccBufs) & 1, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      tc_fence_after_sync();
      const bool go = __shfl_sync(0xffffffffu, ok && !*abort_flag, 0);
      if (!go) {
        if (lane == 0 && !ok) set_error(args.err, kErrTimeout);
        break;
      }
      const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * C::kAccCols;
      if (!near) {
        // rare, so small rather than fast: lane = channel, element stores, the tokens looked up again
#pragma unroll 1
        for (int i = 0; i < kChunks; ++i) {
          const int cb = 16 * part_c + 64 * i;
          if (cb >= c.N) break;
          __syncwarp();
          uint32_t v0[16], v1[16];
          tmem_load_16(lane_base + cb, v0);
          if (kBoxes == 2) tmem_load_16(lane_base + kNmax + cb, v1);
          tmem_load_wait();
          float sc;
          int to;
          token_at(c, cb + (lane & 15), sc, to);
#pragma unroll
          for (int p = 0; p < 16; ++p) {
            const float sx = __shfl_sync(0xffffffffu, sc, p);
            const int row = __shfl_sync(0xffffffffu, to, p);
            if (row < 0) continue;
            float r0 = int8_value(sx, s0, static_cast<int>(v0[p]));
            const float r1 = kBoxes == 2 ? int8_value(sx, s1, static_cast<int>(v1[p])) : 0.0f;
            if (kMode == kUp) r0 = silu_mul(r0, r1);
            const size_t at = static_cast<size_t>(row) * args.out_ld;
            auto put = [&](int ch, float r) {
              if (ch >= args.rows_per_expert) return;
              if (kMode == kDense && args.out_f32)
                static_cast<float*>(args.out)[at + ch] = r;
              else
                static_cast<__nv_bfloat16*>(args.out)[at + ch] = __float2bfloat16_rn(r);
            };
            put(ch0, r0);
            if (kMode != kUp && kBoxes == 2) put(ch1, r1);
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_addr(&acc_empty[buf], 0));
        continue;
      }
      if (kMode == kDense && args.out_plain) {
        // fp32 results, or rows that take no 16-byte stores: lane = channel, one store per token and half
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int cb = 16 * part_c + 64 * i;
          if (cb >= c.N) break;
#pragma unroll
          for (int half = 0; half < kBoxes; ++half) {
            uint32_t v[16];
            tmem_load_16(lane_base + half * kNmax + cb, v);
            tmem_load_wait();
            const int ch = half ? ch1 : ch0;
            const float sc = half ? s1 : s0;
#pragma unroll
            for (int p = 0; p < 16; ++p) {
              const int row = __shfl_sync(0xffffffffu, tok_row[i], p);
              const float r = (__shfl_sync(0xffffffffu, tok_s[i], p) * sc) * static_cast<float>(static_cast<int>(v[p]));
              if (row < 0 || ch >= args.rows_per_expert) continue;
              const size_t at = static_cast<size_t>(row) * args.out_ld + ch;
              if (args.out_f32)
                static_cast<float*>(args.out)[at] = r;
              else
                static_cast<__nv_bfloat16*>(args.out)[at] = __float2bfloat16_rn(r);
            }
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_addr(&acc_empty[buf], 0));
        continue;
      }
      // 1. drain: lane l holds channel ch0 (ch1) for the tokens of its chunks; scaled and packed as bf16 token
      //    pairs, then the accumulator is released at once, so the next tile's MMAs run while this one is stored
      constexpr int kOuts = kMode == kUp ? 1 : kBoxes;  // output halves
      constexpr int kWords = 8 * kOuts;
      uint32_t pk[kChunks][kWords];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int cb = 16 * part_c + 64 * i;
        if (cb >= c.N) break;
        uint32_t v0[16], v1[16];
        tmem_load_16(lane_base + cb, v0);
        if (kBoxes == 2) tmem_load_16(lane_base + kNmax + cb, v1);
        tmem_load_wait();
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          float a[2], b[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float sx = __shfl_sync(0xffffffffu, tok_s[i], 2 * p + u);
            a[u] = (sx * s0) * static_cast<float>(static_cast<int>(v0[2 * p + u]));
            b[u] = kBoxes == 2 ? (sx * s1) * static_cast<float>(static_cast<int>(v1[2 * p + u])) : 0.0f;
          }
          if (kMode == kUp) {
            pk[i][p] = pack_bf16x2(silu_mul(a[0], b[0]), silu_mul(a[1], b[1]));
          } else {
            pk[i][p] = pack_bf16x2(a[0], a[1]);
            if (kBoxes == 2) pk[i][kWords - 8 + p] = pack_bf16x2(b[0], b[1]);
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&acc_empty[buf], 0));
      // 2. store: the 8 x 8 transpose in each group of 8 lanes gives lane 8 g + b tokens 2 b and 2 b + 1 of the
      //    chunk at channels colbase + 8 g .. + 7: 16-byte row stores
      const int col8 = colbase + 8 * g8;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int cb = 16 * part_c + 64 * i;
        if (cb >= c.N) break;
        const int d0 = __shfl_sync(0xffffffffu, tok_row[i], 2 * b8);
        const int d1 = __shfl_sync(0xffffffffu, tok_row[i], 2 * b8 + 1);
#pragma unroll
        for (int half = 0; half < kOuts; ++half) {
          uint32_t w[8];
#pragma unroll
          for (int p = 0; p < 8; ++p) w[p] = pk[i][8 * half + p];
          transpose8x8(w, b8);
          const uint4 r0 = make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410),
                                      __byte_perm(w[4], w[5], 0x5410), __byte_perm(w[6], w[7], 0x5410));
          const uint4 r1 = make_uint4(__byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632),
                                      __byte_perm(w[4], w[5], 0x7632), __byte_perm(w[6], w[7], 0x7632));
          const int cc = col8 + half * 2 * kBM;
          if (cc >= args.rows_per_expert) continue;  // a multiple of 8 here
          uint16_t* out = static_cast<uint16_t*>(args.out);
          if (d0 >= 0) *reinterpret_cast<uint4*>(out + static_cast<size_t>(d0) * args.out_ld + cc) = r0;
          if (d1 >= 0) *reinterpret_cast<uint4*>(out + static_cast<size_t>(d1) * args.out_ld + cc) = r1;
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the other may still use its shared or tensor memory
  if (warp == kMmaWarp) tmem_dealloc_pair(tmem, 512);
}

template <int kMode, int kNmax, int kStages, int kBoxes = 2>
cudaError_t launch_pairs(const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b, const Int8GemmArgs& args,
                         int num_sms, cudaStream_t stream) {
  using C = PCfg<kNmax, kStages, kBoxes>;
  auto kern = int8_pair_kernel<kMode, kNmax, kStages, kBoxes>;
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
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms & ~1));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a0, a1, b, args);
}

}  // namespace

cudaError_t launch_int8_pair_up(const CUtensorMap& w_gate, const CUtensorMap& w_up, const CUtensorMap& x_rows,
                                const Int8GemmArgs& args, int nmax, int num_sms, cudaStream_t stream) {
  if (nmax >= 256) return launch_pairs<kUp, 256, 4>(w_gate, w_up, x_rows, args, num_sms, stream);
  return launch_pairs<kUp, 128, 5>(w_gate, w_up, x_rows, args, num_sms, stream);
}

cudaError_t launch_int8_pair_down(const CUtensorMap& w_down, const CUtensorMap& h_rows, const Int8GemmArgs& args,
                                  int nmax, int num_sms, cudaStream_t stream) {
  if (nmax >= 256) return launch_pairs<kDown, 256, 4>(w_down, w_down, h_rows, args, num_sms, stream);
  return launch_pairs<kDown, 128, 5>(w_down, w_down, h_rows, args, num_sms, stream);
}

cudaError_t launch_int8_pair_dense(const CUtensorMap& w, const CUtensorMap& x_rows, const Int8GemmArgs& args,
                                   int num_sms, cudaStream_t stream) {
  if (args.tile_n < 32 || args.tile_n > 256 || args.tile_n % 32 != 0) return cudaErrorInvalidValue;
  if (args.tile_boxes == 1) return launch_pairs<kDense, 256, 6, 1>(w, w, x_rows, args, num_sms, stream);
  return launch_pairs<kDense, 256, 4>(w, w, x_rows, args, num_sms, stream);
}

}  // namespace moe
