// Routing from given logits with expert groups (moe_route_logits): scores, a bias that shifts the selection
// only, the best groups, the best experts of those groups, weights.
//
//   p_e   = 1 / (1 + e^-z_e), or e^(z_e - max) / sum_j e^(z_j - max)
//   key_e = p_e + bias_e
//   s_g   = the largest key of group g, or the sum of its two largest
//   the topk_group groups with the largest s_g stay; of their experts the top_k with the largest keys, ties to
//   the lower id;  w_k = p_k, or p_k / sum_j p_j, times routed_scale.
//
// The choice is a comparison of rounded numbers, so it is defined in fp64: p, keys and group scores.  fp64 arithmetic
// is slow (a token of 256 experts: 20 us alone, and 168 us for 32767 tokens), so a token is first routed in fp32 with
// a bound on what fp32 may be off by, and only where two candidates next to each other are nearer than that (or a
// number is not finite, or far out) its warp computes it again in fp64.  The result is the fp64 one either way.
//
// fp32 path, one warp per token:
//  1. logits in (coalesced, each read once), keys to shared memory.  Without a bias the key is the logit itself (the
//     scores grow with it), so equal keys are equal logits and no bound is needed between different ones.
//  2. group scores: 32 / n_group lanes (a power of two) scan each group's keys for the two largest.
//  3. the kept groups' keys into registers, as integers that order like the numbers; top_k + 1 rounds of a warp
//     maximum (redux) and the lowest id that has it.  The round past the last one shows the gap behind the choice.
//  4. weights from the K logits.
// Errors (ex2.approx and rcp are within 2 ulp; the scaled argument of the exponential adds |z| 2^-23.4 relative):
//   sigmoid: |p32 - p| <= p (1 - p) (|z| 2^-23.4 + 2^-21.5) + p 2^-21 < 2^-20
//   softmax: relative 2^-19 + |z - max| 2^-23, and p <= e^-|z - max| / denom: below 2^-18 / denom
// plus 2^-24 of each sum that follows.  Two keys further apart than both errors are in the right order.
// Bound: issue slots (about 400 instructions per token of 256 experts), not memory.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kWarps = 4;  // one token per warp

__device__ __forceinline__ double shfl_xor_d(double v, int off) { return __shfl_xor_sync(0xffffffffu, v, off); }

// NaN ranks below every number.
__device__ __forceinline__ double rank_key(double v) { return isnan(v) ? -INFINITY : v; }

template <bool kBf16>
__device__ __forceinline__ float raw_logit(const void* row, int e) {
  if (kBf16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(row)[e]) << 16);
  return static_cast<const float*>(row)[e];
}

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* row, int e) {
  const float z = raw_logit<kBf16>(row, e);
  return isnan(z) ? -INFINITY : z;
}

// The hardware's base-2 exponential and reciprocal, results below 2^-126 flushed to 0 (within the bound of 2^-20).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// e^(z - zmax) with the limits: a row whose largest logit is +inf shares among its +inf entries, a row of
// -inf only has no scores.
__device__ __forceinline__ double exp_score(double z, double zmax) {
  if (zmax == -INFINITY) return 0.0;
  if (zmax == INFINITY) return z == INFINITY ? 1.0 : 0.0;
  return exp(z - zmax);
}

// One token in fp64, whatever its logits hold: the definition, and the answer for the tokens that the fp32 path
// leaves.  One warp; `key`: E doubles of shared memory.
template <bool kBf16>
__device__ __noinline__ void route_token_fp64(const void* row, const float* bias, int E, int K,
                                              const RouteGroupOpts& o, double* key, int32_t* ids, float* w) {
  const int lane = threadIdx.x & 31;
  __syncwarp();

  double zmax = -INFINITY, denom = 1.0;
  if (o.scoring == MOE_SCORE_SOFTMAX) {
    for (int e = lane; e < E; e += 32) zmax = fmax(zmax, static_cast<double>(load_logit<kBf16>(row, e)));
    for (int off = 16; off >= 1; off >>= 1) zmax = fmax(zmax, shfl_xor_d(zmax, off));
    denom = 0.0;
    for (int e = lane; e < E; e += 32) denom += exp_score(load_logit<kBf16>(row, e), zmax);
    for (int off = 16; off >= 1; off >>= 1) denom += shfl_xor_d(denom, off);
  }
  auto score = [&](int e) {
    const double z = load_logit<kBf16>(row, e);
    if (o.scoring == MOE_SCORE_SOFTMAX) return denom > 0.0 ? exp_score(z, zmax) / denom : 0.0;
    return 1.0 / (1.0 + exp(-z));
  };
  for (int e = lane; e < E; e += 32)
    key[e] = rank_key(bias != nullptr ? score(e) + static_cast<double>(bias[e]) : score(e));
  __syncwarp();

  // groups: lane g keeps the score of group g and whether it stays
  const int gs = E / o.n_group;
  unsigned kept = 0xffffffffu;
  if (o.topk_group < o.n_group) {
    double mine = -INFINITY;
    for (int g = 0; g < o.n_group; ++g) {
      double a = -INFINITY, b = -INFINITY;  // two largest keys
      for (int i = lane; i < gs; i += 32) {
        const double v = key[g * gs + i];
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
      }
      for (int off = 16; off >= 1; off >>= 1) {
        const double oa = shfl_xor_d(a, off), ob = shfl_xor_d(b, off);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
      }
      if (lane == g) mine = (o.group_score == MOE_GROUP_TOP2 && gs > 1) ? rank_key(a + b) : a;
    }
    int before = 0;
    for (int g = 0; g < o.n_group; ++g) {
      const double v = __shfl_sync(0xffffffffu, mine, g);
      before += v > mine || (v == mine && g < lane);
    }
    kept = __ballot_sync(0xffffffffu, lane < o.n_group && before < o.topk_group);
  }
  uint32_t live = 0;  // bit i: expert lane + 32 i may be chosen
  for (int e = lane, i = 0; e < E; e += 32, ++i)
    if ((kept >> (e / gs)) & 1u) live |= 1u << i;

  int sel = 0;
  for (int k = 0; k < K; ++k) {
    double bv = -INFINITY;
    int bi = 0x7fffffff;
    for (int e = lane, i = 0; e < E; e += 32, ++i)
      if (((live >> i) & 1u) && (bi == 0x7fffffff || key[e] > bv)) {
        bv = key[e];
        bi = e;
      }
    for (int off = 16; off >= 1; off >>= 1) {
      const double ov = shfl_xor_d(bv, off);
      const int oi = __shfl_xor_sync(0xffffffffu, bi, off);
      if (ov > bv || (ov == bv && oi < bi)) {
        bv = ov;
        bi = oi;
      }
    }
    if ((bi & 31) == lane) live &= ~(1u << (bi >> 5));
    if (lane == k) sel = bi;
  }
  double p = lane < K ? score(sel) : 0.0;
  double total = p;
  for (int off = 16; off >= 1; off >>= 1) total += shfl_xor_d(total, off);
  if (o.renormalize) p = total > 0.0 ? p / total : 0.0;
  if (lane < K) {
    ids[lane] = sel;
    w[lane] = static_cast<float>(p * static_cast<double>(o.routed_scale));
  }
}

// Integers that order like the numbers; 0 is below every finite one.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 -> +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_order_bits(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

// kPer: candidates per lane, the kept groups' experts / 32 rounded up to a power of two.
template <bool kBf16, int kPer>
__global__ void __launch_bounds__(32 * kWarps) route_group_kernel(const void* __restrict__ logits, int64_t ld,
                                                                  const float* __restrict__ bias, int M, int E, int K,
                                                                  RouteGroupOpts o, int32_t* __restrict__ topk_ids,
                                                                  float* __restrict__ topk_w) {
  extern __shared__ double keys_smem[];
  __shared__ uint8_t kept_groups[kWarps][32];  // the groups that stay, in order
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= M) return;
  float* zs = reinterpret_cast<float*>(keys_smem + warp * E);  // logits [E]
  float* key = zs + E;                                         // keys [E]
  const uint8_t* row = static_cast<const uint8_t*>(logits) + static_cast<size_t>(t) * ld * (kBf16 ? 2 : 4);
  int32_t* ids = topk_ids + static_cast<size_t>(t) * K;
  float* w = topk_w + static_cast<size_t>(t) * K;
  const bool softmax = o.scoring == MOE_SCORE_SOFTMAX;
  const bool groups = o.topk_group < o.n_group;
  const bool by_logit = bias == nullptr;
  const bool group_sums = groups && o.group_score == MOE_GROUP_TOP2 && E > o.n_group;

  // ---- 1. logits and keys
  uint32_t zbits = 0;  // largest |z| as bits: from 0x7f800000 on a logit is not finite
  float zmax = -INFINITY;
  for (int e0 = lane; e0 < E; e0 += 256) {  // eight loads in flight
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = e0 + 32 * i < E ? raw_logit<kBf16>(row, e0 + 32 * i) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (e0 + 32 * i >= E) break;
      zs[e0 + 32 * i] = z[i];
      zbits = max(zbits, __float_as_uint(z[i]) & 0x7fffffffu);
      zmax = fmaxf(zmax, z[i]);
    }
  }
  uint32_t kbits = 0;
  if (softmax) zmax = from_order_bits(__reduce_max_sync(0xffffffffu, order_bits(zmax)));
  float denom = 1.0f;
  if (softmax && !(by_logit && !group_sums && o.renormalize)) {
    denom = 0.0f;
    for (int e = lane; e < E; e += 32) denom += expf(zs[e] - zmax);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) denom += __shfl_xor_sync(0xffffffffu, denom, off);
  }
  const float inv_denom = 1.0f / denom;
  auto score32 = [&](float z) {
    constexpr float kLog2e = 1.4426950408889634f;
    return softmax ? exp2_approx((z - zmax) * kLog2e) * inv_denom : rcp_approx(1.0f + exp2_approx(-z * kLog2e));
  };
  if (by_logit && !group_sums) {
    key = zs;
  } else {
#pragma unroll 4
    for (int e = lane; e < E; e += 32) {
      const float v = by_logit ? score32(zs[e]) : score32(zs[e]) + bias[e];
      key[e] = v;
      kbits = max(kbits, __float_as_uint(v) & 0x7fffffffu);
    }
    kbits = __reduce_max_sync(0xffffffffu, kbits);
  }
  // what a key that holds a score may be off by
  const float off_key = (softmax ? 0x1p-18f * inv_denom : 0x1p-20f) + __uint_as_float(kbits) * 0x1p-23f;
  bool fine = __reduce_max_sync(0xffffffffu, zbits) < 0x7f800000u && kbits < 0x7f800000u;
  __syncwarp();

  // Two logits give scores that fp64 tells apart, in their order: they differ by more than 2^-30, and neither score
  // is so near to 1 or to 0 that the difference is lost there.
  auto logits_apart = [&](float hi, float lo) {
    if (hi == lo) return true;  // the same score: the lower id, as found
    if (!(hi - lo > 0x1p-30f)) return false;
    return softmax ? lo - zmax > -600.0f : (hi < 12.0f && lo > -600.0f);
  };

  // ---- 2. groups
  const int gs = E / o.n_group;
  if (groups && fine) {
    const int per_group = 1 << (31 - __clz(32 / o.n_group));  // lanes
    const int g = lane / per_group, sub = lane % per_group;
    float a = -INFINITY, b = -INFINITY;
    if (g < o.n_group) {
      const int turn = (g * per_group) % gs;  // each group starts elsewhere, so that the lanes read different banks
#pragma unroll 4
      for (int i = sub; i < gs; i += per_group) {
        const float v = key[g * gs + (i + turn < gs ? i + turn : i + turn - gs)];
        b = fmaxf(b, fminf(a, v));
        a = fmaxf(a, v);
      }
    }
    for (int off = per_group >> 1; off >= 1; off >>= 1) {
      const float oa = __shfl_xor_sync(0xffffffffu, a, off), ob = __shfl_xor_sync(0xffffffffu, b, off);
      b = fmaxf(fminf(a, oa), fmaxf(b, ob));
      a = fmaxf(a, oa);
    }
    // lane q: group q's score and its place among them
    float s = group_sums ? a + b : a;
    s = __shfl_sync(0xffffffffu, s, (lane * per_group) & 31);
    int before = 0;
    for (int q = 0; q < o.n_group; ++q) {
      const float v = __shfl_sync(0xffffffffu, s, q);
      before += v > s || (v == s && q < lane);
    }
    const bool mine = lane < o.n_group;
    const bool stays = mine && before < o.topk_group;
    const unsigned kept = __ballot_sync(0xffffffffu, stays);
    if (stays) kept_groups[warp][__popc(kept & ((1u << lane) - 1u))] = static_cast<uint8_t>(lane);
    __syncwarp();
    // the last group that stays against the first that does not
    const int last = __ffs(__ballot_sync(0xffffffffu, mine && before == o.topk_group - 1)) - 1;
    const int next = __ffs(__ballot_sync(0xffffffffu, mine && before == o.topk_group)) - 1;
    const float hi = __shfl_sync(0xffffffffu, s, last), lo = __shfl_sync(0xffffffffu, s, next);
    if (by_logit && !group_sums)
      fine = logits_apart(hi, lo);
    else
      fine = hi - lo > (group_sums ? 4.0f : 2.0f) * off_key + fabsf(hi) * 0x1p-22f;
  }

  // ---- 3. experts
  int sel = 0;
  float zsel = 0.0f;
  if (fine) {
    const float* order = by_logit ? zs : key;
    const int ncand = o.topk_group * gs;
    const float inv_gs = 1.0f / static_cast<float>(gs);
    uint32_t u[kPer];
    int id[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = lane + 32 * i;
      u[i] = 0;
      id[i] = 0x7fffffff;
      if (c < ncand) {
        int e = c;
        if (groups) {
          // c / gs: (c + 1/2) / gs is at least 1/2048 from a whole number, the product off by 2^-13 at most
          const int q = static_cast<int>((static_cast<float>(c) + 0.5f) * inv_gs);
          e = kept_groups[warp][q] * gs + (c - q * gs);
        }
        id[i] = e;
        u[i] = order_bits(order[e]);
      }
    }
    if (kPer <= 4) {
      // each lane's candidates in descending order (neighbours change places only if the later one is larger, so
      // equal ones keep the lower id first): a round takes a lane's first and moves the others up
#pragma unroll
      for (int i = 1; i < kPer; ++i)
#pragma unroll
        for (int l = i; l >= 1; --l) {
          const bool swap = u[l] > u[l - 1];
          const uint32_t hi_u = swap ? u[l] : u[l - 1], lo_u = swap ? u[l - 1] : u[l];
          const int hi_id = swap ? id[l] : id[l - 1], lo_id = swap ? id[l - 1] : id[l];
          u[l - 1] = hi_u;
          u[l] = lo_u;
          id[l - 1] = hi_id;
          id[l] = lo_id;
        }
    }
    uint32_t mine = 0, top = 0;  // the key of round `lane`; of the last round
    const int rounds = min(K + 1, ncand);
    for (int k = 0; k < rounds; ++k) {
      uint32_t best = u[0];
      int bid = id[0];
      if (kPer > 4) {
#pragma unroll
        for (int i = 1; i < kPer; ++i)
          if (u[i] > best) {  // ids grow with i: the first of equal ones stays
            best = u[i];
            bid = id[i];
          }
      }
      top = __reduce_max_sync(0xffffffffu, best);
      const int win = static_cast<int>(__reduce_min_sync(0xffffffffu, best == top ? bid : 0x7fffffff));
      if (kPer > 4) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (id[i] == win) u[i] = 0;
      } else if (bid == win) {
#pragma unroll
        for (int i = 1; i < kPer; ++i) {
          u[i - 1] = u[i];
          id[i - 1] = id[i];
        }
        u[kPer - 1] = 0;
        id[kPer - 1] = 0x7fffffff;
      }
      if (lane == k) {
        mine = top;
        sel = win;
      }
    }
    // every choice against the next one: lane k compares rounds k and k + 1 (round 32 is in no lane)
    const uint32_t after = __shfl_down_sync(0xffffffffu, mine, 1);
    const int after_id = __shfl_down_sync(0xffffffffu, sel, 1);
    bool good = true;
    if (lane + 1 < rounds) {
      const float hi = from_order_bits(mine), lo = from_order_bits(lane < 31 ? after : top);
      if (by_logit)
        good = logits_apart(hi, lo);
      else
        good = hi - lo > 2.0f * off_key ||
               (lane < 31 && hi == lo && zs[sel] == zs[after_id] && bias[sel] == bias[after_id]);
    }
    if (lane < K) {
      zsel = zs[sel];
      // scores far below the fp32 range are the fp64 path's
      good = good && !((softmax ? zsel - zmax : zsel) < -80.0f);
    }
    fine = __all_sync(0xffffffffu, good);
  }
  if (!fine) {
    route_token_fp64<kBf16>(row, bias, E, K, o, reinterpret_cast<double*>(zs), ids, w);
    return;
  }

  // ---- 4. weights
  float p = 0.0f;
  if (lane < K) p = softmax ? expf(zsel - zmax) : __fdiv_rn(1.0f, 1.0f + expf(-zsel));
  float total = p;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  if (lane < K) {
    ids[lane] = sel;
    w[lane] = __fdiv_rn(p, o.renormalize ? total : denom) * o.routed_scale;
  }
}

template <bool kBf16>
cudaError_t launch_typed(const void* logits, int64_t ld, const float* bias, int M, int E, int K,
                         const RouteGroupOpts& o, int32_t* topk_ids, float* topk_w, cudaStream_t stream) {
  const dim3 grid((M + kWarps - 1) / kWarps);
  const size_t smem = sizeof(double) * kWarps * E;  // at most 32 KB
  const int per = (o.topk_group * (E / o.n_group) + 31) / 32;
  auto run = [&](auto kern) { kern<<<grid, 32 * kWarps, smem, stream>>>(logits, ld, bias, M, E, K, o, topk_ids, topk_w); };
  if (per <= 1)
    run(route_group_kernel<kBf16, 1>);
  else if (per <= 2)
    run(route_group_kernel<kBf16, 2>);
  else if (per <= 4)
    run(route_group_kernel<kBf16, 4>);
  else if (per <= 8)
    run(route_group_kernel<kBf16, 8>);
  else if (per <= 16)
    run(route_group_kernel<kBf16, 16>);
  else
    run(route_group_kernel<kBf16, 32>);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route_group(const void* logits, bool bf16, int64_t ld, const float* bias, int M, int E, int K,
                               const RouteGroupOpts& o, int32_t* topk_ids, float* topk_w, cudaStream_t stream) {
  return bf16 ? launch_typed<true>(logits, ld, bias, M, E, K, o, topk_ids, topk_w, stream)
              : launch_typed<false>(logits, ld, bias, M, E, K, o, topk_ids, topk_w, stream);
}

}  // namespace moe
