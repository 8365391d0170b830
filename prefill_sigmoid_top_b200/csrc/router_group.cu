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
// number is NaN, +inf or far out) its warp computes it again in fp64.  The result is the fp64 one either way.
//
// fp32 path, one warp per token, no shared memory.  What bounds it is the ALU pipe (compare, select, minimum and
// integer logic issue at half rate), so keys are shaped with multiply-adds and compared as few times as can be:
//  1. 32 / n_group lanes (a power of two) hold a group, each up to kPer neighbouring experts in registers (16-byte
//     loads where rows allow).  Without a bias the key is the logit itself (the scores grow with it).
//  2. a key becomes an integer, its place between kmax - range and kmax in 2^23 (2^22) steps, with the inverted expert
//     id below: two multiply-adds and one integer multiply-add.  All are different; larger key first, lower id first.
//     A lane sorts its own in lists of 8 (Batcher's network: one minimum and one maximum per exchange).
//  3. group scores from the two first integers of each lane, joined over the group's lanes by shuffles; the groups that
//     stay by one warp maximum each.
//  4. top_k + 1 rounds of ONE warp maximum (redux) over the lists' first integers; the owner moves its list up.  The
//     round past the last shows the gap behind the choice.
//  5. weights from the K logits, in fp64.
// Two keys are in the right order where their integers are 3 or more apart (one is off by less than a step) and that
// distance exceeds what the keys may be off by:
//   sigmoid: |p32 - p| <= p (1 - p) (|z| 2^-23.4 + 2^-22) + p (2^-24 + 2^-23) < 1.5 * 2^-22 (ex2.approx is within 2^-22,
//            rcp.approx within 2^-23; the scaled argument of the exponential adds |z| 2^-23.4 relative)
//   softmax: relative 2^-19 + |z - max| 2^-23, and p <= e^-|z - max| / denom: below 2^-18 / denom
//            (exponentials 2^-22, their sum 11 roundings, reciprocal and product 2^-22: less than 2^-19)
// plus 2^-23 of each sum that follows.  Of bf16 logits, two that are nearer than their spacing are equal: a tie.
// Weights: exponentials of the K chosen logits, their sum and the quotients in fp64 (a few instructions each: far fewer
// bits are needed than exp() and a division give), rounded to fp32 once: within 2^-24 (1 + 2^-5).  A softmax that is not
// renormalised has a denominator over all experts, whose exponentials in fp64 would cost more than the choice: they are
// expf (within 4 units of 2^-24), times a factor for the rounding of z - max (1), summed in fp32 in a lane (up to 6
// levels) and in fp64 over the lanes: with the last rounding within 12 units, 2^-20.  Weights in fp32 throughout were
// off by up to 28 units (measured: 1.2) and took 21.6 us instead of 23.4 for 32767 tokens.
// Keys below the range, -inf among them, share the lowest integer: where one counts in the sum of a group that stays,
// the token is fp64's.  About 1 token in 1000 of normal logits and a small bias has two
// neighbours too near (2 in 100 with 1024 experts and K = 32).  Where that is all, the K + 1 listed keys are computed
// exactly, one per lane, and put in order; the rest goes to the fp64 path as a whole, whose 10 to 40 us for one token
// would otherwise be the tail of every large call.
//
// Measured (256 experts in 8 groups, 4 kept, K = 8, sigmoid and bias, fp32): 8 tokens 2.5 us, 32767 tokens 23.4 us
// (1.5 TB/s; 630 instructions per token, 53 of them for the weights in fp64, 81% of the issue slots in use; more warps
// per SM change nothing); 2048 tokens of bf16 logits, softmax, K = 16: 4.3 us; a part of the experts masked by -inf
// changes nothing (softmax: 32 -> 40 us).  Tried and slower, before the weights were in fp64 (21.6 us): persistent warps that
// fetch their next token ahead (35 us), keys and ids in shared memory with two warp reductions per choice (50 us).
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

// The hardware's base-2 exponential and reciprocal, results below 2^-126 flushed to 0 (within the bounds above).
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

// e^x for x in [-100, 81], within 2^-31 (relative): x = k ln 2 + r with |r| <= ln 2 / 2, then Taylor's series to r^8 (the
// next term is below 2^-32).  k leaves the sum with 1.5 * 2^52 as its low word.
__device__ __forceinline__ double exp_reduced(double x) {
  constexpr double kRound = 6755399441055744.0;
  const double t = fma(x, 1.4426950408889634, kRound);
  const double r = fma(kRound - t, 0.6931471805599453, x);
  double p = 1.0 / 40320.0;
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return __hiloint2double(__double2hiint(p) + (__double2loint(t) << 20), __double2loint(p));
}
// 1 / d for a d in fp32's normal range, within 2^-44: one step of Newton's method from the fp32 reciprocal.
__device__ __forceinline__ double reciprocal(double d) {
  const double y = static_cast<double>(rcp_approx(static_cast<float>(d)));
  return fma(y, fma(-d, y, 1.0), y);
}

// e^(z - zmax) at the limits: a row whose largest logit is +inf shares among its +inf entries, a row of -inf only has
// no scores.
__device__ __forceinline__ double exp_limits(double z, double zmax) {
  return zmax == INFINITY && z == INFINITY ? 1.0 : 0.0;
}

// The score of one logit (softmax: from the row's maximum and sum; sigmoid: denom 0).  Not inlined: the fp64 path runs
// cold, and its time is that of fetching its code.
__device__ __noinline__ double score_fp64(double z, double zmax, double denom) {
  const bool sigmoid = denom == 0.0;
  const bool limits = !sigmoid && !(fabs(zmax) < INFINITY);
  const double e = exp(sigmoid ? -z : z - zmax);
  if (sigmoid) return 1.0 / (1.0 + e);
  return (limits ? exp_limits(z, zmax) : e) / denom;
}

// Which experts a lane holds: 32 / n_group lanes (rounded down to a power of two) per group, neighbours in each.
struct Share {
  int lanes_log, group, n, e0;  // lanes per group (log2); this lane's group, experts, first expert
  __device__ __forceinline__ Share(int lane, const RouteGroupOpts& o) {
    const int n_group = o.n_group, gs = o.group_size;
    lanes_log = o.lanes_log;
    group = lane >> lanes_log;
    const int chunk = (gs + (1 << lanes_log) - 1) >> lanes_log;  // <= kPer
    const int from = (lane & ((1 << lanes_log) - 1)) * chunk;
    n = group < n_group ? max(0, min(chunk, gs - from)) : 0;
    e0 = n > 0 ? group * gs + from : 0;
  }
};

// One token in fp64, whatever its logits hold: the definition, and the answer for the tokens that the fp32 path
// leaves.  One warp, keys in registers; few tokens come here, so what counts is the time of one (it can be the last
// of the grid): the exponentials of a lane are independent chains, a choice is three warp reductions.
template <bool kBf16, int kPer>
__device__ __noinline__ void route_token_fp64(const void* row, const float* bias, int E, int K,
                                              const RouteGroupOpts o, int32_t* ids, float* w) {
  const int lane = threadIdx.x & 31;
  const int gs = o.group_size;
  const Share me(lane, o);
  const bool softmax = o.scoring == MOE_SCORE_SOFTMAX;
  double v[kPer];
  double zmax = -INFINITY, denom = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = i < me.n ? load_logit<kBf16>(row, me.e0 + i) : -INFINITY;
  if (softmax) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) zmax = fmax(zmax, v[i]);
    for (int off = 16; off >= 1; off >>= 1) zmax = fmax(zmax, shfl_xor_d(zmax, off));
    denom = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) denom += i < me.n ? score_fp64(v[i], zmax, 1.0) : 0.0;
    for (int off = 16; off >= 1; off >>= 1) denom += shfl_xor_d(denom, off);
    if (!(denom > 0.0)) denom = 1.0;  // a row of -inf only: every score is 0
  }
  auto score = [&](double z) { return score_fp64(z, zmax, denom); };
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const double p = score(v[i]);
    v[i] = rank_key(bias != nullptr && i < me.n ? p + static_cast<double>(bias[me.e0 + i]) : p);
  }

  // group scores, in every lane of the group
  bool kept = me.group < o.n_group;
  if (o.topk_group < o.n_group) {
    double a = -INFINITY, b = -INFINITY;  // two largest keys
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < me.n) {
        b = fmax(b, fmin(a, v[i]));
        a = fmax(a, v[i]);
      }
    for (int off = 1 << me.lanes_log >> 1; off >= 1; off >>= 1) {
      const double oa = shfl_xor_d(a, off), ob = shfl_xor_d(b, off);
      b = fmax(fmin(a, oa), fmax(b, ob));
      a = fmax(a, oa);
    }
    const double s = (o.group_score == MOE_GROUP_TOP2 && gs > 1) ? rank_key(a + b) : a;
    int before = 0;
    for (int q = 0; q < o.n_group; ++q) {
      const double x = __shfl_sync(0xffffffffu, s, q << me.lanes_log);
      before += x > s || (x == s && q < me.group);
    }
    kept = kept && before < o.topk_group;
  }
  // as integers that order like the numbers; 0: not (or no more) a candidate
  uint64_t u[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const uint64_t x = static_cast<uint64_t>(__double_as_longlong(v[i] + 0.0));
    u[i] = kept && i < me.n ? ((x >> 63) ? ~x : (x | 0x8000000000000000ull)) : 0ull;
  }
  int sel = 0;
  for (int k = 0; k < K; ++k) {
    uint64_t best = u[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < kPer; ++i)
      if (u[i] > best) {  // the first of equal ones stays
        best = u[i];
        bi = i;
      }
    const uint32_t hi = static_cast<uint32_t>(best >> 32);
    const uint32_t top = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t low = hi == top ? static_cast<uint32_t>(best) : 0u;
    const uint32_t low_top = __reduce_max_sync(0xffffffffu, low);
    const bool has = hi == top && static_cast<uint32_t>(best) == low_top && best != 0;
    const int win = static_cast<int>(__reduce_min_sync(0xffffffffu, has ? me.e0 + bi : E - 1));
    if (has && me.e0 + bi == win) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i == bi) u[i] = 0;
    }
    if (lane == k) sel = win;
  }
  double p = lane < K ? score(load_logit<kBf16>(row, sel)) : 0.0;
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

// Descending order by Batcher's odd-even merge network (n a power of two).
template <int kN>
__device__ __forceinline__ void sort_descending(uint32_t (&v)[kN]) {
#pragma unroll
  for (int p = 1; p < kN; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < kN; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < kN && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t a = v[i + j], b = v[i + j + k];
            v[i + j] = max(a, b);
            v[i + j + k] = min(a, b);
          }
}

// f(from) + .. + f(from + kN - 1) in pairs: log2(kN) roundings deep.
template <int kN, class F>
__device__ __forceinline__ float tree_sum(const F& f, int from = 0) {
  if constexpr (kN == 1)
    return f(from);
  else
    return tree_sum<kN / 2>(f, from) + tree_sum<kN / 2>(f, from + kN / 2);
}

// kPer: experts per lane, rounded up to a power of two.  kFull: every lane has exactly kPer, and every lane's logits
// start at a multiple of 16 bytes (or 8 experts or fewer at one of their own size).
template <bool kBf16, int kPer, bool kFull>
__global__ void __launch_bounds__(32 * kWarps) route_group_kernel(const void* __restrict__ logits, int64_t ld,
                                                                  const float* __restrict__ bias, int M, int E, int K,
                                                                  RouteGroupOpts o, int32_t* __restrict__ topk_ids,
                                                                  float* __restrict__ topk_w) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= M) return;
  const uint8_t* row = static_cast<const uint8_t*>(logits) + static_cast<size_t>(t) * ld * (kBf16 ? 2 : 4);
  int32_t* ids = topk_ids + static_cast<size_t>(t) * K;
  float* w = topk_w + static_cast<size_t>(t) * K;
  const bool softmax = o.scoring == MOE_SCORE_SOFTMAX;
  const bool groups = o.topk_group < o.n_group;
  const bool by_logit = bias == nullptr;
  const int gs = o.group_size;
  const bool group_sums = groups && o.group_score == MOE_GROUP_TOP2 && gs > 1;

  // ---- 1. this lane's experts and their keys
  const Share me(lane, o);
  const int lanes_log = me.lanes_log, group = me.group;
  const int n = kFull ? kPer : me.n;
  const int e0 = kFull ? kPer * lane : me.e0;
  float v[kPer];
  if (kFull) {
    constexpr int kBytes = kPer * (kBf16 ? 2 : 4);
    uint32_t x[(kBytes + 3) / 4];
    const uint8_t* src = row + static_cast<size_t>(lane) * kBytes;
    if (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 q = reinterpret_cast<const uint4*>(src)[i];
        x[(4 * i) % (kBytes / 4)] = q.x;
        x[(4 * i + 1) % (kBytes / 4)] = q.y;
        x[(4 * i + 2) % (kBytes / 4)] = q.z;
        x[(4 * i + 3) % (kBytes / 4)] = q.w;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        v[i] = !kBf16 ? __uint_as_float(x[i % (kBytes / 4)])
                      : (i & 1) ? bf16_hi(x[(i / 2) % (kBytes / 4)]) : bf16_lo(x[(i / 2) % (kBytes / 4)]);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = raw_logit<kBf16>(row, e0 + i);
    }
  } else if (kPer >= 4 && o.logits_by_4) {
#pragma unroll
    for (int i = 0; i + 3 < kPer; i += 4) {
      float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (i < n) {
        if (kBf16) {
          const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(static_cast<const void*>(row)) + e0 + i);
          q[0] = bf16_lo(x.x), q[1] = bf16_hi(x.x), q[2] = bf16_lo(x.y), q[3] = bf16_hi(x.y);
        } else {
          const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(row) + e0 + i);
          q[0] = x.x, q[1] = x.y, q[2] = x.z, q[3] = x.w;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) v[i + u] = q[u];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = i < n ? raw_logit<kBf16>(row, e0 + i) : 0.0f;
  }
  float zmax = 0.0f, denom = 1.0f;
  double denom64 = 1.0;  // of the weights, where they are shares of all experts
  if (softmax) {
    zmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (kFull || i < n) zmax = fmaxf(zmax, v[i]);
    zmax = from_order_bits(__reduce_max_sync(0xffffffffu, order_bits(zmax)));
    if (!o.renormalize) {
      // the rounding of z - max counts in full in the exponential of a far logit: it goes in as a factor
      denom64 = tree_sum<kPer>([&](int i) {
        if (!kFull && i >= n) return 0.0f;
        const float d = v[i] - zmax, back = d + zmax;
        const float lost = (v[i] - back) + ((back - d) - zmax);  // z - max = d + lost
        const float e = expf(d);
        return e > 0.0f ? fmaf(e, lost, e) : 0.0f;
      });
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) denom64 += shfl_xor_d(denom64, off);
      denom = static_cast<float>(denom64);
    } else if (!by_logit || group_sums) {
      denom = tree_sum<kPer>([&](int i) { return kFull || i < n ? expf(v[i] - zmax) : 0.0f; });
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) denom += __shfl_xor_sync(0xffffffffu, denom, off);
    }
  }
  const float inv_denom = rcp_approx(denom);
  auto score32 = [&](float z) {
    constexpr float kLog2e = 1.4426950408889634f;
    return softmax ? exp2_approx((z - zmax) * kLog2e) * inv_denom : rcp_approx(1.0f + exp2_approx(-z * kLog2e));
  };
  if (!by_logit) {
    if (kPer >= 4 && o.bias_by_4) {  // a lane's experts are neighbours: one by one its loads would touch 32 lines each
#pragma unroll
      for (int i = 0; i + 3 < kPer; i += 4)
        if (kFull || i < n) {
          const float4 b = *reinterpret_cast<const float4*>(bias + e0 + i);
          v[i] = score32(v[i]) + b.x;
          v[i + 1] = score32(v[i + 1]) + b.y;
          v[i + 2] = score32(v[i + 2]) + b.z;
          v[i + 3] = score32(v[i + 3]) + b.w;
        }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (kFull || i < n) v[i] = score32(v[i]) + bias[e0 + i];
    }
  }
  float hi = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (kFull || i < n) hi = fmaxf(hi, v[i]);
  const float kmax = from_order_bits(__reduce_max_sync(0xffffffffu, order_bits(hi)));
  // NaN as soon as a key is not finite; what a logit's NaN, or under softmax +inf, does to its key (a sigmoid of an
  // infinity is 0 or 1)
  float whole = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) whole = fmaf(v[i], 0.0f, whole);

  // ---- 2. integers
  const int id_bits = max(8, 32 - __clz(E - 1));  // E <= 1024: at most 10
  const uint32_t id_mask = (1u << id_bits) - 1u;
  const float steps = id_bits <= 9 ? 8388606.0f : 4194302.0f;  // 2^min(23, 32 - id_bits) - 2
  const float range = by_logit ? fmaf(0.5f, fabsf(kmax), 4.0f) : fabsf(kmax) + 2.0f;
  const float inv_range = rcp_approx(range);
  const float low = fmaf(-kmax, inv_range, 1.0f);  // key * inv_range + low: 1 at kmax, 0 at kmax - range
  const float step = range * (id_bits <= 9 ? 1.0f / 8388606.0f : 1.0f / 4194302.0f);
  const float sure = step * 0.9999f;               // of two keys n + 2 integers apart: n of these at least
  constexpr int kLen = kPer < 8 ? kPer : 8, kLists = kPer / kLen;
  uint32_t u[kLists][kLen];  // sorted lists of up to 8
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float at = __saturatef(fmaf(v[i], inv_range, low));
    // 2^23 + 1 .. 2^23 + steps + 1: shifting by id_bits >= 8 leaves the integer alone (bit 23 of 0x4b000000 is 0)
    const uint32_t q = __float_as_uint(fmaf(at, steps, 8388609.0f));
    u[i / kLen][i % kLen] = q * (id_mask + 1u) + (id_mask - static_cast<uint32_t>(e0 + i));
    if (!kFull && i >= n) u[i / kLen][i % kLen] = 0u;
  }
#pragma unroll
  for (int c = 0; c < kLists; ++c) sort_descending(u[c]);
  // what the keys may be off by, and the range that the integers show
  const float top_abs = by_logit ? 1.0f : fabsf(kmax) + range;
  const float off_key = (softmax ? 0x1p-18f * inv_denom : 0x1.8p-22f) + top_abs * 0x1p-23f;
  // a key from its integer: within two steps and the rounding of range and step (4 steps)
  auto value_of = [&](uint32_t q) { return fmaf(static_cast<float>(q), step, kmax - range); };

  // Two logits give scores that fp64 tells apart, in their order: they differ by more than 2^-30, and neither score
  // is so near to 1 or to 0 that the difference is lost there (e^-80 is above whatever lies below e^-600).
  auto clear_of_limits = [&](float zhi, float zlo) {
    return softmax ? (zlo - zmax > -600.0f || zhi - zmax > -80.0f) : (zhi < 12.0f && (zlo > -600.0f || zhi > -80.0f));
  };
  // Two logits with the integers q and q - apart: a tie, or apart as above (in the lowest integer anything may be).
  auto logits_clear = [&](uint32_t q, int apart, float zhi, float zlo) {
    if (kBf16 && q > 2 && fabsf(zhi) > 0x1p-20f && 5.0f * step < fabsf(zhi) * 0x1p-8f)
      return clear_of_limits(zhi, zlo);  // equal, or further apart than 4 steps and 2^-28
    return static_cast<float>(apart - 2) * sure > 0x1p-30f && clear_of_limits(zhi, zlo);
  };
  bool groups_good = true;

  // ---- 3. groups
  if (groups) {
    uint32_t a = u[0][0], b = kLen > 1 ? u[0][1 % kLen] : 0u;
#pragma unroll
    for (int c = 1; c < kLists; ++c) {
      b = max(min(a, u[c][0]), max(b, u[c][1 % kLen]));
      a = max(a, u[c][0]);
    }
    for (int off = 1 << lanes_log >> 1; off >= 1; off >>= 1) {
      const uint32_t oa = __shfl_xor_sync(0xffffffffu, a, off), ob = __shfl_xor_sync(0xffffffffu, b, off);
      b = max(min(a, oa), max(b, ob));
      a = max(a, oa);
    }
    a >>= id_bits;
    b >>= id_bits;
    // as an integer in every lane of the group: steps, or the bits of a (positive) sum of scores
    uint32_t s = a;
    if (group_sums) s = by_logit ? __float_as_uint(score32(value_of(a)) + score32(value_of(b))) : a + b;
    // the last group that stays (shi) and the first that does not (slo), ties to the lower group
    const bool real = group < o.n_group;
    bool stays;
    uint32_t shi = 0, slo;
    if (!(group_sums && by_logit)) {  // integers below 2^26: with the inverted group below, a maximum per group
      const uint32_t key = real ? (s << 5) + (31u - group) : 0u;
      uint32_t left = key, best = 0;
      for (int k = 0; k < o.topk_group; ++k) {
        best = __reduce_max_sync(0xffffffffu, left);
        left = left == best ? 0u : left;
      }
      stays = key >= best;
      shi = best >> 5;
      slo = __reduce_max_sync(0xffffffffu, left) >> 5;
    } else {
      int before = 0;  // groups ahead of this lane's
#pragma unroll 4
      for (int q = 0; q < o.n_group; ++q) {
        const uint32_t x = __shfl_sync(0xffffffffu, s, q << lanes_log);
        before += x > s || (x == s && q < group);
      }
      const unsigned last = __ballot_sync(0xffffffffu, real && before == o.topk_group - 1);
      const unsigned next = __ballot_sync(0xffffffffu, real && before == o.topk_group);
      shi = __shfl_sync(0xffffffffu, s, (__ffs(last) - 1) & 31);
      slo = __shfl_sync(0xffffffffu, s, (__ffs(next) - 1) & 31);
      stays = real && before < o.topk_group;
    }
    const int apart = static_cast<int>(shi - slo);
    if (!by_logit) {
      groups_good = static_cast<float>(apart - 4) * sure > 4.0f * off_key;
    } else if (group_sums) {
      const float fhi = __uint_as_float(shi);
      groups_good = fhi - __uint_as_float(slo) > 4.0f * (off_key + 6.0f * step) + fhi * 0x1p-22f;
    } else {
      groups_good = logits_clear(shi, apart, value_of(shi), value_of(slo));
    }
    // the lowest integer stands for anything below the range: a sum with it is an upper bound, which will do for a
    // group that goes (the lowest key comes out as 1 or 2)
    if (group_sums && stays && b <= 2) groups_good = false;
    if (!stays) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) u[i / kLen][i % kLen] = 0;
    }
  }

  // ---- 4. experts
  const int rounds = min(K + 1, o.topk_group * gs);
  uint32_t mine = 0, top = 0;  // of round `lane`; of the last round
  // of a list that gave `top` away, what `needed` more rounds can ask for moves up
  auto round = [&](int k, int needed) {
    uint32_t best = u[0][0];
#pragma unroll
    for (int c = 1; c < kLists; ++c) best = max(best, u[c][0]);
    top = __reduce_max_sync(0xffffffffu, best);
    if (best == top) {  // the owner, in one of its lists
#pragma unroll
      for (int c = 0; c < kLists; ++c)
        if (kLists == 1 || u[c][0] == top) {
#pragma unroll
          for (int i = 1; i < kLen; ++i)
            if (i <= needed) u[c][i - 1] = u[c][i];
          if (needed >= kLen) u[c][kLen - 1] = 0;
        }
    }
    if (lane == k) mine = top;
  };
  constexpr int kFew = 9;
  if (kLists == 1 && rounds <= kFew && rounds + 3 > kFew) {
    // 6 to 8 choices: nine rounds without a loop (one too many costs less than leaving early), each of which needs one
    // less of every list
#pragma unroll
    for (int k = 0; k < kFew; ++k) round(k, kFew - k);
  } else {
    for (int k = 0; k < rounds; ++k) round(k, kLen);
  }
  // every choice against the next one: lane k compares rounds k and k + 1 (round 32 is in no lane)
  auto id_of = [&](uint32_t x) { return min(static_cast<int>(id_mask - (x & id_mask)), E - 1); };
  int sel = id_of(mine);
  float zsel = lane < rounds ? raw_logit<kBf16>(row, sel) : 0.0f;
  const uint32_t below = __shfl_down_sync(0xffffffffu, mine, 1);
  float zlo = __shfl_down_sync(0xffffffffu, zsel, 1);
  bool good = true;
  if (lane + 1 < rounds) {
    const uint32_t other = lane < 31 ? below : top;
    if (lane == 31) zlo = raw_logit<kBf16>(row, id_of(other));
    const int apart = static_cast<int>(mine >> id_bits) - static_cast<int>(other >> id_bits);
    good = by_logit ? logits_clear(mine >> id_bits, apart, zsel, zlo)
                    : static_cast<float>(apart - 2) * sure > 2.0f * off_key;
  }
  // Not finite: an expert masked by -inf, in its logit or its bias, has the lowest integer like all that is far below;
  // +inf and NaN, and rows without a finite key, are the fp64 path's.
  bool usable = whole == 0.0f;
  if (!__all_sync(0xffffffffu, usable)) {
    usable = fabsf(kmax) < INFINITY && fabsf(zmax) < INFINITY;
#pragma unroll 1
    for (int i = 0; i < n; ++i)
      usable = usable && raw_logit<kBf16>(row, e0 + i) < INFINITY && (by_logit || bias[e0 + i] < INFINITY);
  }
  // scores far below the fp32 range are the fp64 path's
  const bool plain = groups_good && usable && !(lane < K && (softmax ? zsel - zmax : zsel) < -80.0f);
  bool settled = __all_sync(0xffffffffu, plain && good);
  if (!settled && __all_sync(0xffffffffu, plain) && (by_logit || !softmax) && K < 32) {
    // only neighbours in the list are too near: put the list in order by exact keys.  Nothing outside it can belong
    // to the choice if the best of the rest is clear of the K-th.
    const int listed = rounds;
    bool ok = true;
    if (o.topk_group * gs > listed) {
      uint32_t rest = u[0][0];
#pragma unroll
      for (int c = 1; c < kLists; ++c) rest = max(rest, u[c][0]);
      const uint32_t extra = __shfl_sync(0xffffffffu, mine, listed & 31);  // of a round too many
      if (listed < 32) rest = max(rest, extra);
      rest = __reduce_max_sync(0xffffffffu, rest);
      const int apart =
          static_cast<int>(__shfl_sync(0xffffffffu, mine, K - 1) >> id_bits) - static_cast<int>(rest >> id_bits);
      ok = static_cast<float>(apart - 2) * sure > (by_logit ? 0x1p-30f : 2.0f * off_key);
      if (by_logit) ok = ok && clear_of_limits(__shfl_sync(0xffffffffu, zsel, K - 1), value_of(rest >> id_bits));
    }
    if (ok) {
      double exact = zsel;  // the score grows with it
      if (!by_logit) exact = score_fp64(zsel, 0.0, 0.0) + static_cast<double>(bias[lane < listed ? sel : 0]);
      int place = 0, moved = sel;
      for (int j = 0; j < listed; ++j) {
        const double other = __shfl_sync(0xffffffffu, exact, j);
        const int id = __shfl_sync(0xffffffffu, sel, j);
        place += other > exact || (other == exact && id < sel);
      }
      for (int j = 0; j < listed; ++j) {
        const int at = __shfl_sync(0xffffffffu, place, j), id = __shfl_sync(0xffffffffu, sel, j);
        if (at == lane) moved = id;
      }
      sel = moved;
      if (lane < listed) zsel = raw_logit<kBf16>(row, sel);
      zlo = __shfl_down_sync(0xffffffffu, zsel, 1);
      if (by_logit && lane + 1 < listed)
        ok = zsel == zlo || (zsel - zlo > 0x1p-30f && clear_of_limits(zsel, zlo));
      ok = ok && !(lane < K && (softmax ? zsel - zmax : zsel) < -80.0f);
    }
    settled = __all_sync(0xffffffffu, ok);
  }
  if (!settled) {
    route_token_fp64<kBf16, kPer>(row, bias, E, K, o, ids, w);
    return;
  }

  // ---- 5. weights
  double p = 0.0;
  if (lane < K) {  // z >= -80 here (softmax: z - zmax)
    const double z = static_cast<double>(zsel);
    const double e = exp_reduced(softmax ? z - static_cast<double>(zmax) : -fmin(z, 100.0));
    p = softmax ? e : reciprocal(1.0 + e);
  }
  double total = denom64;
  if (o.renormalize) {
    total = p;
    if (K > 8) {
      total += shfl_xor_d(total, 16);
      total += shfl_xor_d(total, 8);
    }
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) total += shfl_xor_d(total, off);
  }
  if (lane < K) {
    ids[lane] = sel;
    w[lane] = static_cast<float>(p * (reciprocal(total) * static_cast<double>(o.routed_scale)));
  }
}

template <bool kBf16, int kPer>
cudaError_t launch_per(const void* logits, int64_t ld, const float* bias, int M, int E, int K, const RouteGroupOpts& o,
                       int32_t* topk_ids, float* topk_w, cudaStream_t stream) {
  const dim3 grid((M - 1) / kWarps + 1);  // M + kWarps - 1 may pass 2^31
  const int size = kBf16 ? 2 : 4;
  const int vec = kPer * size < 16 ? size : 16;  // bytes of a load
  const bool full = E == 32 * kPer && (o.n_group & (o.n_group - 1)) == 0 && (ld * size) % vec == 0 &&
                    (reinterpret_cast<uintptr_t>(logits) & (vec - 1)) == 0;
  if (full)
    route_group_kernel<kBf16, kPer, true>
        <<<grid, 32 * kWarps, 0, stream>>>(logits, ld, bias, M, E, K, o, topk_ids, topk_w);
  else
    route_group_kernel<kBf16, kPer, false>
        <<<grid, 32 * kWarps, 0, stream>>>(logits, ld, bias, M, E, K, o, topk_ids, topk_w);
  return cudaGetLastError();
}

template <bool kBf16>
cudaError_t launch_typed(const void* logits, int64_t ld, const float* bias, int M, int E, int K,
                         RouteGroupOpts o, int32_t* topk_ids, float* topk_w, cudaStream_t stream) {
  o.group_size = E / o.n_group;
  o.lanes_log = 0;
  while ((2 << o.lanes_log) * o.n_group <= 32) ++o.lanes_log;
  const int per = (o.group_size + (1 << o.lanes_log) - 1) >> o.lanes_log;
  // whether every lane's experts start and end at a multiple of four, and the rows (the bias) can be read so
  const bool fours = per % 4 == 0 && o.group_size % 4 == 0;
  const int size = kBf16 ? 2 : 4;
  o.logits_by_4 = fours && ld % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & (4 * size - 1)) == 0;
  o.bias_by_4 = fours && (reinterpret_cast<uintptr_t>(bias) & 15u) == 0;
  // experts per lane: at most 60 (17 groups, one lane each)
  auto run = [&](auto f) { return f(logits, ld, bias, M, E, K, o, topk_ids, topk_w, stream); };
  if (per <= 1) return run(launch_per<kBf16, 1>);
  if (per <= 2) return run(launch_per<kBf16, 2>);
  if (per <= 4) return run(launch_per<kBf16, 4>);
  if (per <= 8) return run(launch_per<kBf16, 8>);
  if (per <= 16) return run(launch_per<kBf16, 16>);
  if (per <= 32) return run(launch_per<kBf16, 32>);
  return run(launch_per<kBf16, 64>);
}

}  // namespace

cudaError_t launch_route_group(const void* logits, bool bf16, int64_t ld, const float* bias, int M, int E, int K,
                               const RouteGroupOpts& o, int32_t* topk_ids, float* topk_w, cudaStream_t stream) {
  return bf16 ? launch_typed<true>(logits, ld, bias, M, E, K, o, topk_ids, topk_w, stream)
              : launch_typed<false>(logits, ld, bias, M, E, K, o, topk_ids, topk_w, stream);
}

}  // namespace moe
