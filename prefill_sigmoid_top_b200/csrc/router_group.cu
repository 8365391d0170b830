// Routing from given logits with expert groups (moe_route_logits): scores, a bias that shifts the selection
// only, the best groups, the best experts of those groups, weights.
//
//   p_e   = 1 / (1 + e^-z_e), or e^(z_e - max) / sum_j e^(z_j - max)
//   key_e = p_e + bias_e
//   s_g   = the largest key of group g, or the sum of its two largest
//   the topk_group groups with the largest s_g stay; of their experts the top_k with the largest keys, ties to
//   the lower id;  w_k = p_k, or p_k / sum_j p_j, times routed_scale.
//
// The choice is a comparison of sums of rounded numbers, so it is defined in 64 bits: p, keys and group scores
// in fp64.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kWarps = 4;  // one token per warp

__device__ __forceinline__ double shfl_xor_d(double v, int off) { return __shfl_xor_sync(0xffffffffu, v, off); }

// NaN ranks below every number.
__device__ __forceinline__ double rank_key(double v) { return isnan(v) ? -INFINITY : v; }

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* row, int e) {
  float z;
  if (kBf16)
    z = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(row)[e]) << 16);
  else
    z = static_cast<const float*>(row)[e];
  return isnan(z) ? -INFINITY : z;
}

// e^(z - zmax) with the limits: a row whose largest logit is +inf shares among its +inf entries, a row of
// -inf only has no scores.
__device__ __forceinline__ double exp_score(double z, double zmax) {
  if (zmax == -INFINITY) return 0.0;
  if (zmax == INFINITY) return z == INFINITY ? 1.0 : 0.0;
  return exp(z - zmax);
}

template <bool kBf16>
__global__ void __launch_bounds__(32 * kWarps) route_group_kernel(const void* __restrict__ logits, int64_t ld,
                                                                  const float* __restrict__ bias, int M, int E, int K,
                                                                  RouteGroupOpts o, int32_t* __restrict__ topk_ids,
                                                                  float* __restrict__ topk_w) {
  extern __shared__ double keys_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= M) return;
  double* key = keys_smem + warp * E;
  const uint8_t* row = static_cast<const uint8_t*>(logits) + static_cast<size_t>(t) * ld * (kBf16 ? 2 : 4);

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
    topk_ids[static_cast<size_t>(t) * K + lane] = sel;
    topk_w[static_cast<size_t>(t) * K + lane] = static_cast<float>(p * static_cast<double>(o.routed_scale));
  }
}

}  // namespace

cudaError_t launch_route_group(const void* logits, bool bf16, int64_t ld, const float* bias, int M, int E, int K,
                               const RouteGroupOpts& o, int32_t* topk_ids, float* topk_w, cudaStream_t stream) {
  const dim3 grid((M + kWarps - 1) / kWarps);
  const size_t smem = sizeof(double) * kWarps * E;  // at most 32 KB
  if (bf16)
    route_group_kernel<true><<<grid, 32 * kWarps, smem, stream>>>(logits, ld, bias, M, E, K, o, topk_ids, topk_w);
  else
    route_group_kernel<false><<<grid, 32 * kWarps, smem, stream>>>(logits, ld, bias, M, E, K, o, topk_ids, topk_w);
  return cudaGetLastError();
}

}  // namespace moe
