// The router's choice for one token: sigmoid, bias, group-limited top-k, gates.
//
// Reading of "DSV3-style router" (Cursor blog summary, "method points"):
// s = sigmoid(logit) in the specified fp32 arithmetic below, v = s + bias,
// group score = sum of the two largest v of the group, keep the topk_groups
// best groups (ties to the lower group), take the k best v among kept
// experts (ties to the lower expert), slots in descending-v order, gates
// w = s / sum(s) summed in slot order.
#pragma once
#include "moe_internal.h"

namespace moe {

// sigma(l) = 1 / (1 + E(-clamp(l, -80, 80))), E by Cody-Waite reduction
// (W. J. Cody and W. Waite, 1980) and a degree-7 Taylor polynomial, every
// operation an IEEE binary32 round-to-nearest op without contraction.
__device__ __forceinline__ float sigmoid_spec(float l) {
  constexpr double kLn2 = 0.6931471805599453094;
  constexpr float kLog2e = static_cast<float>(1.0 / kLn2);
  constexpr float kC1 = 355.0f / 512.0f;                               // ln2 to 9 significant bits
  constexpr float kC2 = static_cast<float>(kLn2 - 355.0 / 512.0);      // remainder
  constexpr float c0 = 1.0f, c1 = 1.0f, c2 = 0.5f;
  constexpr float c3 = static_cast<float>(1.0 / 6.0), c4 = static_cast<float>(1.0 / 24.0);
  constexpr float c5 = static_cast<float>(1.0 / 120.0), c6 = static_cast<float>(1.0 / 720.0);
  constexpr float c7 = static_cast<float>(1.0 / 5040.0);
  const float lc = fminf(fmaxf(l, -80.0f), 80.0f);
  const float z = -lc;
  const float n = rintf(__fmul_rn(z, kLog2e));
  const float r = __fsub_rn(__fsub_rn(z, __fmul_rn(n, kC1)), __fmul_rn(n, kC2));
  float p = c7;
  p = __fadd_rn(__fmul_rn(p, r), c6);
  p = __fadd_rn(__fmul_rn(p, r), c5);
  p = __fadd_rn(__fmul_rn(p, r), c4);
  p = __fadd_rn(__fmul_rn(p, r), c3);
  p = __fadd_rn(__fmul_rn(p, r), c2);
  p = __fadd_rn(__fmul_rn(p, r), c1);
  p = __fadd_rn(__fmul_rn(p, r), c0);
  const float two_n = __int_as_float((static_cast<int>(n) + 127) << 23);
  const float e = __fmul_rn(p, two_n);
  return __fdiv_rn(1.0f, __fadd_rn(1.0f, e));
}

// (v1, e1) ranks above (v2, e2): larger value, ties to the lower index.
__device__ __forceinline__ bool better(float v1, int e1, float v2, int e2) {
  return v1 > v2 || (v1 == v2 && e1 < e2);
}

__device__ __forceinline__ void warp_best(float& v, int& e) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float ov = __shfl_xor_sync(0xffffffffu, v, o);
    const int oe = __shfl_xor_sync(0xffffffffu, e, o);
    if (better(ov, oe, v, e)) { v = ov; e = oe; }
  }
}

// The best pair of a warp, in every lane's e, by shuffles or by warp-wide integer reductions: the same choice among numbers. A
// kernel with few tokens waits for the choice: with reductions, in a loop, compiled for the experts a lane has, it takes 3 us
// from the last logit, where shuffles unrolled for 512 experts took 8.6.
struct BestByShuffles {
  static constexpr int kRounds = 8;        // selection rounds unrolled
  static __device__ __forceinline__ void of(float& v, int& e) { warp_best(v, e); }
};
struct BestByRedux {
  static constexpr int kRounds = 1;        // (one launch for a few tokens fetches the code once: a round's code again costs more than a loop)
  static __device__ __forceinline__ void of(float& v, int& e) {
    const uint32_t bits = __float_as_uint(v + 0.0f);       // (-0 counts as 0)
    const uint32_t key = v != v ? 0u : bits ^ (bits >> 31 ? 0xffffffffu : 0x80000000u);
    const uint32_t top = __reduce_max_sync(0xffffffffu, key);
    e = static_cast<int>(__reduce_min_sync(0xffffffffu, key == top ? static_cast<uint32_t>(e) : 0x7fffffffu));
  }
};

// One warp chooses for one token. Lane l owns experts e = l + 32 i, i < kMaxPerLane
// (a compile-time bound on ceil(E / 32), so the per-lane loops have no dead
// iterations at the common expert counts). logit(e) and bias(e) read the token's
// values; sv is scratch of E floats in shared memory. Lane j < k gets slot j: its
// expert, its score s, and the sum of all slots' scores.
template <int kMaxPerLane, typename Best, typename Logit, typename Bias>
__device__ __forceinline__ void choose_experts(Logit logit, Bias bias, int E, int k, int G, int gtop, float* sv, int lane,
                                               int& my_e, float& my_s, float& tot) {
  float s[kMaxPerLane], v[kMaxPerLane];
  const int per_lane = (E + 31) / 32;
#pragma unroll
  for (int i = 0; i < kMaxPerLane; ++i) {
    const int e = lane + 32 * i;
    if (i < per_lane && e < E) {
      s[i] = sigmoid_spec(logit(e));
      v[i] = __fadd_rn(s[i], bias(e));
      sv[e] = v[i];
    } else {
      s[i] = 0.0f;
      v[i] = -INFINITY;
    }
  }
  __syncwarp();
  uint32_t kept = 0xffffffffu;
  if (G > 1) {
    const int per = E / G;
    float gs = -INFINITY;
    if (lane < G) {
      float m1 = -INFINITY, m2 = -INFINITY;
      for (int e = lane * per; e < (lane + 1) * per; ++e) {
        const float x = sv[e];
        if (x > m1) { m2 = m1; m1 = x; } else if (x > m2) { m2 = x; }
      }
      gs = __fadd_rn(m1, m2);
    }
    kept = 0;
    for (int r = 0; r < gtop; ++r) {
      float bv = (lane < G && !((kept >> lane) & 1u)) ? gs : -INFINITY;
      int be = lane < G && !((kept >> lane) & 1u) ? lane : 0x7fffffff;
      Best::of(bv, be);
      kept |= 1u << be;
    }
  }
  // This lane's candidates (experts of kept groups), one bit per slot i:
  // the group of each slot is found once, not in every selection round.
  const int per = G > 1 ? E / G : E;
  uint32_t cand = 0;
#pragma unroll
  for (int i = 0; i < kMaxPerLane; ++i) {
    const int e = lane + 32 * i;
    if (i < per_lane && e < E && ((kept >> (e / per)) & 1u)) cand |= 1u << i;
  }
  uint32_t taken = 0;
  tot = my_s = 0.0f;
  my_e = 0;
#pragma unroll(Best::kRounds)
  for (int j = 0; j < 8; ++j) {            // k <= 8 (checked by the API)
    if (j >= k) break;                     // k is the same in every lane
    float bv = -INFINITY;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i) {
      const int e = lane + 32 * i;
      if (((cand & ~taken) >> i) & 1u) {
        if (better(v[i], e, bv, be)) { bv = v[i]; be = e; }
      }
    }
    Best::of(bv, be);
    if ((be & 31) == lane) taken |= 1u << (be >> 5);
    float sw = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i)
      if (i == (be >> 5)) sw = s[i];
    const float sj = __shfl_sync(0xffffffffu, sw, be & 31);
    // every lane sums the selected scores in slot order; lane j holds slot j
    tot = j == 0 ? sj : __fadd_rn(tot, sj);
    if (lane == j) {
      my_s = sj;
      my_e = be;
    }
  }
}

}  // namespace moe
