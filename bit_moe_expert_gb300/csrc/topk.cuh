// Top-k selection and routing weights for one token, by one warp.  Used by the
// routing kernel and by the decode kernel when it routes its own tokens, so
// both produce the same bits.
//
// "Perplexity's Lily Beats MLX-LM on MacBook M5", section "Why Qwen3.6-35B-A3B
// is a weird workload": the router scores 256 experts and picks 8.  Selection
// is on the raw fp32 logits (softmax is monotone); a lower expert index wins a
// tie; the weights are the softmax over the selected logits, computed in fp64
// (exp(l_j - l_max), summed in selection order) and rounded once to fp32.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"

namespace bm {

// Monotone 32-bit key of a logit: a larger float gives a larger unsigned key;
// -0.0 becomes +0.0 first, so equal floats always get equal keys.
__device__ __forceinline__ uint32_t topk_key(float v) {
  if (v == 0.0f) v = 0.0f;
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float topk_key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// Lane l's eight logits 8l .. 8l+7 of a row of E <= 256 (zero past E).
__device__ __forceinline__ void topk_load_row8(const float* __restrict__ row, int E, int lane, float (&xv)[8]) {
  if (E == 256 && (reinterpret_cast<uintptr_t>(row) & 15u) == 0) {
    // two 16-byte loads per lane: the warp reads the row as eight whole lines
    const float4 lo = __ldcg(reinterpret_cast<const float4*>(row) + 2 * lane);
    const float4 hi = __ldcg(reinterpret_cast<const float4*>(row) + 2 * lane + 1);
    xv[0] = lo.x, xv[1] = lo.y, xv[2] = lo.z, xv[3] = lo.w;
    xv[4] = hi.x, xv[5] = hi.y, xv[6] = hi.z, xv[7] = hi.w;
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) xv[c] = 8 * lane + c < E ? __ldcg(row + 8 * lane + c) : 0.0f;
  }
}

// k rounds over the lanes' eight values each (see warp_topk_select_sorted_vals;
// 0 is no candidate): lane j < k receives the key and the expert of round j.
__device__ __forceinline__ void warp_topk_rounds8(uint64_t (&v)[8], int k, int lane, uint32_t& sel_key, int& sel_i) {
  constexpr int kNet[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                               {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
  for (int c = 0; c < 19; ++c) {
    const uint64_t a = v[kNet[c][0]], b = v[kNet[c][1]];
    v[kNet[c][0]] = a > b ? a : b;
    v[kNet[c][1]] = a > b ? b : a;
  }
  sel_key = 0;
  sel_i = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t hk = static_cast<uint32_t>(v[0] >> 32);
    const uint32_t kmax = __reduce_max_sync(0xffffffffu, hk);
    const unsigned cand = __ballot_sync(0xffffffffu, hk == kmax && v[0] != 0ull);
    const int win = __ffs(cand) - 1;
    const uint32_t wlow = __shfl_sync(0xffffffffu, static_cast<uint32_t>(v[0]), win);
    if (lane == j) {
      sel_key = kmax;
      sel_i = static_cast<int>(~wlow);
    }
    if (lane == win) {
#pragma unroll
      for (int c = 0; c < 7; ++c) v[c] = v[c + 1];
      v[7] = 0ull;
    }
  }
}

// Selection for E <= 256 from the lanes' loaded logits: lane l holds experts
// 8l .. 8l+7 as 64-bit values (key << 32 | ~expert), so a larger value is a
// larger logit or, for equal logits, a lower expert; it sorts them once (a
// 19-comparator network), and each of the k rounds takes the largest head key
// over the lanes (the lowest lane among equal heads holds the lowest expert,
// lanes holding contiguous experts) and pops that lane's head.
__device__ __forceinline__ void warp_topk_select_sorted_vals(const float (&xv)[8], int E, int k, int lane,
                                                             int& sel_i, float& sel_v, bool& all_finite) {
  uint64_t v[8];
  bool finite = true;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const int e = 8 * lane + c;
    finite &= e >= E || isfinite(xv[c]);
    v[c] = e < E ? (static_cast<uint64_t>(topk_key(xv[c])) << 32) | static_cast<uint32_t>(~e) : 0ull;
  }
  all_finite = __all_sync(0xffffffffu, finite);
  uint32_t sel_key;
  warp_topk_rounds8(v, k, lane, sel_key, sel_i);
  sel_v = topk_key_value(sel_key);
}

__device__ __forceinline__ void warp_topk_select_sorted(const float* __restrict__ row, int E, int k, int lane,
                                                        int& sel_i, float& sel_v, bool& all_finite) {
  float xv[8];
  topk_load_row8(row, E, lane, xv);
  warp_topk_select_sorted_vals(xv, E, k, lane, sel_i, sel_v, all_finite);
}

// The same for E <= 32 * kPL with expert lane + 32 c at key[c]; a set bit c of
// `taken` is no candidate.
template <int kPL>
__device__ __forceinline__ void warp_topk_rounds_wide(const uint32_t (&key)[kPL], uint32_t taken, int k, int lane,
                                                      uint32_t& sel_key, int& sel_i) {
  sel_key = 0;  // lane j keeps the j-th selected key
  sel_i = 0;
  for (int j = 0; j < k; ++j) {
    // lane-local best: largest key, lowest index among equal keys
    uint32_t bk = 0;
    int bi = 0x7FFFFFFF;
#pragma unroll
    for (int c = 0; c < kPL; ++c) {
      if (!((taken >> c) & 1u) && (key[c] > bk || bi == 0x7FFFFFFF)) {
        bk = key[c];
        bi = lane + 32 * c;
      }
    }
    const uint32_t kmax = __reduce_max_sync(0xffffffffu, bi == 0x7FFFFFFF ? 0u : bk);
    const int win = static_cast<int>(
        __reduce_min_sync(0xffffffffu, (bi != 0x7FFFFFFF && bk == kmax) ? static_cast<uint32_t>(bi) : 0xFFFFFFFFu));
    if ((win & 31) == lane) taken |= 1u << (win >> 5);
    if (lane == j) {
      sel_key = kmax;
      sel_i = win;
    }
  }
}

// Selection.  row: E <= 32 * kPL fp32 logits.  On return lane j < k holds the
// j-th selected expert (descending logit) in sel_i and its logit in sel_v;
// every lane learns whether the row was all finite.
template <int kPL>
__device__ __forceinline__ void warp_topk_select(const float* __restrict__ row, int E, int k, int lane, int& sel_i,
                                                 float& sel_v, bool& all_finite) {
  if constexpr (kPL == 8) {
    warp_topk_select_sorted(row, E, k, lane, sel_i, sel_v, all_finite);
    return;
  }
  // Monotone 32-bit keys: a larger float gives a larger unsigned key.  -0.0
  // becomes +0.0 first, so equal floats always get equal keys.
  uint32_t key[kPL];
  uint32_t taken = 0;
  bool finite = true;
#pragma unroll
  for (int c = 0; c < kPL; ++c) {
    const int e = lane + 32 * c;
    const bool in = e < E;
    float v = in ? __ldg(row + e) : 0.0f;
    finite &= !in || isfinite(v);
    if (v == 0.0f) v = 0.0f;
    const uint32_t u = __float_as_uint(v);
    key[c] = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    if (!in) taken |= 1u << c;
  }
  all_finite = __all_sync(0xffffffffu, finite);

  uint32_t sel_key;
  warp_topk_rounds_wide<kPL>(key, taken, k, lane, sel_key, sel_i);
  // back from key to float
  const uint32_t su = (sel_key & 0x80000000u) ? (sel_key & 0x7FFFFFFFu) : ~sel_key;
  sel_v = __uint_as_float(su);
}

// Weights of a selection (sel_v of lanes 0..k-1, lane 0 the largest): the
// softmax over the selected logits in fp64, summed in selection order, rounded
// once to fp32.  Lane j < k receives weight j.
__device__ __forceinline__ float warp_topk_weights(float sel_v, int k, int lane) {
  const float top = __shfl_sync(0xffffffffu, sel_v, 0);
  const double ex = (lane < k) ? exp(static_cast<double>(sel_v) - static_cast<double>(top)) : 0.0;
  double sum = 0.0;
  for (int j = 0; j < k; ++j) sum += __shfl_sync(0xffffffffu, ex, j);
  return static_cast<float>(ex / sum);
}

// ------------------------------------------------------------------ scores, bias, groups
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) { return topk_key_value(__reduce_max_sync(0xffffffffu, topk_key(v))); }

// The expert at position c of a lane's kPL logits (the layouts of the two
// selections above).
template <int kPL>
__device__ __forceinline__ int lane_expert(int lane, int c) {
  return kPL == 8 ? 8 * lane + c : lane + 32 * c;
}

// Selection and weights of one row by scores: xv holds the lane's logits
// (anything past E).  On return lane j < k holds the j-th expert and its weight;
// every lane learns whether the row and the bias had no NaN and no +infinity.
// buf: E floats of shared memory of this warp's own, used with groups only.
//
// Groups: the values go to shared memory and lane g reads group g's, each lane
// starting at another place of its run so that runs of 32 do not meet in one
// bank.  With 8 groups of 32 that is 32 loads for the two largest of every
// group, where a reduction over the lanes' registers takes ten shuffles a group
// and value.
template <int kPL>
__device__ __forceinline__ void warp_scored_topk(const float (&xv)[kPL], const RouteScore& sc, int E, int k, int lane,
                                                 float* buf, int& sel_i, float& sel_w, bool& all_ok) {
  const float kNone = -INFINITY;
  float s[kPL];         // scores
  float choice[kPL];
  bool ok = true;
  float mx = kNone;
#pragma unroll
  for (int c = 0; c < kPL; ++c) {
    const bool in = lane_expert<kPL>(lane, c) < E;
    const bool bad = in && !(xv[c] < INFINITY);
    ok &= !bad;
    choice[c] = in && !bad ? xv[c] : kNone;  // the logit, -infinity for a masked expert
    mx = fmaxf(mx, choice[c]);
  }
  if (sc.sigmoid) {
#pragma unroll
    for (int c = 0; c < kPL; ++c) s[c] = 1.0f / (1.0f + expf(-choice[c]));  // exp(inf) = inf: a masked expert gets 0
  } else {
    mx = warp_max(mx);
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kPL; ++c) {
      s[c] = choice[c] > kNone ? expf(choice[c] - mx) : 0.0f;
      sum += s[c];
    }
    sum = warp_sum(sum);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int c = 0; c < kPL; ++c) s[c] *= inv;
  }
  if (sc.bias) {
#pragma unroll
    for (int c = 0; c < kPL; ++c) {
      const int e = lane_expert<kPL>(lane, c);
      if (e < E) {
        const float b = __ldg(sc.bias + e);
        const float v = s[c] + b;
        ok &= v == v;
        choice[c] = choice[c] > kNone && v == v ? v : kNone;
      }
    }
  }
  all_ok = __all_sync(0xffffffffu, ok);

  uint32_t kept = 0xffffffffu;  // groups that are selected from
  const int gsize = E / sc.n_group;
  if (sc.n_group > 1) {
#pragma unroll
    for (int c = 0; c < kPL; ++c) {
      const int e = lane_expert<kPL>(lane, c);
      if (e < E) buf[e] = sc.bias || !(choice[c] > kNone) ? choice[c] : s[c];
    }
    __syncwarp();
    float m1 = kNone, m2 = kNone;
    if (lane < sc.n_group) {
      int i = lane % gsize;
      for (int n = 0; n < gsize; ++n) {
        const float v = buf[lane * gsize + i];
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
        if (++i == gsize) i = 0;
      }
    }
    const float mine = sc.group_top == 2 && m2 > kNone ? m1 + m2 : m1;
    int rank = 0;
    for (int g = 0; g < sc.n_group; ++g) {
      const float v = __shfl_sync(0xffffffffu, mine, g);
      rank += (v > mine || (v == mine && g < lane)) ? 1 : 0;
    }
    kept = __ballot_sync(0xffffffffu, lane < sc.n_group && rank < sc.topk_group);
    __syncwarp();  // buf may be written for the next row
  }

  uint32_t sel_key;
  if constexpr (kPL == 8) {
    uint64_t v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int e = 8 * lane + c;
      const bool in = e < E && (sc.n_group == 1 || ((kept >> (e / gsize)) & 1u));
      v[c] = in ? (static_cast<uint64_t>(topk_key(choice[c])) << 32) | static_cast<uint32_t>(~e) : 0ull;
    }
    warp_topk_rounds8(v, k, lane, sel_key, sel_i);
  } else {
    uint32_t key[kPL], taken = 0;
#pragma unroll
    for (int c = 0; c < kPL; ++c) {
      const int e = lane + 32 * c;
      const bool in = e < E && (sc.n_group == 1 || ((kept >> (e / gsize)) & 1u));
      key[c] = topk_key(choice[c]);
      if (!in) taken |= 1u << c;
    }
    warp_topk_rounds_wide<kPL>(key, taken, k, lane, sel_key, sel_i);
  }

  const int owner = kPL == 8 ? sel_i >> 3 : sel_i & 31;
  const int at = kPL == 8 ? sel_i & 7 : sel_i >> 5;
  float w = 0.0f;
#pragma unroll
  for (int c = 0; c < kPL; ++c) {
    const float v = __shfl_sync(0xffffffffu, s[c], owner);
    if (at == c) w = v;
  }
  if (lane >= k) w = 0.0f;
  if (sc.renormalize) {
    const float sum = warp_sum(w);
    w = sum > 0.0f ? w / sum : 0.0f;
  }
  sel_w = w * sc.scale;
}

}  // namespace bm
