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
  constexpr int kNet[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                               {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
  for (int c = 0; c < 19; ++c) {
    const uint64_t a = v[kNet[c][0]], b = v[kNet[c][1]];
    v[kNet[c][0]] = a > b ? a : b;
    v[kNet[c][1]] = a > b ? b : a;
  }
  uint32_t sel_key = 0;
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
  sel_v = topk_key_value(sel_key);
}

__device__ __forceinline__ void warp_topk_select_sorted(const float* __restrict__ row, int E, int k, int lane,
                                                        int& sel_i, float& sel_v, bool& all_finite) {
  float xv[8];
  topk_load_row8(row, E, lane, xv);
  warp_topk_select_sorted_vals(xv, E, k, lane, sel_i, sel_v, all_finite);
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

  uint32_t sel_key = 0;  // lane j keeps the j-th selected key
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

// Shared memory of a warp that selects by scores: the list of candidates, then,
// where groups do not fall on whole lanes (group_shift -1), E floats.
// Rows of up to 256 experts keep 32 candidates, wider ones 128.
template <int kPL>
constexpr int kScoredList = kPL == 8 ? 32 : 128;
template <int kPL>
struct ScoredList {
  uint2 key_e[kScoredList<kPL>];
  float s[kScoredList<kPL>];
};

// A row's logits and the bias, in flight together (-infinity and 0 past E).
template <int kPL>
__device__ __forceinline__ void scored_load(const float* __restrict__ row, const float* __restrict__ bias, int E,
                                            int pl, int lane, float (&x)[kPL], float (&b)[kPL]) {
  if (kPL == 8 && E == 256 && ((reinterpret_cast<uintptr_t>(row) | reinterpret_cast<uintptr_t>(bias)) & 15u) == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(row) + 2 * lane + h);
      const float4 u = bias ? __ldg(reinterpret_cast<const float4*>(bias) + 2 * lane + h) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[4 * h] = v.x, x[4 * h + 1] = v.y, x[4 * h + 2] = v.z, x[4 * h + 3] = v.w;
      b[4 * h] = u.x, b[4 * h + 1] = u.y, b[4 * h + 2] = u.z, b[4 * h + 3] = u.w;
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < kPL; ++c) {
    const int e = pl * lane + c;
    const bool in = c < pl && e < E;
    x[c] = in ? __ldcg(row + e) : -INFINITY;
    b[c] = in && bias ? __ldg(bias + e) : 0.0f;
  }
}

// Selection and weights of one row by scores (include/moe.h, moe_scoring), x
// and b from scored_load.  Calls publish(j, expert, weight) once for every slot
// j < k, each in some lane; returns whether the row and the bias had no NaN and
// no +infinity.
//
// No serial rounds over k: the k-th largest of the lanes' own maxima bounds the
// k-th largest choice from below, so the experts at or above it (about k to 2k
// of them) go to a list in shared memory, and each lane counts for one of them
// how many come before it.  k rounds of a maximum over the warp took 3,400
// cycles of a token's 8,400 with k = 8; more candidates than the list holds (k
// close to 32, or many equal choices) still take them.
template <int kPL, typename Publish>
__device__ __forceinline__ bool warp_scored_topk(const float (&x)[kPL], const float (&b)[kPL], const RouteScore& sc,
                                                 int E, int k, int lane, ScoredList<kPL>* list, Publish publish) {
  const float kNone = -INFINITY;
  const uint32_t kAll = 0xffffffffu;
  const int pl = sc.per_lane;
  float s[kPL], choice[kPL];
  bool ok = true;
  float mx = kNone;
#pragma unroll
  for (int c = 0; c < kPL; ++c) {
    const bool bad = !(x[c] < INFINITY);
    ok &= !bad;
    choice[c] = bad ? kNone : x[c];  // the logit, -infinity for a masked expert
    mx = fmaxf(mx, choice[c]);
  }
  if (sc.sigmoid) {
    // from -80 down 1 / (1 + e^-l) is e^l in fp32, to its smallest subnormal: the approximate quotient is 0 for a
    // denominator from 2^126 on (l < -87.3)
#pragma unroll
    for (int c = 0; c < kPL; ++c) {
      const bool low = choice[c] < -80.0f;  // a masked expert: e^-inf = 0
      const float z = expf(low ? choice[c] : -choice[c]);
      s[c] = low ? z : __fdividef(1.0f, 1.0f + z);
    }
  } else {
    mx = topk_key_value(__reduce_max_sync(kAll, topk_key(mx)));
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kPL; ++c) {
      s[c] = choice[c] > kNone ? expf(choice[c] - mx) : 0.0f;
      sum += s[c];
    }
    sum = warp_sum(sum);
    const float inv = sum > 0.0f ? __fdividef(1.0f, sum) : 0.0f;
#pragma unroll
    for (int c = 0; c < kPL; ++c) s[c] *= inv;
  }
  if (sc.bias) {
#pragma unroll
    for (int c = 0; c < kPL; ++c) {
      const float v = s[c] + b[c];
      ok &= v == v;
      choice[c] = choice[c] > kNone && v == v ? v : kNone;
    }
  }
  ok = __all_sync(kAll, ok);

  uint32_t kept = kAll;  // groups that are selected from
  const int size = sc.group_size;
  const bool whole = sc.group_shift >= 0;
  if (sc.n_group > 1) {
    // group g's value ends up in lane g (smem) or in all of its lanes
    float m1 = kNone, m2 = kNone, mine;
    int group, shift;
    if (whole) {
#pragma unroll
      for (int c = 0; c < kPL; ++c) {
        const float v = sc.bias || !(choice[c] > kNone) ? choice[c] : s[c];
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
      for (int off = 1; off < (1 << sc.group_shift); off <<= 1) {
        const float o1 = __shfl_xor_sync(kAll, m1, off), o2 = __shfl_xor_sync(kAll, m2, off);
        m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
        m1 = fmaxf(m1, o1);
      }
      group = lane >> sc.group_shift;
      shift = sc.group_shift;
    } else {
      float* buf = reinterpret_cast<float*>(list + 1);
#pragma unroll
      for (int c = 0; c < kPL; ++c) {
        const int e = pl * lane + c;
        if (c < pl && e < E) buf[e] = sc.bias || !(choice[c] > kNone) ? choice[c] : s[c];
      }
      __syncwarp();
      if (lane < sc.n_group) {
        // each lane starts at another place of its run, so that runs of 32 do not meet in one bank
        int i = lane % size;
        for (int n = 0; n < size; ++n) {
          const float v = buf[lane * size + i];
          m2 = fmaxf(m2, fminf(m1, v));
          m1 = fmaxf(m1, v);
          if (++i == size) i = 0;
        }
      }
      group = lane;
      shift = 0;
    }
    mine = sc.group_top == 2 && m2 > kNone ? m1 + m2 : m1;
    int rank = 0;
    for (int g0 = 0; g0 < sc.n_group; g0 += 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = __shfl_sync(kAll, mine, (g0 + i) << shift);
        if (g0 + i < sc.n_group) rank += (v > mine || (v == mine && g0 + i < group)) ? 1 : 0;
      }
    }
    kept = __ballot_sync(kAll, group < sc.n_group && rank < sc.topk_group);
  }

  // keys: 0 for an expert that cannot be selected (a choice's key is never 0)
  uint32_t key[kPL];
  uint32_t lane_max = 0;
#pragma unroll
  for (int c = 0; c < kPL; ++c) {
    const int e = pl * lane + c;
    bool in = c < pl && e < E;
    if (sc.n_group > 1) in = in && ((kept >> (whole ? lane : (e * sc.group_inv) >> 20)) & 1u);
    key[c] = in ? topk_key(choice[c]) : 0u;
    lane_max = max(lane_max, key[c]);
  }
  int above = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) above += __shfl_sync(kAll, lane_max, j) > lane_max ? 1 : 0;
  const uint32_t theta = max(1u, __reduce_min_sync(kAll, above < k ? lane_max : kAll));

  int n = 0;
#pragma unroll
  for (int c = 0; c < kPL; ++c) {
    const bool is = key[c] >= theta;
    const uint32_t m = __ballot_sync(kAll, is);
    const int at = n + __popc(m & ((1u << lane) - 1u));
    if (is && at < kScoredList<kPL>) {
      list->key_e[at] = make_uint2(key[c], static_cast<uint32_t>(pl * lane + c));
      list->s[at] = s[c];
    }
    n += __popc(m);
  }
  if (n > 32 && n <= kScoredList<kPL>) {
    // as below, up to four candidates a lane; the selection goes to the list's front
    __syncwarp();
    constexpr int kEach = kScoredList<kPL> / 32;
    uint2 c[kEach];
    float cs[kEach];
    int cr[kEach];
#pragma unroll
    for (int h = 0; h < kEach; ++h) {
      const bool in = lane + 32 * h < n;
      c[h] = in ? list->key_e[lane + 32 * h] : make_uint2(0u, 0u);
      cs[h] = in ? list->s[lane + 32 * h] : 0.0f;
      cr[h] = in ? 0 : k;
    }
    for (int j = 0; j < n; ++j) {
      const uint2 o = list->key_e[j];
#pragma unroll
      for (int h = 0; h < kEach; ++h) cr[h] += (o.x > c[h].x || (o.x == c[h].x && o.y < c[h].y)) ? 1 : 0;
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < kEach; ++h) {
      if (cr[h] < k) {
        list->key_e[cr[h]] = c[h];
        list->s[cr[h]] = cs[h];
      }
    }
    n = k;
  } else if (n > 32) {
    // k rounds: the largest key, the lowest expert among equals
    uint32_t sel_e = 0;
    float sel_s = 0.0f;
    for (int j = 0; j < k; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int c = 0; c < kPL; ++c) best = max(best, key[c]);
      const uint32_t top = __reduce_max_sync(kAll, best);
      const int owner = __ffs(__ballot_sync(kAll, best == top)) - 1;  // the lowest lane holds the lowest experts
      uint32_t e = 0;
      float es = 0.0f;
      bool found = lane != owner;
#pragma unroll
      for (int c = 0; c < kPL; ++c) {
        if (!found && key[c] == top) {
          found = true;
          e = pl * lane + c;
          es = s[c];
          key[c] = 0;
        }
      }
      e = __shfl_sync(kAll, e, owner);
      es = __shfl_sync(kAll, es, owner);
      if (lane == j) sel_e = e, sel_s = es;
    }
    __syncwarp();
    if (lane < k) {
      list->key_e[lane] = make_uint2(static_cast<uint32_t>(32 - lane), sel_e);  // in order already
      list->s[lane] = sel_s;
    }
    n = k;
  }
  __syncwarp();
  const uint2 me = lane < n ? list->key_e[lane] : make_uint2(0u, 0u);
  float w = lane < n ? list->s[lane] : 0.0f;
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const uint2 o = list->key_e[j];
    rank += (o.x > me.x || (o.x == me.x && o.y < me.y)) ? 1 : 0;
  }
  const bool selected = lane < n && rank < k;
  if (!selected) w = 0.0f;
  if (sc.renormalize) {
    float sum = warp_sum(w);
    if (sum < 0x1p-64f) {  // up to where the approximate reciprocal holds; exact
      sum *= 0x1p100f;
      w *= 0x1p100f;
    }
    // A quotient by the reciprocal, corrected once by its residual (Markstein, 1990): a selection of one then has
    // weight 1 and equal scores have equal shares, exactly, as the sums of products that a rounding of Y to bf16 finds
    // halfway between two values need.  (An IEEE division took 0.3 us of a token's 4.1.)
    const float inv = __fdividef(1.0f, sum), q = w * inv;
    w = sum > 0.0f ? fmaf(fmaf(-q, sum, w), inv, q) : 0.0f;
  }
  if (selected) publish(rank, static_cast<int>(me.y), w * sc.scale);
  __syncwarp();  // the list may be written for the next row
  return ok;
}

}  // namespace bm
