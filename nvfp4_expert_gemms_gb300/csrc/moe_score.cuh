// One warp scores one token's experts and picks top_k of them (the rule is moe_router_t's in
// include/moe_gb300.h).
//
// Lanes own consecutive experts, group by group: with G = groups rounded up to a power of two, the
// 32 / G lanes of group g hold its S = E / groups experts, ceil(S / (32 / G)) each, in registers.  So
// lane order is expert order (a ballot's lowest lane is the lowest index of a tie), and a group's two
// largest values meet in log2(32 / G) shuffles.
//
// Which expert is chosen must not depend on rounding that another evaluation of the same formula
// would do otherwise: keys are the logits themselves or one correctly rounded sum of a score and its
// bias, a score is expf and one correctly rounded reciprocal, and a softmax's common denominator is
// left out of comparisons where it can be.
#pragma once
#include "moe_block.cuh"

namespace moe {

struct ScoreGeom {
  int S, lanes_log2, per;  // experts per group, log2 of lanes per group, experts per lane
  bool wide;               // a lane's logits are whole 16-byte pieces
};

// Order-preserving key: larger key = larger value, 0 = no candidate; -0 counts as +0, NaN as -inf.
__device__ __forceinline__ uint32_t order_key(float v) {
  v = isnan(v) ? -INFINITY : v == 0.f ? 0.f : v;
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float load_logit(const ScoreArgs& a, int64_t at) {
  float v;
  load_any<1>(a.logits, a.dtype, at, &v);
  return isnan(v) ? -INFINITY : v;
}

// 1 / (1 + e^-l), each step rounded once.
__device__ __forceinline__ float sigmoid_rn(float l) { return __frcp_rn(__fadd_rn(1.f, expf(-l))); }
// e^(l - m); 0 for an empty row (m = -inf)
__device__ __forceinline__ float exp_rn(float l, float m) { return m == -INFINITY ? 0.f : expf(__fsub_rn(l, m)); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Writes the token's top_k experts and weights; returns the lane's expert (lane < k).  VT >= g.per.
template <int VT>
__device__ __forceinline__ int score_token(const ScoreArgs& a, const ScoreGeom& g, int t, int k, int lane,
                                           int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  const int lanes = 1 << g.lanes_log2, grp = lane >> g.lanes_log2, sub = lane & (lanes - 1);
  const int e0 = grp * g.S + sub * g.per;
  const int cnt = grp < a.r.groups ? min(max(g.S - sub * g.per, 0), g.per) : 0;
  const int64_t row = (int64_t)t * a.ld;
  float l[VT];
  if (g.wide && VT % 4 == 0) {  // per == VT, every lane whole
#pragma unroll
    for (int i = 0; i < VT; i += 4) {
      const float4 q = cnt ? *(const float4*)((const float*)a.logits + row + e0 + i)
                           : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      l[i] = q.x;
      l[i + 1 < VT ? i + 1 : 0] = q.y;
      l[i + 2 < VT ? i + 2 : 0] = q.z;
      l[i + 3 < VT ? i + 3 : 0] = q.w;
    }
#pragma unroll
    for (int i = 0; i < VT; ++i) l[i] = isnan(l[i]) ? -INFINITY : l[i];
  } else {
#pragma unroll
    for (int i = 0; i < VT; ++i) l[i] = i < cnt ? load_logit(a, row + e0 + i) : -INFINITY;
  }
  const bool softmax = a.r.score == MOE_SCORE_SOFTMAX, biased = a.bias != nullptr;
  const bool two = a.r.groups > 1 && a.r.group_top == 2;
  float m = 0.f, den = 1.f;  // the row's maximum and sum of e^(l - m), where a score needs them
  if (softmax && (biased || two || !a.r.renormalize)) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < VT; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    if (biased || !a.r.renormalize) {
      den = 0.f;
#pragma unroll
      for (int i = 0; i < VT; ++i) den += exp_rn(l[i], m);
      den = warp_sum(den);
    }
  }
  uint32_t key[VT];
  float b1 = -INFINITY, b2 = -INFINITY;  // the lane's two largest group values
#pragma unroll
  for (int i = 0; i < VT; ++i) {
    float kv = l[i], gv = l[i];
    if (biased) {
      const float s = softmax ? (den > 0.f ? __fdiv_rn(exp_rn(l[i], m), den) : 0.f) : sigmoid_rn(l[i]);
      kv = gv = __fadd_rn(s, i < cnt ? a.bias[e0 + i] : 0.f);
    } else if (two) {
      gv = softmax ? exp_rn(l[i], m) : sigmoid_rn(l[i]);
    }
    key[i] = i < cnt ? order_key(kv) : 0u;
    gv = i < cnt && !isnan(gv) ? gv : -INFINITY;
    b2 = fmaxf(b2, fminf(b1, gv));
    b1 = fmaxf(b1, gv);
  }
  if (a.r.groups > 1) {
    for (int off = lanes >> 1; off > 0; off >>= 1) {
      const float o1 = __shfl_xor_sync(0xffffffffu, b1, off), o2 = __shfl_xor_sync(0xffffffffu, b2, off);
      b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
      b1 = fmaxf(b1, o1);
    }
    const uint32_t gk = order_key(two && g.S > 1 ? __fadd_rn(b1, b2) : b1);
    int better = 0;  // groups in front of this one
    for (int h = 0; h < a.r.groups; ++h) {
      const uint32_t o = __shfl_sync(0xffffffffu, gk, h << g.lanes_log2);
      better += o > gk || (o == gk && h < grp);
    }
    if (better >= a.r.top_groups)
#pragma unroll
      for (int i = 0; i < VT; ++i) key[i] = 0u;
  }
  int mine = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t bk = key[0];
    int be = 0;
#pragma unroll
    for (int i = 1; i < VT; ++i)
      if (key[i] > bk) {
        bk = key[i];
        be = i;
      }
    const uint32_t wk = __reduce_max_sync(0xffffffffu, bk);
    const int wl = __ffs(__ballot_sync(0xffffffffu, bk == wk)) - 1;
    const int we = __shfl_sync(0xffffffffu, e0 + be, wl);
#pragma unroll
    for (int i = 0; i < VT; ++i)
      if (lane == wl && i == be) key[i] = 0u;  // taken
    if (lane == j) mine = we;
  }
  float s = 0.f;
  if (softmax && a.r.renormalize) {
    const float ls = lane < k ? load_logit(a, row + mine) : -INFINITY;
    const float ms = warp_max(ls);
    s = lane < k ? exp_rn(ls, ms) : 0.f;
  } else if (lane < k) {
    const float ls = load_logit(a, row + mine);
    s = softmax ? (den > 0.f ? exp_rn(ls, m) / den : 0.f) : sigmoid_rn(ls);
  }
  if (a.r.renormalize) {
    float tot = s;
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, off);
    s = tot == 0.f ? 0.f : s / tot;
  }
  if (lane < k) {
    topk_idx[(int64_t)t * k + lane] = mine;
    topk_w[(int64_t)t * k + lane] = s * a.r.scale;
  }
  return mine;
}

inline ScoreGeom score_geom(const ScoreArgs& a, int E) {
  ScoreGeom g;
  int G = 1, lg = 5;
  while (G < a.r.groups) {
    G *= 2;
    --lg;
  }
  g.S = E / a.r.groups;
  g.lanes_log2 = lg;
  g.per = (g.S + (1 << lg) - 1) >> lg;
  g.wide = a.dtype == MOE_DT_F32 && g.per % 4 == 0 && (g.per & (g.per - 1)) == 0 && g.S == g.per << lg &&
           a.ld % 4 == 0 && (uintptr_t)a.logits % 16 == 0;
  return g;
}

}  // namespace moe
