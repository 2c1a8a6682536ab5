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
  bool wide;               // a lane's logits are whole aligned 8- or 16-byte pieces; so is its share of the bias
};

// A candidate's place while a warp sorts out the best ones.
struct ScoreCand {
  float key;
  int expert;
};
constexpr float kNoKey = __builtin_nanf("");  // not a candidate: compares false with everything, loses every max

__device__ __forceinline__ float load_logit(const ScoreArgs& a, int64_t at) {
  float v;
  load_any<1>(a.logits, a.dtype, at, &v);
  return fmaxf(v, -INFINITY);  // NaN counts as -infinity
}

// Largest value over the warp; NaNs do not count (NaN if there is nothing else).
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// 1 / (1 + e^-l), each step rounded once.
__device__ __forceinline__ float sigmoid_rn(float l) { return __frcp_rn(__fadd_rn(1.f, expf(-l))); }
// e^(l - m); 0 for an empty row (m = -inf)
__device__ __forceinline__ float exp_rn(float l, float m) { return m == -INFINITY ? 0.f : expf(__fsub_rn(l, m)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The experts e0 .. e0 + cnt - 1 of a lane, their logits as fp32 (NaN as -infinity; -infinity past cnt).
template <int VT>
__device__ __forceinline__ void load_logits(const ScoreArgs& a, const ScoreGeom& g, int64_t at, int cnt, float (&l)[VT]) {
  if (a.dtype == MOE_DT_F32) {
    const float* p = (const float*)a.logits + at;
    if (VT >= 4 && g.wide) {
#pragma unroll
      for (int i = 0; i < VT / 4; ++i) {
        const float4 q = cnt ? ((const float4*)p)[i] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        l[4 * i] = q.x;
        l[(4 * i + 1) % VT] = q.y;
        l[(4 * i + 2) % VT] = q.z;
        l[(4 * i + 3) % VT] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VT; ++i) l[i] = i < cnt ? p[i] : -INFINITY;
    }
  } else {
    const uint16_t* p = (const uint16_t*)a.logits + at;
    uint32_t w[VT];
    if (VT >= 4 && g.wide) {
#pragma unroll
      for (int i = 0; i < VT / 4; ++i) {
        const uint2 q = cnt ? ((const uint2*)p)[i] : make_uint2(0, 0);
        w[4 * i] = q.x & 0xFFFFu;
        w[(4 * i + 1) % VT] = q.x >> 16;
        w[(4 * i + 2) % VT] = q.y & 0xFFFFu;
        w[(4 * i + 3) % VT] = q.y >> 16;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VT; ++i) w[i] = i < cnt ? p[i] : 0u;
    }
    if (a.dtype == MOE_DT_BF16) {
#pragma unroll
      for (int i = 0; i < VT; ++i) l[i] = i < cnt ? __uint_as_float(w[i] << 16) : -INFINITY;
    } else {
#pragma unroll
      for (int i = 0; i < VT; ++i) l[i] = i < cnt ? __half2float(__ushort_as_half((unsigned short)w[i])) : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < VT; ++i) l[i] = fmaxf(l[i], -INFINITY);
}

// The experts of the k largest keys, in descending order, ties to the lower expert: returned in lanes
// 0 .. k-1.  Lane order is expert order.
//
// Of the lanes' own maxima, the k-th largest bounds the k-th largest key from below, so only keys at
// least that large can be chosen: about k of them.  They move to one lane each and a lane counts how many
// stand in front of its own -- a few instructions per candidate in place of k rounds over every key.
//
// SURE: key holds the keys, and there is always an answer (more than 32 keys at the bound, which takes
// many equal ones, go through k rounds after all).  Else key holds estimates, each at most slack(estimate)
// off: the candidates are those that could be chosen, final_key(l, expert) gives a candidate's key from
// val, the logits, and false is returned where that does not decide.
__device__ __forceinline__ float key_slack(float key) { return 9.6e-7f + 2.4e-7f * fabsf(key); }

template <bool SURE, int VT, class FinalKey>
__device__ __forceinline__ bool pick_top(float (&key)[VT], const float (&val)[VT], int e0, int k, int lane,
                                         ScoreCand* cand, FinalKey final_key, int& chosen) {
  if constexpr (VT >= 4) {
    float rem = key[0], bound = 0.f;
#pragma unroll
    for (int i = 1; i < VT; ++i) rem = fmaxf(rem, key[i]);
    for (int j = 0; j < k; ++j) {  // equal maxima leave together: the bound is then a little lower
      bound = redux_max(rem);
      rem = rem == bound ? kNoKey : rem;
    }
    bound = fmaxf(bound, -INFINITY);  // NaN, fewer than k lanes with candidates: every candidate
    if (!SURE) {
      if (isinf(bound)) return false;
      bound -= 2.f * key_slack(bound);
    }
    int c = 0;
#pragma unroll
    for (int i = 0; i < VT; ++i) c += key[i] >= bound;
    int incl = c;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    if (total <= 32) {
      ScoreCand* to = cand + incl - c;
#pragma unroll
      for (int i = 0; i < VT; ++i)
        if (key[i] >= bound) *to++ = ScoreCand{SURE ? key[i] : val[i], e0 + i};
      __syncwarp();
      ScoreCand mine = lane < total ? cand[lane] : ScoreCand{kNoKey, 0};
      if (!SURE && lane < total) mine.key = final_key(mine.key, mine.expert);
      int front = 0;
#pragma unroll 4
      for (int j = 0; j < total; ++j) {
        const float o = __shfl_sync(0xffffffffu, mine.key, j);
        front += j < lane ? o >= mine.key : o > mine.key;
      }
      if (lane < total && front < k) cand[32 + front].expert = mine.expert;
      __syncwarp();
      chosen = cand[32 + (lane < k ? lane : 0)].expert;
      __syncwarp();
      return true;
    }
    if (!SURE) return false;
  }
  for (int j = 0; j < k; ++j) {
    float bk = key[0];
    int be = 0;
#pragma unroll
    for (int i = 1; i < VT; ++i) {
      const bool up = key[i] > bk || (isnan(bk) && !isnan(key[i]));
      bk = up ? key[i] : bk;
      be = up ? i : be;
    }
    const float m = redux_max(bk);
    const int wl = __ffs(__ballot_sync(0xffffffffu, bk == m)) - 1;
    const int we = __shfl_sync(0xffffffffu, e0 + be, wl);
#pragma unroll
    for (int i = 0; i < VT; ++i)
      if (lane == wl && i == be) key[i] = kNoKey;  // taken
    if (lane == j) chosen = we;
  }
  return true;
}

// A group's value from its lanes' two largest (in every lane of the group): their sum, or the largest.
__device__ __forceinline__ float group_value(float b1, float b2, int lanes, bool both) {
  for (int off = lanes >> 1; off > 0; off >>= 1) {
    const float o1 = __shfl_xor_sync(0xffffffffu, b1, off), o2 = __shfl_xor_sync(0xffffffffu, b2, off);
    b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
    b1 = fmaxf(b1, o1);
  }
  return fmaxf(both ? __fadd_rn(b1, b2) : b1, -INFINITY);
}

// Writes the token's top_k experts and weights; returns the lane's expert (lane < k).  VT >= g.per; cand:
// 64 entries of shared memory for this warp.
template <int VT>
__device__ __forceinline__ int score_token(const ScoreArgs& a, const ScoreGeom& g, int t, int k, int lane,
                                           int32_t* __restrict__ topk_idx, float* __restrict__ topk_w, ScoreCand* cand) {
  const int lanes = 1 << g.lanes_log2, grp = lane >> g.lanes_log2, sub = lane & (lanes - 1);
  const int e0 = grp * g.S + sub * g.per;
  const int cnt = grp < a.r.groups ? min(max(g.S - sub * g.per, 0), g.per) : 0;
  const int64_t row = (int64_t)t * a.ld;
  const bool softmax = a.r.score == MOE_SCORE_SOFTMAX, biased = a.bias != nullptr;
  const bool two = a.r.groups > 1 && a.r.group_top == 2;
  float l[VT], bv[VT];
  load_logits<VT>(a, g, row + e0, cnt, l);
  if (biased) {
    if (VT >= 4 && g.wide) {
#pragma unroll
      for (int i = 0; i < VT / 4; ++i) {
        const float4 q = cnt ? ((const float4*)(a.bias + e0))[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        bv[4 * i] = q.x;
        bv[(4 * i + 1) % VT] = q.y;
        bv[(4 * i + 2) % VT] = q.z;
        bv[(4 * i + 3) % VT] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VT; ++i) bv[i] = i < cnt ? a.bias[e0 + i] : 0.f;
    }
  }
  float m = 0.f, den = 1.f;  // the row's maximum and sum of e^(l - m), where a score needs them
  if (softmax && (biased || two || !a.r.renormalize)) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < VT; ++i) m = fmaxf(m, l[i]);
    m = redux_max(m);
    if (biased || !a.r.renormalize) {
      den = 0.f;
#pragma unroll
      for (int i = 0; i < VT; ++i) den += exp_rn(l[i], m);
      den = warp_sum(den);
    }
  }
  int mine = 0;
  bool done = false;
  if constexpr (VT >= 4) {
    // Sigmoid keys with a bias: the fast exponential and division place every key to within key_slack
    // (__expf: 2 + 1.173 |l| units, less than 1e-7 of the score after its slope; the division 2 units;
    // the sum's rounding), which leaves few experts that could be chosen, and only those get their exact
    // key.  Where groups or keys stand closer than that, everything is done exactly below.
    if (biased && !softmax) {
      float est[VT], b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < VT; ++i) {
        const float v = __fdividef(1.f, 1.f + __expf(-l[i])) + bv[i];
        est[i] = i < cnt ? fmaxf(v, -INFINITY) : kNoKey;
      }
      bool clear = true;
      if (a.r.groups > 1) {
#pragma unroll
        for (int i = 0; i < VT; ++i) {
          const float s = fmaxf(est[i], -INFINITY);
          b2 = fmaxf(b2, fminf(b1, s));
          b1 = fmaxf(b1, s);
        }
        const bool both = two && g.S > 1;
        const float gv = group_value(b1, b2, lanes, both);
        const float gap = 4.f * key_slack(gv), hi = gv + gap, lo = gv - gap;
        int front = 0, near = 0;  // groups surely in front, and those that may be
        for (int h = 0; h < a.r.groups; ++h) {
          const float o = __shfl_sync(0xffffffffu, gv, h << g.lanes_log2);
          front += o > hi;
          near += o >= lo;
        }
        // itself counts among the near ones
        clear = grp >= a.r.groups || (!isinf(gv) && (front < a.r.top_groups) == (near - 1 < a.r.top_groups));
        if (front >= a.r.top_groups)
#pragma unroll
          for (int i = 0; i < VT; ++i) est[i] = kNoKey;
      }
      if (__all_sync(0xffffffffu, clear))
        done = pick_top<false, VT>(est, l, e0, k, lane, cand,
                                   [&](float lv, int e) { return fmaxf(__fadd_rn(sigmoid_rn(lv), a.bias[e]), -INFINITY); },
                                   mine);
    }
  }
  if (!done) {
    float key[VT];
    if (biased) {
#pragma unroll
      for (int i = 0; i < VT; ++i) {
        const float s = softmax ? (den > 0.f ? __fdiv_rn(exp_rn(l[i], m), den) : 0.f) : sigmoid_rn(l[i]);
        key[i] = i < cnt ? fmaxf(__fadd_rn(s, bv[i]), -INFINITY) : kNoKey;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VT; ++i) key[i] = i < cnt ? l[i] : kNoKey;
    }
    if (a.r.groups > 1) {
      float b1 = -INFINITY, b2 = -INFINITY;  // the lane's two largest group values
      if (!biased && two) {
#pragma unroll
        for (int i = 0; i < VT; ++i) {
          const float s = i < cnt ? (softmax ? exp_rn(l[i], m) : sigmoid_rn(l[i])) : -INFINITY;
          b2 = fmaxf(b2, fminf(b1, s));
          b1 = fmaxf(b1, s);
        }
      } else {
#pragma unroll
        for (int i = 0; i < VT; ++i) {
          const float s = fmaxf(key[i], -INFINITY);
          b2 = fmaxf(b2, fminf(b1, s));
          b1 = fmaxf(b1, s);
        }
      }
      const float gv = group_value(b1, b2, lanes, two && g.S > 1);
      int front = 0;  // groups in front of this one
      for (int h = 0; h < a.r.groups; ++h) {
        const float o = __shfl_sync(0xffffffffu, gv, h << g.lanes_log2);
        front += o > gv || (o == gv && h < grp);
      }
      if (front >= a.r.top_groups)
#pragma unroll
        for (int i = 0; i < VT; ++i) key[i] = kNoKey;
    }
    pick_top<true, VT>(key, l, e0, k, lane, cand, [](float v, int) { return v; }, mine);
  }
  float s = 0.f;
  if (softmax && a.r.renormalize) {
    const float ls = lane < k ? load_logit(a, row + mine) : -INFINITY;
    const float ms = redux_max(ls);
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
  g.wide = g.per % 4 == 0 && (g.per & (g.per - 1)) == 0 && g.S == g.per << lg && a.ld % 4 == 0 &&
           (uintptr_t)a.logits % (4 * dtype_size(a.dtype)) == 0 && (uintptr_t)a.bias % 16 == 0;
  return g;
}

}  // namespace moe
