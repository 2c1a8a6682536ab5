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
//
// Bound: instructions (some 640 per token at 256 experts, sigmoid, bias, 8 groups; 70% of issue slots): 16384
// tokens 12.4 us, 2.7 by HBM.  By k rounds over all keys, every score exact, it took 22.5.
#pragma once
#include "moe_block.cuh"

namespace moe {

struct ScoreGeom {
  int S, lanes_log2, per;  // experts per group, log2 of lanes per group, experts per lane
  bool wide;               // a lane's logits are whole aligned 8- or 16-byte pieces; so is its share of the bias
  bool full;               // and every lane has its VT experts
};

// What a warp keeps in shared memory while it sorts out the best ones.
struct ScoreScratch {
  int cand[32];    // experts that could be chosen, and (few experts per lane) their logits
  float logit[32];
  int expert[8];   // the chosen, in order, and their scores
  float score[8];
};
constexpr float kNoKey = __builtin_nanf("");  // not a candidate: compares false with everything, loses every max

__device__ __forceinline__ float load_logit(const ScoreArgs& a, int64_t at) {
  return fmaxf(load_any(a.logits, a.dtype, at), -INFINITY);  // NaN counts as -infinity
}

// Largest value over the warp; NaNs do not count (NaN if there is nothing else).
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// 1 / (1 + e^-l), each step rounded once.
__device__ __forceinline__ float sigmoid_rn(float l) { return __frcp_rn(__fadd_rn(1.f, expf(-l))); }
// The same to within 3e-7 (see score_token), in five instructions: what is subnormal on the way counts as zero.
__device__ __forceinline__ float sigmoid_fast(float l) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}
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
        const float4 q = g.full || cnt ? ((const float4*)p)[i] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
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

// How far an estimated key may be off (see score_token).
__device__ __forceinline__ float key_slack(float key) { return 9.6e-7f + 2.4e-7f * fabsf(key); }

// A lane's largest key (kNoKey: it has none) and, where asked, its second (-infinity: it has none).  FULL: every
// key is one.
template <bool FULL, int VT>
__device__ __forceinline__ float lane_top(const float (&key)[VT], int cnt, bool second, float& b2) {
  const auto value = [](float v) { return FULL ? v : fmaxf(v, -INFINITY); };
  float hi = key[0];
  if (!second) {
#pragma unroll
    for (int i = 1; i < VT; ++i) hi = fmaxf(hi, key[i]);
    return hi;
  }
  b2 = -INFINITY;
  hi = value(hi);
#pragma unroll
  for (int i = 1; i < VT; i += 2) {  // a pair, and with it the two best so far
    const float u = value(key[i]), w = i + 1 < VT ? value(key[i + 1 < VT ? i + 1 : i]) : -INFINITY;
    const float p = fmaxf(u, w);
    b2 = fmaxf(fmaxf(b2, fminf(u, w)), fminf(hi, p));
    hi = fmaxf(hi, p);
  }
  return FULL || cnt > 0 ? hi : kNoKey;
}

// The value of a lane's group, in every lane of the group, from its lanes' largest and second keys: their
// sum, or the largest.  reach: how far it may be off where the keys are estimates, which goes by the keys' sizes and
// not by the sum's, where they cancel.
__device__ __forceinline__ float group_value(float b1, float b2, int lanes, bool both, float& reach) {
  b1 = fmaxf(b1, -INFINITY);
  for (int off = lanes >> 1; off > 0; off >>= 1) {
    const float o1 = __shfl_xor_sync(0xffffffffu, b1, off);
    if (both) {
      const float o2 = __shfl_xor_sync(0xffffffffu, b2, off);
      b2 = fmaxf(fmaxf(fminf(b1, o1), b2), o2);
    }
    b1 = fmaxf(b1, o1);
  }
  reach = key_slack(b1) + (both ? key_slack(b2) : 0.f);
  return fmaxf(both ? __fadd_rn(b1, b2) : b1, -INFINITY);
}

// The experts of the k largest keys, in descending order, ties to the lower expert, and their scores:
// returned in lanes 0 .. k-1.  Lane order is expert order.
//
// Of the lanes' own maxima (`top`; kNoKey: the lane has no candidate), the k-th largest bounds the k-th
// largest key from below, so only keys at least that large can be chosen: about k of them.  They move to
// one lane each, which computes its candidate's key and counts how many stand in front of it -- a few
// instructions per candidate in place of k rounds over every key.  key holds the keys, or (slack) values
// that are at most key_slack off.  False where that leaves more than 32, or a bound without slack.
template <int VT, class KeyOf>
__device__ __forceinline__ bool pick_top(const float (&key)[VT], const float (&l)[VT], float top, bool slack, int e0, int k, int lane,
                                         ScoreScratch& sc, KeyOf key_of, int& chosen, float& score) {
  float bound = 0.f, rem = top;
#pragma unroll 4
  for (int j = 0; j < k; ++j) {  // equal maxima leave together: the bound is then a little lower
    bound = redux_max(rem);
    rem = rem == bound ? kNoKey : rem;
  }
  bound = fmaxf(bound, -INFINITY);  // NaN, fewer than k lanes with candidates: every candidate
  if (slack) {
    if (bound == INFINITY) return false;
    bound -= 2.f * key_slack(bound);  // -infinity stays
  }
  uint32_t mask = 0;
  if (!isnan(top)) {
#pragma unroll
    for (int i = 0; i < VT; ++i) mask |= key[i] >= bound ? 1u << i : 0u;
  }
  const int c = __popc(mask);
  int incl = c;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  const int total = __shfl_sync(0xffffffffu, incl, 31);
  if (total > 32) return false;
  int at = incl - c;
  if constexpr (VT <= 4) {
#pragma unroll
    for (int i = 0; i < VT; ++i)
      if (mask >> i & 1) {
        sc.cand[at] = e0 + i;
        sc.logit[at++] = l[i];
      }
  } else {  // the logit is read again: cheaper than picking it out of VT registers
    for (; mask; mask &= mask - 1) sc.cand[at++] = e0 + __ffs(mask) - 1;
  }
  __syncwarp();
  const int e = sc.cand[lane < total ? lane : 0];
  float sv;
  const float mine = key_of(e, VT <= 4 ? sc.logit[lane < total ? lane : 0] : kNoKey, sv);
  int front = 0;
#pragma unroll 4
  for (int j = 0; j < total; ++j) {
    const float o = __shfl_sync(0xffffffffu, mine, j);
    front += j < lane ? o >= mine : o > mine;
  }
  if (lane < total && front < k) {
    sc.expert[front] = e;
    sc.score[front] = sv;
  }
  __syncwarp();
  chosen = sc.expert[lane & 7];
  score = sc.score[lane & 7];
  __syncwarp();
  return true;
}

// The same by k rounds over every key: few keys per lane, or very many equal ones.
template <int VT>
__device__ __forceinline__ int pick_by_rounds(float (&key)[VT], int e0, int k, int lane) {
  int chosen = 0;
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
  return chosen;
}

// Writes the token's top_k experts and weights; returns the lane's expert (lane < k).  VT >= g.per; sc:
// this warp's.
template <int VT>
__device__ __forceinline__ int score_token(const ScoreArgs& a, const ScoreGeom& g, int t, int k, int lane,
                                           int32_t* __restrict__ topk_idx, float* __restrict__ topk_w, ScoreScratch& sc) {
  const int lanes = 1 << g.lanes_log2, grp = lane >> g.lanes_log2, sub = lane & (lanes - 1);
  const int e0 = grp * g.S + sub * g.per;
  const int cnt = g.full ? VT : grp < a.r.groups ? min(max(g.S - sub * g.per, 0), g.per) : 0;
  const int64_t row = (int64_t)t * a.ld;
  const bool softmax = a.r.score == MOE_SCORE_SOFTMAX, biased = a.bias != nullptr;
  const bool grouped = a.r.groups > 1, two = grouped && a.r.group_top == 2 && g.S > 1;
  float l[VT];
  load_logits<VT>(a, g, row + e0, cnt, l);
  float m = 0.f, den = 1.f;  // the row's maximum and sum of e^(l - m), where a score needs them
  if (softmax && (biased || two || !a.r.renormalize)) {
    float none;
    m = redux_max(lane_top<false, VT>(l, cnt, false, none));
    if (biased || !a.r.renormalize) {
      den = 0.f;
#pragma unroll
      for (int i = 0; i < VT; ++i) den += exp_rn(l[i], m);
      den = warp_sum(den);
    }
  }
  // a logit's softmax: 0 in an empty row, NaN in one with a +inf logit
  auto softmax_of = [&](float v) { return den == 0.f ? 0.f : __fdiv_rn(exp_rn(v, m), den); };
  // expert e's key (known: its logit, with few experts per lane); sv: its sigmoid score, or its logit where the score is a softmax's
  auto key_of = [&](int e, float known, float& sv) {
    const float lv = VT <= 4 ? known : load_logit(a, row + e);
    sv = softmax ? lv : sigmoid_rn(lv);
    if (!biased) return lv;
    const float s = softmax ? softmax_of(lv) : sv;
    return fmaxf(__fadd_rn(s, a.bias[e]), -INFINITY);
  };
  int mine = 0;
  float sv = 0.f, b2 = -INFINITY;
  bool done = false;
  if constexpr (VT >= 4) {
    // Sigmoid keys with a bias: the fast exponential and reciprocal place every key to within key_slack
    // (the power of two 2^-22 and 2^-23 |l|, the rounded product with its constant, relative, which the sigmoid's
    // slope s (1 - s) <= 1/4, |l| s (1 - s) < 0.23, makes less than 1e-7 of the score; the sum and the reciprocal
    // 2^-24 and 2^-23; the key's own rounding), which leaves few experts that could be chosen, and only those get
    // their exact key.  Where groups or keys stand closer than that, everything is done exactly below.
    if (biased && !softmax) {
      float est[VT];
      if (g.full) {
#pragma unroll
        for (int i = 0; i < VT / 4; ++i) {
          const float4 q = ((const float4*)(a.bias + e0))[i];
          est[4 * i] = q.x;
          est[4 * i + 1] = q.y;
          est[4 * i + 2] = q.z;
          est[4 * i + 3] = q.w;
        }
#pragma unroll
        for (int i = 0; i < VT; ++i) est[i] = fmaxf(sigmoid_fast(l[i]) + est[i], -INFINITY);
      } else {
#pragma unroll
        for (int i = 0; i < VT; ++i) est[i] = i < cnt ? a.bias[e0 + i] : 0.f;
#pragma unroll
        for (int i = 0; i < VT; ++i)
          est[i] = i < cnt ? fmaxf(sigmoid_fast(l[i]) + est[i], -INFINITY) : kNoKey;
      }
      float top = g.full ? lane_top<true, VT>(est, cnt, two, b2) : lane_top<false, VT>(est, cnt, two, b2);
      bool clear = true;
      if (grouped) {
        float reach;
        const float gv = group_value(top, b2, lanes, two, reach);
        float bound = 0.f, rem = grp < a.r.groups ? gv : kNoKey;
#pragma unroll 4
        for (int j = 0; j < a.r.top_groups; ++j) {
          bound = redux_max(rem);
          rem = rem == bound ? kNoKey : rem;
        }
        // the last group kept, and no other within reach of it (-infinity is no estimate, and far from any other)
        const float gap = reach + redux_max(gv == bound ? reach : kNoKey);
        const uint32_t near = __ballot_sync(0xffffffffu, grp < a.r.groups && gv > -INFINITY && fabsf(gv - bound) <= gap);
        const uint32_t kept = __ballot_sync(0xffffffffu, grp < a.r.groups && gv >= bound);
        clear = __popc(near) == lanes && __popc(kept) == lanes * a.r.top_groups && !isinf(bound);
        if (!(gv >= bound)) top = kNoKey;
      }
      if (clear) done = pick_top<VT>(est, l, top, true, e0, k, lane, sc, key_of, mine, sv);
    }
  }
  if (!done) {
    float key[VT];
    if (biased) {
#pragma unroll
      for (int i = 0; i < VT; ++i) {
        const float s = softmax ? softmax_of(l[i]) : sigmoid_rn(l[i]);
        key[i] = i < cnt ? fmaxf(__fadd_rn(s, a.bias[e0 + i]), -INFINITY) : kNoKey;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VT; ++i) key[i] = i < cnt ? l[i] : kNoKey;
    }
    b2 = -INFINITY;
    float top = lane_top<false, VT>(key, cnt, two, b2);
    if (grouped) {
      float g1 = top;
      if (two && !biased) {  // scores in place of logits, whose order they have
        const bool none = softmax && m == INFINITY;  // softmax's scores are all NaN
        g1 = isnan(top) || none ? -INFINITY : softmax ? exp_rn(top, m) : sigmoid_rn(top);
        b2 = cnt < 2 || none ? -INFINITY : softmax ? exp_rn(b2, m) : sigmoid_rn(b2);
      }
      float reach;  // unused: the keys are exact
      const float gv = group_value(g1, b2, lanes, two, reach);
      int front = 0;  // groups in front of this one
      for (int h = 0; h < a.r.groups; ++h) {
        const float o = __shfl_sync(0xffffffffu, gv, h << g.lanes_log2);
        front += o > gv || (o == gv && h < grp);
      }
      if (front >= a.r.top_groups) {
        top = kNoKey;
#pragma unroll
        for (int i = 0; i < VT; ++i) key[i] = kNoKey;
      }
    }
    if constexpr (VT >= 4)
      done = pick_top<VT>(key, l, top, false, e0, k, lane, sc, key_of, mine, sv);
    if (!done) {
      mine = pick_by_rounds<VT>(key, e0, k, lane);
      if (lane < k) {
        sv = load_logit(a, row + mine);
        if (!softmax) sv = sigmoid_rn(sv);
      }
    }
  }
  float s = lane < k ? sv : 0.f;
  if (softmax) {
    const float ms = a.r.renormalize ? redux_max(lane < k ? sv : -INFINITY) : m;
    s = lane < k ? exp_rn(sv, ms) : 0.f;
    if (!a.r.renormalize) s = den == 0.f ? 0.f : s / den;
    if (m == INFINITY) s = kNoKey;  // no score of the row is a number, whichever are chosen
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
  g.full = g.wide && G == a.r.groups;
  return g;
}

}  // namespace moe
