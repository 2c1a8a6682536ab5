// A whole mixture-of-experts layer for a few tokens (moe_layer_few): argument checks and the router's product.
#include "moe_few.cuh"
#include "moe_formats.cuh"

namespace moe {

namespace {

// A sum kept as an unevaluated pair of fp32 numbers, hi + lo: adding v loses nothing of hi + v (the rounding error of
// a sum is itself a number that fp32 holds, found by subtracting what was added), and lo collects what hi lost.
struct Pair {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b)));
    hi = s;
  }
  __device__ __forceinline__ void add_product(float a, float b) {
    const float p = __fmul_rn(a, b);
    lo = __fadd_rn(lo, __fmaf_rn(a, b, -p));  // 0 where both are bf16
    add(p);
  }
  __device__ __forceinline__ void add(const Pair& o) {
    lo = __fadd_rn(lo, o.lo);
    add(o.hi);
  }
  // the sum rounded once; past fp32's range lo is not a number and hi alone counts
  __device__ __forceinline__ float rounded() const { return isfinite(hi) ? __fadd_rn(hi, lo) : hi; }
};

constexpr int kRouterThreads = 256;
constexpr int kRouterTokens = 4;  // tokens per pass over an expert's row

// logits[t, e] = sum over h of x[t, h] w[e, h], one block per expert.  The sum is carried in pairs, so that it is the
// exact sum rounded once (but for one case in some 2^20): which experts a token gets must not hang on the order of a
// sum.
__global__ void __launch_bounds__(kRouterThreads) few_router_kernel(const FewArgs a) {
  __shared__ Pair part[kRouterThreads / 32][kRouterTokens];
  const int e = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H = a.d.H;
  pdl_wait();
  pdl_trigger();
  if (e == 0 && threadIdx.x == 0) a.status[0] = 0;
  for (int t0 = 0; t0 < a.T; t0 += kRouterTokens) {
    const int nt = min(kRouterTokens, a.T - t0);
    Pair acc[kRouterTokens];
    for (int i = threadIdx.x; i < H; i += kRouterThreads) {
      const float w = load_any(a.wr, a.w_dtype, e * a.ldw + i);
#pragma unroll
      for (int t = 0; t < kRouterTokens; ++t)
        if (t < nt) acc[t].add_product(__bfloat162float(a.x[(t0 + t) * a.ldx + i]), w);
    }
#pragma unroll
    for (int t = 0; t < kRouterTokens; ++t) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        Pair o;
        o.hi = __shfl_xor_sync(0xffffffffu, acc[t].hi, off);
        o.lo = __shfl_xor_sync(0xffffffffu, acc[t].lo, off);
        acc[t].add(o);
      }
      if (lane == 0) part[warp][t] = acc[t];
    }
    __syncthreads();
    if (threadIdx.x < nt) {
      Pair s = part[0][threadIdx.x];
      for (int w = 1; w < kRouterThreads / 32; ++w) s.add(part[w][threadIdx.x]);
      a.logits[(t0 + threadIdx.x) * a.d.E + e] = s.rounded();
    }
    __syncthreads();
  }
}

// One weight, dequantized: element (n, k) of expert e's gate/up (which = 0) or down matrix.
__device__ float weight_at(const FewArgs& a, int which, int e, int n, int k) {
  const int N = which ? a.d.H : 2 * a.d.I, K = which ? a.d.I : a.d.H;
  const char* A = a.packed + a.d.offset[which ? MOE_T_D_A : MOE_T_GU_A];
  const char* B = a.packed + a.d.offset[which ? MOE_T_D_B : MOE_T_GU_B];
  const size_t at = ((size_t)e * N + n) * K + k;
  switch (a.d.fmt) {
    case MOE_FMT_BF16:
      return bf16_to_f32(((const uint16_t*)A)[at]);
    case MOE_FMT_FP8_B128_W8A16:
    case MOE_FMT_FP8_B128_W8A8:
      return e4m3_to_f32(((const uint8_t*)A)[at]) * ((const float*)B)[((size_t)e * (N / 128) + n / 128) * (K / 128) + k / 128];
    case MOE_FMT_INT4_G128_W4A16: {
      const uint32_t w = ((const uint32_t*)A)[((size_t)e * (K / 8) + k / 8) * N + n];
      return ((int)((w >> (4 * (k % 8))) & 15u) - 8) * __half2float(((const __half*)B)[((size_t)e * (K / 128) + k / 128) * N + n]);
    }
    default: {
      const uint8_t c = ((const uint8_t*)A)[at / 2];
      const float gs = ((const float*)(a.packed + a.d.offset[which ? MOE_T_D_GS : MOE_T_GU_GS]))[e];
      return e2m1_to_f32(k & 1 ? c >> 4 : c & 15) * e4m3_to_f32(((const uint8_t*)B)[at / 16]) / gs;
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// One warp per (slot, feature).
__global__ void few_gate_up_kernel(const FewArgs a) {
  pdl_wait();
  pdl_trigger();
  const int f = blockIdx.x * 8 + (threadIdx.x >> 5), r = blockIdx.y, lane = threadIdx.x & 31;
  if (f >= a.d.I) return;
  const int e = a.idx[r];
  float g = 0.f, u = 0.f;
  for (int k = lane; k < a.d.H; k += 32) {
    const float xv = __bfloat162float(a.x[(r / a.k) * a.ldx + k]);
    g = fmaf(weight_at(a, 0, e, f, k), xv, g);
    u = fmaf(weight_at(a, 0, e, a.d.I + f, k), xv, u);
  }
  g = warp_sum(g);
  u = warp_sum(u);
  if (lane == 0) a.h[(size_t)r * a.d.I + f] = g / (1.f + expf(-g)) * u;
}

// One warp per (token, feature).
__global__ void few_down_kernel(const FewArgs a) {
  pdl_wait();
  pdl_trigger();
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5), t = blockIdx.y, lane = threadIdx.x & 31;
  float y = 0.f;
  for (int j = 0; j < a.k; ++j) {
    const int r = t * a.k + j, e = a.idx[r];
    float s = 0.f;
    for (int k = lane; k < a.d.I; k += 32) s = fmaf(weight_at(a, 1, e, n, k), a.h[(size_t)r * a.d.I + k], s);
    y = fmaf(a.wt[r], warp_sum(s), y);
  }
  if (lane == 0) a.out[t * a.ldo + n] = __float2bfloat16_rn(y);
}

}  // namespace

FewLayout few_layout(const moe_packed_desc_t& d, int T, int k) {
  FewLayout L;
  size_t cur = 0;
  auto take = [&](size_t bytes) {
    const size_t o = cur;
    cur += (bytes + 255) / 256 * 256;
    return o;
  };
  const size_t R = (size_t)T * k;
  L.status = take(256);
  L.idx = take(4 * R);
  L.wt = take(4 * R);
  L.logits = take(4 * (size_t)T * d.E);
  L.h = take(4 * R * d.I);
  L.total = cur;
  return L;
}

cudaError_t launch_few(const FewArgs& a, const ScoreArgs& r, int32_t* idx, float* wt, cudaStream_t s) {
  note_launches(3);
  cudaError_t e = launch_pdl(few_router_kernel, dim3(a.d.E), dim3(kRouterThreads), 0, s, a);
  if (e == cudaSuccess) e = launch_route_scored(r, a.T, a.d.E, a.k, idx, wt, s);
  if (e == cudaSuccess) e = launch_pdl(few_gate_up_kernel, dim3((a.d.I + 7) / 8, a.T * a.k), dim3(256), 0, s, a);
  if (e == cudaSuccess) e = launch_pdl(few_down_kernel, dim3(a.d.H / 8, a.T), dim3(256), 0, s, a);
  return e;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_layer_few_workspace_size(const moe_packed_desc_t* desc, int T, int top_k, size_t* bytes) {
  if (!bytes || !packed_desc_ok(desc) || T < 0 || T > kFewTokens || top_k < 1 || top_k > kMaxTopK || top_k > desc->E)
    return MOE_ERR_INVALID_ARG;
  *bytes = few_layout(*desc, T, top_k).total;
  return MOE_OK;
}

extern "C" moe_status_t moe_layer_few(const void* x, int64_t ldx, const void* w_router, int64_t ldw, int w_dtype,
                                      const moe_router_t* router, const float* bias, int T, const moe_packed_desc_t* desc,
                                      const void* packed, int top_k, void* out, int64_t ldo, int32_t* topk_idx,
                                      float* topk_w, void* workspace, size_t ws_bytes, moe_stream_t stream) {
  if (!packed_desc_ok(desc) || T < 0 || T > kFewTokens || !router_ok(router, desc->E, top_k) || !dtype_ok(w_dtype))
    return MOE_ERR_INVALID_ARG;
  const int E = desc->E, H = desc->H;
  if (ldx < H || ldw < H || ldo < H || ldx % 8 != 0 || ldo % 8 != 0 || ldw % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!x || !w_router || !packed || !out || !workspace)) return MOE_ERR_INVALID_ARG;
  if ((uintptr_t)x % 16 || (uintptr_t)w_router % 16 || (uintptr_t)out % 16 || (uintptr_t)packed % 256 ||
      (uintptr_t)workspace % 256 || (uintptr_t)bias % 4 || (uintptr_t)topk_idx % 4 || (uintptr_t)topk_w % 4)
    return MOE_ERR_INVALID_ARG;
  const FewLayout L = few_layout(*desc, T, top_k);
  if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  const moe_status_t dv = device_ok();
  if (dv != MOE_OK) return dv;
  if (T == 0) return MOE_OK;
  char* ws = (char*)workspace;
  FewArgs a;
  a.d = *desc;
  a.packed = (const char*)packed;
  a.x = (const __nv_bfloat16*)x;
  a.ldx = ldx;
  a.wr = w_router;
  a.ldw = ldw;
  a.w_dtype = w_dtype;
  a.out = (__nv_bfloat16*)out;
  a.ldo = ldo;
  a.T = T;
  a.k = top_k;
  a.logits = (float*)(ws + L.logits);
  int32_t* idx = topk_idx ? topk_idx : (int32_t*)(ws + L.idx);
  float* wt = topk_w ? topk_w : (float*)(ws + L.wt);
  a.idx = idx;
  a.wt = wt;
  a.h = (float*)(ws + L.h);
  a.status = (int*)(ws + L.status);
  const ScoreArgs r = {*router, a.logits, E, MOE_DT_F32, bias};
  return launch_few(a, r, idx, wt, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
