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

// Eight elements of the router's row, as fp32.
__device__ __forceinline__ void load_router8(const void* base, int dt, int64_t at, float (&w)[8]) {
  if (dt == MOE_DT_F32) {
    const float4 a = ((const float4*)((const float*)base + at))[0], b = ((const float4*)((const float*)base + at))[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    return;
  }
  const uint4 u = *(const uint4*)((const uint16_t*)base + at);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = dt == MOE_DT_F16 ? to_f32(((const __half*)&u)[i]) : to_f32(((const __nv_bfloat16*)&u)[i]);
}

// Blocks below E: logits[t, e] = sum over h of x[t, h] w[e, h], one block per expert.  The sum is carried in pairs, so
// that it is the exact sum rounded once (but for one case in some 2^20): which experts a token gets must not hang on the
// order of a sum.  Blocks from E on: a token's row scaled into fp16 for the experts.  Block 0 zeroes the counters.
__global__ void __launch_bounds__(kRouterThreads) few_router_kernel(const FewArgs a, int zero_words) {
  __shared__ Pair part[kRouterThreads / 32][kRouterTokens];
  __shared__ uint32_t s_max[kRouterThreads / 32];
  const int e = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H = a.d.H;
  pdl_wait();
  pdl_trigger();
  if (e == 0)
    for (int i = threadIdx.x; i < zero_words; i += kRouterThreads) a.status[i] = 0;
  if (e >= a.d.E) {
    const int t = e - a.d.E;
    uint32_t m = 0;
    for (int i = threadIdx.x; i < H / 8; i += kRouterThreads) {
      const uint4 u = *(const uint4*)(a.x + t * a.ldx + 8 * i);
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu)));
    }
    m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int w = 0; w < kRouterThreads / 32; ++w) m = max(m, s_max[w]);
    const float scale = row_scale(m << 16);
    if (threadIdx.x == 0) a.xinv[t] = row_scale_inv(m << 16);
    for (int i = threadIdx.x; i < H / 8; i += kRouterThreads) {
      const uint4 u = *(const uint4*)(a.x + t * a.ldx + 8 * i);
      const uint32_t v[4] = {u.x, u.y, u.z, u.w};
      __half2 o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = __floats2half2_rn(__uint_as_float(v[j] << 16) * scale, __uint_as_float(v[j] & 0xFFFF0000u) * scale);
      *(uint4*)(a.xs + (size_t)t * H + 8 * i) = *(const uint4*)o;
    }
    return;
  }
  for (int t0 = 0; t0 < a.T; t0 += kRouterTokens) {
    const int nt = min(kRouterTokens, a.T - t0);
    Pair acc[kRouterTokens];
    for (int i = 8 * threadIdx.x; i < H; i += 8 * kRouterThreads) {
      float w[8];
      load_router8(a.wr, a.w_dtype, e * a.ldw + i, w);
#pragma unroll
      for (int t = 0; t < kRouterTokens; ++t)
        if (t < nt) {
          const uint4 u = *(const uint4*)(a.x + (t0 + t) * a.ldx + i);
          const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[t].add_product(__uint_as_float(v[j] << 16), w[2 * j]);
            acc[t].add_product(__uint_as_float(v[j] & 0xFFFF0000u), w[2 * j + 1]);
          }
        }
    }
#pragma unroll
    for (int t = 0; t < kRouterTokens; ++t) {
      if (t >= nt) break;
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

}  // namespace

FewLayout few_layout(const moe_packed_desc_t& d, int T, int k) {
  FewLayout L;
  size_t cur = 0;
  auto take = [&](size_t bytes) {
    const size_t o = cur;
    cur += (bytes + 255) / 256 * 256;
    return o;
  };
  const size_t R = (size_t)T * k, active = R < (size_t)d.E ? R : (size_t)d.E;
  L.status = take(256);
  L.done = take(4 * active);
  L.tile = take(4 * (size_t)(d.H / 16));
  L.hmax = take(4 * R);
  L.zero_end = cur;
  L.xinv = take(4 * (size_t)T);
  L.logits = take(4 * (size_t)T * d.E);
  L.xs = take(few_scales_x(d.fmt) ? 2 * (size_t)T * d.H : 0);
  L.h = take(4 * R * d.I);
  L.y = take(4 * R * (size_t)d.H);
  L.total = cur;
  return L;
}

cudaError_t launch_few_router(const FewArgs& a, size_t zero_bytes, cudaStream_t s) {
  note_launches(1);
  const int grid = a.d.E + (few_scales_x(a.d.fmt) ? a.T : 0);
  return launch_pdl(few_router_kernel, dim3(grid), dim3(kRouterThreads), 0, s, a, (int)(zero_bytes / 4));
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
  if (H > kFewWidth || desc->I > kFewWidth) return MOE_ERR_UNSUPPORTED;
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
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.status = (int*)(ws + L.status);
  a.done = (int*)(ws + L.done);
  a.tile = (int*)(ws + L.tile);
  a.hmax = (unsigned*)(ws + L.hmax);
  a.xinv = (float*)(ws + L.xinv);
  a.logits = (float*)(ws + L.logits);
  a.xs = (__half*)(ws + L.xs);
  a.h = (float*)(ws + L.h);
  a.y = (float*)(ws + L.y);
  a.router = {*router, a.logits, E, MOE_DT_F32, bias};
  cudaError_t e = launch_few_router(a, L.zero_end, (cudaStream_t)stream);
  if (e == cudaSuccess) e = launch_few_experts(a, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
