// A whole mixture-of-experts layer for a few tokens (moe_layer_few): argument checks, the router's product and its choice.
#include "moe_few.cuh"
#include "moe_formats.cuh"

namespace moe {

namespace {

constexpr int kCluster = 8;          // blocks per token
constexpr int kRouterWarps = 16, kRouterThreads = 32 * kRouterWarps;

// Two sums at once, each kept as an unevaluated pair of fp32 numbers, hi + lo.  Adding p loses nothing: with s the rounded
// hi + p and b = s - hi, what rounding left out is itself a number that fp32 holds, (hi - (s - b)) + (p - b), and lo collects
// it.  A product of bf16 and a 16-bit number is such a p, which fma computes on the way; of an fp32 number it is the
// rounded product, whose own error lo takes as well.
struct Pairs {
  float2 hi = {0.f, 0.f}, lo = {0.f, 0.f};
  static __device__ __forceinline__ uint64_t bits(float2 v) { return *(const uint64_t*)&v; }
  static __device__ __forceinline__ float2 add(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return *(const float2*)&r;
  }
  static __device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return *(const float2*)&r;
  }
  static __device__ __forceinline__ float2 sub(float2 a, float2 b) { return fma(b, make_float2(-1.f, -1.f), a); }
  static __device__ __forceinline__ float2 neg(float2 a) { return make_float2(-a.x, -a.y); }
  __device__ __forceinline__ void add_product(float2 x, float2 w) {
    const float2 s = fma(x, w, hi), b = sub(s, hi);
    lo = add(lo, add(sub(hi, sub(s, b)), fma(x, w, neg(b))));
    hi = s;
  }
  __device__ __forceinline__ void add_wide_product(float2 x, float2 w) {
    const float2 p = fma(x, w, make_float2(0.f, 0.f)), s = add(hi, p), b = sub(s, hi);
    lo = add(add(lo, fma(x, w, neg(p))), add(sub(hi, sub(s, b)), sub(p, b)));
    hi = s;
  }
};
__device__ __forceinline__ void add_pair(float& hi, float& lo, float ohi, float olo) {
  const float s = __fadd_rn(hi, ohi), b = __fsub_rn(s, hi);
  lo = __fadd_rn(__fadd_rn(lo, olo), __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(ohi, b)));
  hi = s;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// *p of the cluster's first block
__device__ __forceinline__ void store_in_first(float* p, float v) {
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, 0;\n st.shared::cluster.f32 [a], %1;\n}" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(p)),
               "f"(v)
               : "memory");
}

// Eight bf16 or fp16 elements as fp32.
__device__ __forceinline__ void unpack8(const uint4& u, bool f16, float2 (&w)[4]) {
  const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = f16 ? __half22float2(*(const __half2*)&v[i]) : make_float2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xFFFF0000u));
}

// A cluster of eight blocks per token: its logits, its experts and its row scaled into fp16.
//   logits[t, e] = sum over h of x[t, h] w[e, h], a warp per expert.  The sum is carried in pairs: which experts a token gets must not
//   hang on the order of a sum.  Of a pair lo alone is rounded, n = H / 64 times in a lane and twice in each of six meetings, while it grows to
//   n 2^-24 of the largest partial sum: together less than (n + 12)^2 2^-48 of sum |x w| (four times that for fp32 w, whose products add a
//   rounding of their own).  Without cancellation that leaves one logit in some 2^20 that is not the exact sum's nearest.
// Eight blocks of sixteen warps per token because one token's products (E H of them, seven operations each for two) would
// take one SM several microseconds; the logits go straight to the first block's shared memory, where one warp chooses.  Past fp32's range lo is not a number and hi alone counts.  h and y are filled with
// the mark of what is not there yet.
template <int VT, bool F32>
__global__ void __launch_bounds__(kRouterThreads, 1) few_router_kernel(const __grid_constant__ FewArgs a, const ScoreGeom geom, size_t pieces) {
  __shared__ ScoreScratch scratch;
  __shared__ __align__(16) float s_logits[kMaxE];  // the first block's
  constexpr int kAhead = F32 ? 4 : 8;  // pieces of eight a lane loads before it multiplies them
  __shared__ uint32_t s_max[kRouterWarps];
  const int t = blockIdx.x / kCluster, rank = blockIdx.x % kCluster, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H = a.d.H, E = a.d.E;
  const __nv_bfloat16* x = a.x + t * a.ldx;
  cluster_arrive();  // the first block's shared memory is there once all have started
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x < 2) a.status[threadIdx.x] = 0;
  for (size_t i = blockIdx.x * kRouterThreads + threadIdx.x; i < pieces; i += gridDim.x * kRouterThreads)
    ((uint4*)a.h)[i] = make_uint4(kFewUnset, kFewUnset, kFewUnset, kFewUnset);
  __syncwarp();  // (the loop may end inside a warp, and the barrier takes whole ones)
  cluster_wait();
  for (int e = rank * kRouterWarps + warp; e < E; e += kCluster * kRouterWarps) {
    Pairs sum;
    for (int i0 = 8 * lane; i0 < H; i0 += 256 * kAhead) {  // a lane's pieces of eight, the loads of kAhead of them first
      uint4 u[kAhead], w[F32 ? 2 * kAhead : kAhead];
#pragma unroll
      for (int n = 0; n < kAhead; ++n) {
        const int i = i0 + 256 * n;
        if (i >= H) break;
        u[n] = *(const uint4*)(x + i);
        if constexpr (F32) {
          const uint4* p = (const uint4*)((const float*)a.wr + e * a.ldw + i);
          w[2 * n] = p[0], w[2 * n + 1] = p[1];
        } else {
          w[n] = *(const uint4*)((const uint16_t*)a.wr + e * a.ldw + i);
        }
      }
#pragma unroll
      for (int n = 0; n < kAhead; ++n) {
        if (i0 + 256 * n >= H) break;
        float2 xv[4], wv[4];
        unpack8(u[n], false, xv);
        if constexpr (F32) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4& q = w[2 * n + j / 2];
            wv[j] = j % 2 ? make_float2(__uint_as_float(q.z), __uint_as_float(q.w)) : make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
            sum.add_wide_product(xv[j], wv[j]);
          }
        } else {
          unpack8(w[n], a.w_dtype == MOE_DT_F16, wv);
#pragma unroll
          for (int j = 0; j < 4; ++j) sum.add_product(xv[j], wv[j]);
        }
      }
    }
    float hi = sum.hi.x, lo = sum.lo.x;
    add_pair(hi, lo, sum.hi.y, sum.lo.y);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float ohi = __shfl_xor_sync(0xffffffffu, hi, off), olo = __shfl_xor_sync(0xffffffffu, lo, off);
      add_pair(hi, lo, ohi, olo);
    }
    if (lane == 0) store_in_first(s_logits + e, isfinite(hi) ? __fadd_rn(hi, lo) : hi);
  }
  __syncwarp();
  cluster_arrive();
  if (rank == 1 && few_scales_x(a.d.fmt)) {  // the row for the experts
    uint32_t m = 0;
    for (int i = threadIdx.x; i < H / 8; i += kRouterThreads) {
      const uint4 u = *(const uint4*)(x + 8 * i);
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu)));
    }
    m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int w = 0; w < kRouterWarps; ++w) m = max(m, s_max[w]);
    const float scale = row_scale(m << 16);
    if (threadIdx.x == 0) a.xinv[t] = row_scale_inv(m << 16);
    for (int i = threadIdx.x; i < H / 8; i += kRouterThreads) {
      const uint4 u = *(const uint4*)(x + 8 * i);
      const uint32_t v[4] = {u.x, u.y, u.z, u.w};
      __half2 o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = __floats2half2_rn(__uint_as_float(v[j] << 16) * scale, __uint_as_float(v[j] & 0xFFFF0000u) * scale);
      *(uint4*)(a.xs + (size_t)t * H + 8 * i) = *(const uint4*)o;
    }
  }
  __syncwarp();
  cluster_wait();
  if (rank == 0 && warp == 0) {
    ScoreArgs r = a.router;
    r.logits = s_logits;
    score_token<VT>(r, geom, 0, a.k, lane, a.idx + t * a.k, a.wt + t * a.k, scratch);
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
  const size_t R = (size_t)T * k;
  L.status = take(256);
  L.idx = take(4 * R);
  L.wt = take(4 * R);
  L.xinv = take(4 * (size_t)T);
  L.xs = take(few_scales_x(d.fmt) ? 2 * (size_t)T * d.H : 0);
  L.h = take(4 * R * d.I);
  L.y = take(4 * R * (size_t)d.H);
  L.total = cur;
  return L;
}

cudaError_t launch_few_router(const FewArgs& a, size_t fill_bytes, cudaStream_t s) {
  const ScoreGeom g = score_geom(a.router, a.d.E);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.T * kCluster);
  cfg.blockDim = dim3(kRouterThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const size_t pieces = fill_bytes / 16;
  note_launches(1);
  const bool f32 = a.w_dtype == MOE_DT_F32;
  if (g.per <= 1) return cudaLaunchKernelEx(&cfg, f32 ? few_router_kernel<1, true> : few_router_kernel<1, false>, a, g, pieces);
  if (g.per <= 2) return cudaLaunchKernelEx(&cfg, f32 ? few_router_kernel<2, true> : few_router_kernel<2, false>, a, g, pieces);
  if (g.per <= 4) return cudaLaunchKernelEx(&cfg, f32 ? few_router_kernel<4, true> : few_router_kernel<4, false>, a, g, pieces);
  if (g.per <= 8) return cudaLaunchKernelEx(&cfg, f32 ? few_router_kernel<8, true> : few_router_kernel<8, false>, a, g, pieces);
  return cudaLaunchKernelEx(&cfg, f32 ? few_router_kernel<16, true> : few_router_kernel<16, false>, a, g, pieces);
}

}  // namespace moe

using namespace moe;

static thread_local bool t_lose_h = false;

extern "C" void moe_debug_few_timeout(void) { t_lose_h = true; }

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
  a.idx = topk_idx ? topk_idx : (int32_t*)(ws + L.idx);
  a.wt = topk_w ? topk_w : (float*)(ws + L.wt);
  a.status = (int*)(ws + L.status);
  a.xinv = (float*)(ws + L.xinv);
  a.xs = (__half*)(ws + L.xs);
  a.h = (float*)(ws + L.h);
  a.y = (float*)(ws + L.y);
  a.router = {*router, workspace, E, MOE_DT_F32, bias};  // (the logits stay in shared memory)
  const bool lose_h = t_lose_h;
  t_lose_h = false;
  cudaError_t e = launch_few_router(a, L.total - L.h, (cudaStream_t)stream);
  if (e == cudaSuccess) e = launch_few_experts(a, lose_h, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
