// Declarations shared by the operators around the experts (norms with the residual update, scored
// routing, request adapters): element types, wide loads, and the launches.
#pragma once
#include "moe_internal.cuh"

namespace moe {

inline size_t dtype_size(int dt) { return dt == MOE_DT_F32 ? 4 : 2; }
inline bool dtype_ok(int dt) { return dt >= MOE_DT_BF16 && dt <= MOE_DT_F32; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float v, float* p) { *p = v; }
__device__ __forceinline__ void from_f32(float v, __half* p) { *p = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }

// One element of a tensor whose type is only known at run time.
__device__ __forceinline__ float load_any(const void* base, int dt, int64_t at) {
  if (dt == MOE_DT_F32) return ((const float*)base)[at];
  if (dt == MOE_DT_F16) return to_f32(((const __half*)base)[at]);
  return to_f32(((const __nv_bfloat16*)base)[at]);
}

// One call of the norm / residual kernel.  block == null: enter (y = next(x)); else leave.
struct BlockArgs {
  const void *x, *block, *gate;
  void *out, *y;
  int64_t ldx, ldb, ldo, ldy, gate_ld;
  moe_norm_t post, next;  // kind 0: absent
  int gate_step, gate_dtype, gate_act;
  float alpha, beta;
  int T, H;
};
cudaError_t launch_block(const BlockArgs& a, int x_dtype, int act_dtype, cudaStream_t s);

// Scored routing (moe_router_t plus the tensors it reads).
struct ScoreArgs {
  moe_router_t r;
  const void* logits;
  int64_t ld;
  int dtype;
  const float* bias;
};
bool router_ok(const moe_router_t* r, int E, int top_k);
cudaError_t launch_route_scored(const ScoreArgs& a, int T, int E, int k, int32_t* topk_idx, float* topk_w,
                                cudaStream_t s);
// launch_route with the experts chosen by a scored router.
cudaError_t launch_route_by(const ScoreArgs& a, int T, int E, int k, int row_block, const WsLayout& L, char* ws,
                            const RoutePrelude& pre, cudaStream_t s);

struct AdapterArgs {
  const __nv_bfloat16 *x, *base, *A, *B;
  const float* scale;
  const int32_t *rank, *starts, *slot;
  __nv_bfloat16* out;
  int64_t ldx, ldb, ldo;
  int T, R, n, r, H, N;
};
cudaError_t launch_adapters(const AdapterArgs& a, cudaStream_t s);

}  // namespace moe
