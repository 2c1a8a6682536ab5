// Routing alone with a scored router (moe_route_scored): one warp per token, no workspace.
#include "moe_score.cuh"

namespace moe {
namespace {

constexpr int kScoreWarps = 8;

template <int VT>
__global__ void __launch_bounds__(32 * kScoreWarps) score_kernel(const ScoreArgs a, const ScoreGeom g, int T, int k,
                                                                 int32_t* __restrict__ topk_idx,
                                                                 float* __restrict__ topk_w) {
  __shared__ ScoreScratch scratch[kScoreWarps];
  const int warp = threadIdx.x >> 5;
  const uint32_t t = blockIdx.x * kScoreWarps + warp;
  pdl_wait();
  pdl_trigger();
  if (t < (uint32_t)T) score_token<VT>(a, g, (int)t, k, threadIdx.x & 31, topk_idx, topk_w, scratch[warp]);
}

}  // namespace

bool router_ok(const moe_router_t* r, int E, int k) {
  if (!r || (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID)) return false;
  if (E < 1 || E > kMaxE || k < 1 || k > kMaxTopK || k > E) return false;
  if (r->groups < 1 || r->groups > 32 || E % r->groups != 0) return false;
  if (r->top_groups < 1 || r->top_groups > r->groups || r->top_groups * (E / r->groups) < k) return false;
  return (r->group_top == 1 || r->group_top == 2) && (r->renormalize == 0 || r->renormalize == 1) && r->scale == r->scale;
}

cudaError_t launch_route_scored(const ScoreArgs& a, int T, int E, int k, int32_t* topk_idx, float* topk_w,
                                cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  const ScoreGeom g = score_geom(a, E);
  const dim3 grid((unsigned)(((int64_t)T + kScoreWarps - 1) / kScoreWarps)), block(32 * kScoreWarps);
  note_launches(1);
  if (g.per <= 1) return launch_pdl(score_kernel<1>, grid, block, 0, s, a, g, T, k, topk_idx, topk_w);
  if (g.per <= 2) return launch_pdl(score_kernel<2>, grid, block, 0, s, a, g, T, k, topk_idx, topk_w);
  if (g.per <= 4) return launch_pdl(score_kernel<4>, grid, block, 0, s, a, g, T, k, topk_idx, topk_w);
  if (g.per <= 8) return launch_pdl(score_kernel<8>, grid, block, 0, s, a, g, T, k, topk_idx, topk_w);
  return launch_pdl(score_kernel<16>, grid, block, 0, s, a, g, T, k, topk_idx, topk_w);
}

}  // namespace moe

extern "C" moe_status_t moe_route_scored(const moe_router_t* router, const void* logits, int64_t ld, int dtype,
                                         const float* bias, int T, int E, int top_k, int32_t* topk_idx, float* topk_w,
                                         moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || !router_ok(router, E, top_k) || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !topk_idx || !topk_w || ld < E)) return MOE_ERR_INVALID_ARG;
  if ((uintptr_t)logits % dtype_size(dtype) != 0 || (uintptr_t)bias % 4 != 0 || (uintptr_t)topk_idx % 4 != 0 ||
      (uintptr_t)topk_w % 4 != 0)
    return MOE_ERR_INVALID_ARG;
  const moe_status_t dv = device_ok();
  if (dv != MOE_OK) return dv;
  const ScoreArgs a = {*router, logits, ld, dtype, bias};
  return launch_route_scored(a, T, E, top_k, topk_idx, topk_w, (cudaStream_t)stream) == cudaSuccess ? MOE_OK
                                                                                                    : MOE_ERR_CUDA;
}
