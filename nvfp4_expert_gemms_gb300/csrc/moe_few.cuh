// Declarations of the whole layer for a few tokens (moe_layer_few): its workspace and its two kernels' arguments.
#pragma once
#include "moe_block.cuh"

namespace moe {

constexpr int kFewTokens = MOE_FEW_MAX_TOKENS;

// Byte offsets in the workspace.  status: the device error word (as in ws_layout), then what the first kernel zeroes.
struct FewLayout {
  size_t status, idx, wt, logits, h, total;
};
FewLayout few_layout(const moe_packed_desc_t& d, int T, int k);

struct FewArgs {
  moe_packed_desc_t d;
  const char* packed;
  const __nv_bfloat16* x;
  int64_t ldx;
  const void* wr;  // router [E, H]
  int64_t ldw;
  int w_dtype;
  __nv_bfloat16* out;
  int64_t ldo;
  int T, k;
  float* logits;  // [T, E]
  const int32_t* idx;  // [T, k]
  const float* wt;
  float* h;  // [T k, I]
  int* status;
};
cudaError_t launch_few(const FewArgs& a, const ScoreArgs& r, int32_t* idx, float* wt, cudaStream_t s);

}  // namespace moe
