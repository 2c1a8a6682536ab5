// Declarations of the whole layer for a few tokens (moe_layer_few): its workspace and what its two kernels share.
//
// Operands.  The products run on mma.sync m16n8k16 with the weights as the 16-row operand and up to four tokens of an expert in
// the 8-column one (x in four columns; h, in two terms, in eight): bytes set the pace there and not the MMA rate, and the
// operands may come from registers, straight from the decoded codes, with no second trip through shared memory.  More than four tokens
// of one expert read its weights again.
// E4M3, E2M1 x E4M3 and INT4 weights are all exact in fp16, whose products with fp16 activations are exact in the
// fp32 accumulator; a row of activations is scaled by a power of two so that fp16 holds its bf16 values exactly (but for
// what is below 2^-39 of the row's largest, the last place of a subnormal), and an fp32 row of h is held in two fp16 terms.
// bf16 weights meet bf16 activations, h in two bf16 terms.
#pragma once
#include "moe_score.cuh"

namespace moe {

constexpr int kFewTokens = MOE_FEW_MAX_TOKENS;
constexpr int kFewSlots = kFewTokens * kMaxTopK;  // (token, choice) pairs

// What h and y hold before they are there: a NaN that is never written (few_value), so that whoever needs them can see from
// the values alone whether they are, with no flag to fence.
constexpr uint32_t kFewUnset = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t few_value(float v) {
  const uint32_t bits = __float_as_uint(v);
  return bits == kFewUnset ? 0x7FFFFFFFu : bits;
}

// Byte offsets in the workspace.  status: the device error word (as in ws_layout), the ticket counter; h and what follows is
// filled with kFewUnset.
struct FewLayout {
  size_t status, idx, wt, xinv, xs, h, y, total;
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
  ScoreArgs router;  // its logits are the first kernel's own
  int32_t* idx;      // [T, k]: the choice
  float* wt;
  int* status;       // [0] error word, [1] tickets handed out
  __half* xs;        // [T, H]: x scaled by a power of two per row (bf16 weights: unused)
  float* xinv;       // [T]: the scale's inverse
  float* h;          // [T k, I]
  float* y;          // [T k, H]: weighted rows
};
cudaError_t launch_few_router(const FewArgs& a, size_t fill_bytes, cudaStream_t s);
// lose_h: gate/up products are left out and the waits for them run out (moe_debug_few_timeout).
cudaError_t launch_few_experts(const FewArgs& a, bool lose_h, cudaStream_t s);

__host__ __device__ inline bool few_scales_x(int fmt) { return fmt != MOE_FMT_BF16; }

// The power of two that takes a row whose largest magnitude has these bits to below 2^15 (at 2^14 or more, but for rows
// below 2^-112), and its inverse.  A row with infinities or NaN counts as fp32's largest.
__device__ __forceinline__ float row_scale(uint32_t bits) {
  int e = (int)(bits >> 23 & 255u) - 127;
  e = e < -112 ? -112 : e;
  return __uint_as_float((uint32_t)(14 - e + 127) << 23);
}
__device__ __forceinline__ float row_scale_inv(uint32_t bits) {
  int e = (int)(bits >> 23 & 255u) - 127;
  e = e < -112 ? -112 : e;
  return __uint_as_float((uint32_t)(e - 14 + 127 > 0 ? e - 14 + 127 : 0) << 23);
}

}  // namespace moe
