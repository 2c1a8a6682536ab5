// Declarations of the products in the FP8 block format (moe_fp8_quantize, moe_fp8_linear).
#pragma once
#include "moe_block.cuh"

namespace moe {

struct Fp8QuantArgs {
  const void* x;
  int64_t ldx;
  int dtype;
  uint8_t* q;
  int64_t ldq;
  float* sinv;  // [T, groups]
  int T, K, groups;
};
cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, cudaStream_t s);

struct Fp8LinearArgs {
  const uint8_t* q;  // E4M3 [T, K]
  int64_t ldq;
  const float* qs;   // [T, groups]
  const uint8_t* w;  // E4M3 [N, K]
  const float* ws;   // [ceil(N / 128), groups]
  const void* base;  // out's type, or null
  int64_t ldb;
  void* out;
  int64_t ldo;
  int out_dtype;
  int T, K, N, groups;
  int out_n;  // N, or N / 2 with SiLU(gate) * up
};

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + expf(-g)) * u; }

}  // namespace moe
