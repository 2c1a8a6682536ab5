// Shared by the adapter kernels: the tile of a block (moe_adapter_find.cuh), and packed bf16 pairs.
#pragma once
#include "moe_block.cuh"
#include "moe_adapter_find.cuh"

namespace moe {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *(const uint32_t*)&v;
}
__device__ __forceinline__ float lo_f32(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float hi_f32(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }

// The pair f0, f1 as two bf16 terms each.  hi stops at bf16's largest value, so that an infinity, or what bf16 would
// round to one, leaves a rest in lo and not a difference of infinities.
__device__ __forceinline__ void split_pair(float f0, float f1, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(f1), "f"(f0));
  lo = pack_bf16(f0 - lo_f32(hi), f1 - hi_f32(hi));
}

// Long requests on the 5th-generation tensor cores (moe_adapter_tile.cu): tiles of 128 tokens.
bool adapter_tiles_fit(const AdapterArgs& a);
cudaError_t launch_adapter_tiles(const AdapterArgs& a, cudaStream_t s);

}  // namespace moe
