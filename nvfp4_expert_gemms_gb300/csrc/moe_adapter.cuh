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

// The pair f0, f1 as three bf16 terms each, 24 bits of significand: all that fp32 has.  The first two stop at bf16's
// largest value, so that an infinity, or what bf16 would round to one, leaves a rest and not a difference of infinities.
struct Terms {
  uint32_t hi, mid, lo;
};
__device__ __forceinline__ uint32_t pack_bf16_sat(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ Terms split_pair(float f0, float f1) {
  Terms t;
  t.hi = pack_bf16_sat(f0, f1);
  f0 -= lo_f32(t.hi);
  f1 -= hi_f32(t.hi);
  t.mid = pack_bf16_sat(f0, f1);
  t.lo = pack_bf16(f0 - lo_f32(t.mid), f1 - hi_f32(t.mid));
  return t;
}

// Long requests on the 5th-generation tensor cores (moe_adapter_tile.cu): tiles of 128 tokens.
bool adapter_tiles_fit(const AdapterArgs& a);
cudaError_t launch_adapter_tiles(const AdapterArgs& a, cudaStream_t s);

}  // namespace moe
