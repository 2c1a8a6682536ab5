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
  const void* x;     // x_dtype [T, K]; E4M3 codes for the tiles
  int64_t ldx;
  int x_dtype;
  const float* qs;   // [T, groups] with codes
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
// Up to kFp8Rows rows, of any x_dtype (moe_fp8_rows.cu); any number, of codes (moe_fp8_tile.cu).  moe_fp8_linear.cu chooses.
constexpr int kFp8Rows = 16;
cudaError_t launch_fp8_rows(const Fp8LinearArgs& a, cudaStream_t s);
cudaError_t launch_fp8_tiles(const Fp8LinearArgs& a, cudaStream_t s);

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + expf(-g)) * u; }

// The quantizer's scale of a group whose largest magnitude is m.
__device__ __forceinline__ float fp8_scale(float m) { return __fdiv_rn(448.f, fmaxf(m, 1e-12f)); }
// Two values' codes, scaled.
__device__ __forceinline__ uint32_t fp8_codes2(float a, float b, float s) {
  return __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(a, s), __fmul_rn(b, s)), __NV_SATFINITE, __NV_E4M3);
}

// A group's partial sum p is multiplied with two scales, w of the weights and x of the row.  Their product alone may leave fp32's
// normal range where p w x does not (a row near 3e38 and a weight scale of 1000: 0 times infinity where codes are zero).  w and x are
// then on the same side of 1, and p times one and then the other stays in range as long as the result does: p is multiplied with
// scale_before first, and with scale_after then.
__device__ __forceinline__ bool scales_meet(float t) { return fabsf(t) >= 1.17549435e-38f && fabsf(t) <= 3.40282347e38f; }
__device__ __forceinline__ float scale_before(float w, float x) { return scales_meet(w * x) ? 1.f : w; }
__device__ __forceinline__ float scale_after(float w, float x) { return scales_meet(w * x) ? w * x : x; }
// Two scales of which each is at least 2^-63 and below 2^64 meet.
__device__ __forceinline__ bool scale_moderate(float v) { return (__float_as_uint(v) & 0x7FFFFFFFu) - 0x20000000u < 0x3F800000u; }

// Eight elements as fp32; 0 past n.  WIDE: all eight, 16-byte aligned.
template <class T, bool WIDE>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
  if (WIDE) {
    if (sizeof(T) == 4) {
      const float4 a = ((const float4*)p)[0], b = ((const float4*)p)[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 u = *(const uint4*)p;
      const T* e = (const T*)&u;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}

__device__ __forceinline__ void store_any(void* base, int dt, int64_t at, float v) {
  if (dt == MOE_DT_F32) ((float*)base)[at] = v;
  else if (dt == MOE_DT_F16) ((__half*)base)[at] = __float2half_rn(v);
  else ((__nv_bfloat16*)base)[at] = __float2bfloat16_rn(v);
}

}  // namespace moe
