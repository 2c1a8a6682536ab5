// The activation quantizer of the FP8 block format: one scale per 128 consecutive elements of a row.
#include <type_traits>

#include "moe_fp8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Sixteen consecutive elements, and their largest magnitude (NaN left out, as fmaxf leaves it).
template <class T>
struct Sixteen {
  uint4 u[sizeof(T)];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T)); ++i) u[i] = ((const uint4*)p)[i];
  }
  __device__ __forceinline__ float at(int i) const { return to_f32(((const T*)u)[i]); }
  __device__ __forceinline__ float largest() const {
    if constexpr (sizeof(T) == 4) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(at(i)));
      return m;
    } else {
      using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
      const T2* w = (const T2*)u;
      T2 m = __habs2(w[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = __hmax2(m, __habs2(w[i]));
      return fmaxf(to_f32(m.x), to_f32(m.y));
    }
  }
};

// Whole groups, rows on multiples of 16 bytes: eight lanes per group, sixteen elements each.  The place of a lane's next group comes
// by addition, not by division.  Bound: HBM; instructions count too (16384 x 2048 bf16: with eight elements per lane and a
// division per group 25 us, 15 by HBM).
template <class T>
__global__ void __launch_bounds__(kThreads) fp8_quantize_kernel(const Fp8QuantArgs a) {
  pdl_wait();
  pdl_trigger();
  const int sub = threadIdx.x % 8;
  const int64_t i0 = (int64_t)blockIdx.x * (kThreads / 8) + threadIdx.x / 8, step = (int64_t)gridDim.x * (kThreads / 8);
  int64_t t = i0 / a.groups;
  int g = (int)(i0 - t * a.groups);
  const int64_t dt = step / a.groups;
  const int dg = (int)(step - dt * a.groups);
  Sixteen<T> next;
  if (t < a.T) next.load((const T*)a.x + t * a.ldx + 128 * g + 16 * sub);
  while (__any_sync(0xffffffffu, t < a.T)) {  // whole warps stay together
    const Sixteen<T> v = next;
    const bool live = t < a.T;
    const int64_t tt = t;
    const int gg = g;
    t += dt;
    g += dg;
    if (g >= a.groups) g -= a.groups, ++t;
    if (t < a.T) next.load((const T*)a.x + t * a.ldx + 128 * g + 16 * sub);
    float m = v.largest();
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float s = fp8_scale(m);
    if (!live) continue;
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = fp8_codes2(v.at(4 * j), v.at(4 * j + 1), s) | fp8_codes2(v.at(4 * j + 2), v.at(4 * j + 3), s) << 16;
    uint8_t* q = a.q + tt * a.ldq + 128 * gg + 16 * sub;
    if ((uintptr_t)q % 16 == 0) {
      *(uint4*)q = make_uint4(c[0], c[1], c[2], c[3]);
    } else {
      *(uint2*)q = make_uint2(c[0], c[1]);
      *(uint2*)(q + 8) = make_uint2(c[2], c[3]);
    }
    if (sub == 0) a.sinv[tt * a.groups + gg] = __fdiv_rn(1.f, s);
  }
}

// Any others: sixteen lanes per group, eight elements each; WIDE: these are whole and on multiples of 16 bytes (8 of codes), else one
// at a time.
template <class T, bool WIDE>
__global__ void __launch_bounds__(kThreads) fp8_quantize_any_kernel(const Fp8QuantArgs a) {
  pdl_wait();
  pdl_trigger();
  const int sub = threadIdx.x % 16;
  const int64_t n = (int64_t)a.T * a.groups, step = (int64_t)gridDim.x * (kThreads / 16);
  for (int64_t i0 = (int64_t)blockIdx.x * (kThreads / 16); i0 < n; i0 += step) {  // whole warps stay together
    const int64_t i = i0 + threadIdx.x / 16;
    const bool live = i < n;
    const int64_t t = !live ? 0 : n <= UINT32_MAX ? (uint32_t)i / (uint32_t)a.groups : i / a.groups;
    const int g = live ? (int)(i - t * a.groups) : 0, k = 128 * g + 8 * sub, left = live ? a.K - k : 0;
    float v[8];
    if (left > 0) {
      load8<T, WIDE>((const T*)a.x + t * a.ldx + k, left, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float s = fp8_scale(m);
    if (left <= 0) continue;
    uint8_t* q = a.q + t * a.ldq + k;
    if (WIDE) {
      uint32_t c[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) c[j] = fp8_codes2(v[4 * j], v[4 * j + 1], s) | fp8_codes2(v[4 * j + 2], v[4 * j + 3], s) << 16;
      *(uint2*)q = make_uint2(c[0], c[1]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const uint32_t c = fp8_codes2(v[j], v[j + 1], s);
        if (j < left) q[j] = (uint8_t)c;
        if (j + 1 < left) q[j + 1] = (uint8_t)(c >> 8);
      }
    }
    if (sub == 0) a.sinv[i] = __fdiv_rn(1.f, s);
  }
}

template <class T>
cudaError_t launch(const Fp8QuantArgs& a, cudaStream_t s) {
  const bool parts = a.K % 8 == 0 && (uintptr_t)a.x % 16 == 0 && a.ldx * sizeof(T) % 16 == 0 && (uintptr_t)a.q % 8 == 0 && a.ldq % 8 == 0, wide = parts && a.K % 128 == 0;
  const int per = wide ? kThreads / 8 : kThreads / 16;  // groups of a block
  const int64_t blocks = ((int64_t)a.T * a.groups + per - 1) / per, cap = (int64_t)tc_num_sms() * (wide ? 8 : 64);
  const dim3 grid((unsigned)(blocks < cap ? blocks : cap));
  note_launches(1);
  return wide ? launch_pdl(fp8_quantize_kernel<T>, grid, dim3(kThreads), 0, s, a)
         : parts ? launch_pdl(fp8_quantize_any_kernel<T, true>, grid, dim3(kThreads), 0, s, a)
                 : launch_pdl(fp8_quantize_any_kernel<T, false>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (a.dtype == MOE_DT_BF16) return launch<__nv_bfloat16>(a, s);
  if (a.dtype == MOE_DT_F16) return launch<__half>(a, s);
  return launch<float>(a, s);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_fp8_quantize(const void* x, int64_t ldx, int x_dtype, uint8_t* codes, int64_t ldq,
                                         float* scale_inv, int T, int K, moe_stream_t stream) {
  if (T < 0 || K < 1 || K > INT32_MAX - 512 || !dtype_ok(x_dtype) || ldx < K || ldq < K) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!x || !codes || !scale_inv)) return MOE_ERR_INVALID_ARG;
  if ((uintptr_t)x % dtype_size(x_dtype) || (uintptr_t)scale_inv % 4) return MOE_ERR_INVALID_ARG;
  const moe_status_t dv = device_ok();
  if (dv != MOE_OK) return dv;
  const Fp8QuantArgs a = {x, ldx, x_dtype, codes, ldq, scale_inv, T, K, (K + 127) / 128};
  return launch_fp8_quantize(a, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
