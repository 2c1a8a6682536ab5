// The activation quantizer of the FP8 block format: one scale per 128 consecutive elements of a row.
#include "moe_fp8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 16;  // lanes of a group, eight elements each

// Sixteen lanes per group.  NaN does not count for the group's maximum (fmaxf) and stays NaN as a code.
// WIDE: every group is whole and every row starts on a multiple of 16 bytes (8 of codes).
template <class T, bool WIDE>
__global__ void __launch_bounds__(kThreads) fp8_quantize_kernel(const Fp8QuantArgs a) {
  pdl_wait();
  pdl_trigger();
  const int sub = threadIdx.x % kLanes;
  const int64_t n = (int64_t)a.T * a.groups, step = (int64_t)gridDim.x * (kThreads / kLanes);
  for (int64_t i0 = (int64_t)blockIdx.x * (kThreads / kLanes); i0 < n; i0 += step) {  // whole warps stay together
    const int64_t i = i0 + threadIdx.x / kLanes;
    const bool live = i < n;
    const int64_t t = live ? i / a.groups : 0;
    const int g = live ? (int)(i % a.groups) : 0, k = 128 * g + 8 * sub, left = live ? a.K - k : 0;
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
    for (int off = kLanes / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float s = fp8_scale(m);
    if (left <= 0) continue;
    uint32_t c[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) c[j] = fp8_codes2(v[4 * j], v[4 * j + 1], s) | fp8_codes2(v[4 * j + 2], v[4 * j + 3], s) << 16;
    uint8_t* q = a.q + t * a.ldq + k;
    if (WIDE) {
      *(uint2*)q = make_uint2(c[0], c[1]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) q[j] = (uint8_t)(c[j / 4] >> (8 * (j % 4)));
    }
    if (sub == 0) a.sinv[i] = __fdiv_rn(1.f, s);
  }
}

template <class T>
cudaError_t launch(const Fp8QuantArgs& a, cudaStream_t s) {
  const int64_t blocks = ((int64_t)a.T * a.groups + kThreads / kLanes - 1) / (kThreads / kLanes);
  const int64_t cap = (int64_t)tc_num_sms() * 8 * 8;
  const dim3 grid((unsigned)(blocks < cap ? blocks : cap));
  const bool wide = a.K % 128 == 0 && (uintptr_t)a.x % 16 == 0 && a.ldx * sizeof(T) % 16 == 0 && (uintptr_t)a.q % 8 == 0 && a.ldq % 8 == 0;
  note_launches(1);
  return wide ? launch_pdl(fp8_quantize_kernel<T, true>, grid, dim3(kThreads), 0, s, a)
              : launch_pdl(fp8_quantize_kernel<T, false>, grid, dim3(kThreads), 0, s, a);
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
  if (T < 0 || K < 1 || !dtype_ok(x_dtype) || ldx < K || ldq < K) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!x || !codes || !scale_inv)) return MOE_ERR_INVALID_ARG;
  if ((uintptr_t)x % dtype_size(x_dtype) || (uintptr_t)scale_inv % 4) return MOE_ERR_INVALID_ARG;
  const moe_status_t dv = device_ok();
  if (dv != MOE_OK) return dv;
  const Fp8QuantArgs a = {x, ldx, x_dtype, codes, ldq, scale_inv, T, K, (K + 127) / 128};
  return launch_fp8_quantize(a, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
