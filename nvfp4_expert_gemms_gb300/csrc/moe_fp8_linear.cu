// Products in the FP8 block format (moe_fp8_linear): argument checks and the choice of kernel.
#include "moe_fp8.cuh"

namespace moe {
namespace {

// What a call needs beside its tensors: the codes and scales of activations that come unquantized.
size_t codes_bytes(int T, int K) { return ((size_t)T * K + 255) / 256 * 256; }
size_t workspace_bytes(int x_dtype, int T, int K) {
  return x_dtype == MOE_DT_E4M3 ? 0 : codes_bytes(T, K) + 4 * (size_t)T * ((K + 127) / 128);
}
constexpr int kMost = INT32_MAX - 512;  // what rounds up to tiles stays an int
bool sizes_ok(int x_dtype, int T, int K, int N, int act) {
  return (dtype_ok(x_dtype) || x_dtype == MOE_DT_E4M3) && T >= 0 && T <= kMost && K >= 16 && K <= kMost && K % 16 == 0 && N >= 1 && N <= kMost &&
         (act == MOE_ACT_NONE || (act == MOE_ACT_SILU_MUL && N % 2 == 0));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_fp8_linear_workspace_size(int x_dtype, int T, int K, int N, int act, size_t* bytes) {
  if (!bytes || !sizes_ok(x_dtype, T, K, N, act)) return MOE_ERR_INVALID_ARG;
  *bytes = workspace_bytes(x_dtype, T, K);
  return MOE_OK;
}

extern "C" moe_status_t moe_fp8_linear(const void* x, int64_t ldx, int x_dtype, const float* x_scale_inv, const uint8_t* w,
                                       const float* w_scale_inv, int act, const void* base, int64_t ldb, void* out,
                                       int64_t ldo, int out_dtype, int T, int K, int N, void* workspace, size_t ws_bytes,
                                       moe_stream_t stream) {
  if (!sizes_ok(x_dtype, T, K, N, act) || !dtype_ok(out_dtype)) return MOE_ERR_INVALID_ARG;
  const bool coded = x_dtype == MOE_DT_E4M3;
  const int out_n = act == MOE_ACT_SILU_MUL ? N / 2 : N;
  if (ldx < K || ldo < out_n || (base && ldb < out_n)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!x || !w || !w_scale_inv || !out || (coded && !x_scale_inv))) return MOE_ERR_INVALID_ARG;
  const size_t es = dtype_size(out_dtype);
  if ((uintptr_t)x % (coded ? 16 : dtype_size(x_dtype)) || (coded && ldx % 16) || (uintptr_t)x_scale_inv % 4 ||
      (uintptr_t)w % 16 || (uintptr_t)w_scale_inv % 4 || (uintptr_t)out % es || (uintptr_t)base % es)
    return MOE_ERR_INVALID_ARG;
  if (!coded && T > 0 && (!workspace || (uintptr_t)workspace % 256)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < workspace_bytes(x_dtype, T, K)) return MOE_ERR_WORKSPACE;
  const moe_status_t dv = device_ok();
  if (dv != MOE_OK) return dv;
  if (T == 0) return MOE_OK;
  const int groups = (K + 127) / 128;
  const cudaStream_t s = (cudaStream_t)stream;
  Fp8LinearArgs a = {x, ldx, x_dtype, x_scale_inv, w, w_scale_inv, base, ldb, out, ldo, out_dtype, T, K, N, groups, out_n};
  // Few rows in one launch that quantizes on the way.  Its blocks read all of x for 16 weight rows each, which past eight rows and some
  // 2^24 weights costs more than the tiles' second launch (us, one launch and tiles: 8 x 4096 x 14336 18.2 and 20.3, 16 x 2048 x 4096 7.4
  // and 11.2, 16 x 4096 x 3584 13.9 and 14.7, 16 x 4096 x 14336 37.0 and 20.6; at 2^24 itself it goes by the shape, 16 x 4096 x 4096 14.0 and
  // 14.8, 16 x 2048 x 8192 14.4 and 11.9).
  if (T <= kFp8Rows / 2 || (T <= kFp8Rows && (int64_t)N * K < 1 << 24)) return launch_fp8_rows(a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  if (!coded) {
    uint8_t* q = (uint8_t*)workspace;
    float* qs = (float*)(q + codes_bytes(T, K));
    const Fp8QuantArgs qa = {x, ldx, x_dtype, q, K, qs, T, K, groups};
    if (launch_fp8_quantize(qa, s) != cudaSuccess) return MOE_ERR_CUDA;
    a.x = q;
    a.ldx = K;
    a.x_dtype = MOE_DT_E4M3;
    a.qs = qs;
  }
  return launch_fp8_tiles(a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
