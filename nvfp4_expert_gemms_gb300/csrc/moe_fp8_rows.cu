// moe_fp8_linear for a few rows: one kernel that quantizes the rows on the way.
//
// A block takes 16 weight rows (8 gates and the same features' ups), sixteen warps a group of 128 columns each, and up to eight or
// 16 rows of x.  A lane loads its shares of the weights and of eight rows of x straight into registers, all at once; four lanes hold a row's group, so
// its maximum is two shuffles away, and every warp quantizes what it multiplies.  E4M3 times E4M3 is exact in fp16 operands
// with an fp32 accumulator (mma.sync m16n8k16: the weights' bytes set the pace).  The sums meet in shared memory.
// Bound: latency (1 x 2048 x 4096: 3.8 us in a graph, 1.2 by HBM), for large matrices L2, from which every block reads all of x.
#include "moe_fp8.cuh"

namespace moe {
namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kPass = 8;  // rows of x at a time
static_assert(kFp8Rows == 2 * kPass, "one or two passes");

__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t c) {  // the two codes in c's low half
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xFFFFu), __NV_E4M3);
  return *(const uint32_t*)&h;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's 32 codes of a row's group, as the MMA's column operand, and the group's scale_inv (in its four lanes).  The lane's elements: 16 t ..
// and 64 + 16 t .. of the group, which ends at `left` columns.
// (Loaded twice, the second time from L1: 32 values would not stay in registers beside the weights.)
template <class T, bool WIDE>
__device__ __forceinline__ float quantize_group(const T* p, int left, int t, uint32_t (&b)[16]) {
  float m = 0.f, v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = 64 * (j >> 1) + 16 * t + 8 * (j & 1);
    if (left > k) {  // (columns come in 16s)
      load8<T, WIDE>(p + k, 8, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
    }
  }
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const float s = fp8_scale(m);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = 64 * (j >> 1) + 16 * t + 8 * (j & 1);
    if (left > k) {
      load8<T, WIDE>(p + k, 8, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) b[4 * j + i] = e4m3x2_f16(fp8_codes2(v[2 * i], v[2 * i + 1], s));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) b[4 * j + i] = 0;
    }
  }
  return __fdiv_rn(1.f, s);
}

__device__ __forceinline__ float add_scaled(float p, float w, float x, float acc) {
  return fmaf(p * scale_before(w, x), scale_after(w, x), acc);
}

// (Two passes with two blocks per SM, 64 registers a thread, spill: 9 x 2048 x 1536 pairs 5.5 us for 4.6.)
template <bool PAIR, int PASSES>
__global__ void __launch_bounds__(kThreads, PASSES == 1 ? 2 : 1) fp8_rows_kernel(const Fp8LinearArgs a, const bool wide) {
  __shared__ float4 part[kWarps][PASSES][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_trigger();
  const int n0 = blockIdx.x * (PAIR ? 8 : 16);
  // the lane's weight rows (past the end: the last one, not stored)
  const int r0 = min(n0 + g, a.out_n - 1), r1 = PAIR ? a.out_n + r0 : min(n0 + 8 + g, a.N - 1);
  const uint8_t *w0 = a.w + (int64_t)r0 * a.K + 16 * t, *w1 = a.w + (int64_t)r1 * a.K + 16 * t;
  const float *s0 = a.ws + (int64_t)(r0 / 128) * a.groups, *s1 = a.ws + (int64_t)(r1 / 128) * a.groups;
  float acc[PASSES][4] = {};
  for (int grp = warp; grp < a.groups; grp += kWarps) {
    const int k = 128 * grp, left = a.K - k;
    uint4 u[2], v[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const bool in = left > 64 * q + 16 * t;
      u[q] = in ? __ldg((const uint4*)(w0 + k + 64 * q)) : make_uint4(0, 0, 0, 0);
      v[q] = in ? __ldg((const uint4*)(w1 + k + 64 * q)) : make_uint4(0, 0, 0, 0);
    }
    const float f0 = __ldg(s0 + grp), f1 = __ldg(s1 + grp);
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
      const int row = min(kPass * pass + g, a.T - 1);  // the lane's row of x (past the end: the last one, not stored)
      uint32_t b[16];
      float sx;
      if (a.x_dtype == MOE_DT_E4M3) {
        const uint8_t* p = (const uint8_t*)a.x + row * a.ldx + k + 16 * t;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint4 c = left > 64 * q + 16 * t ? *(const uint4*)(p + 64 * q) : make_uint4(0, 0, 0, 0);
          const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) b[8 * q + 2 * j] = e4m3x2_f16(cw[j]), b[8 * q + 2 * j + 1] = e4m3x2_f16(cw[j] >> 16);
        }
        sx = a.qs[(int64_t)row * a.groups + grp];
      } else if (a.x_dtype == MOE_DT_F32) {
        const float* p = (const float*)a.x + row * a.ldx + k;
        sx = wide ? quantize_group<float, true>(p, left, t, b) : quantize_group<float, false>(p, left, t, b);
      } else if (a.x_dtype == MOE_DT_F16) {
        const __half* p = (const __half*)a.x + row * a.ldx + k;
        sx = wide ? quantize_group<__half, true>(p, left, t, b) : quantize_group<__half, false>(p, left, t, b);
      } else {
        const __nv_bfloat16* p = (const __nv_bfloat16*)a.x + row * a.ldx + k;
        sx = wide ? quantize_group<__nv_bfloat16, true>(p, left, t, b) : quantize_group<__nv_bfloat16, false>(p, left, t, b);
      }
      float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t c0[4] = {u[q].x, u[q].y, u[q].z, u[q].w}, c1[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma(p, e4m3x2_f16(c0[j]), e4m3x2_f16(c1[j]), e4m3x2_f16(c0[j] >> 16), e4m3x2_f16(c1[j] >> 16), b[8 * q + 2 * j], b[8 * q + 2 * j + 1]);
      }
      // columns 2 t and 2 t + 1 of the MMA are rows of x that lanes 4 (2 t) and 4 (2 t + 1) quantized
      const float x0 = __shfl_sync(0xffffffffu, sx, 8 * t), x1 = __shfl_sync(0xffffffffu, sx, 8 * t + 4);
      acc[pass][0] = add_scaled(p[0], f0, x0, acc[pass][0]), acc[pass][1] = add_scaled(p[1], f0, x1, acc[pass][1]);
      acc[pass][2] = add_scaled(p[2], f1, x0, acc[pass][2]), acc[pass][3] = add_scaled(p[3], f1, x1, acc[pass][3]);
    }
  }
#pragma unroll
  for (int pass = 0; pass < PASSES; ++pass) part[warp][pass][lane] = make_float4(acc[pass][0], acc[pass][1], acc[pass][2], acc[pass][3]);
  __syncthreads();
  if (threadIdx.x >= 128 * PASSES) return;
  // thread i: value i % 4 of lane i / 4, 128 for each pass
  const int used = min(kWarps, a.groups), pass = threadIdx.x / 128, l = threadIdx.x >> 2 & 31, i = threadIdx.x & 3;
  float y = 0.f;
  for (int w = 0; w < used; ++w) y += ((const float*)&part[w][pass][l])[i];
  const int token = kPass * pass + 2 * (l & 3) + (i & 1);
  if (PAIR) {  // values 0 and 1 are gates, 2 and 3 the same features' ups
    const float up = __shfl_down_sync(0xffffffffu, y, 2);
    const int n = n0 + (l >> 2);
    if (i < 2 && token < a.T && n < a.out_n) {
      y = silu_mul(y, up);
      if (a.base) y += load_any(a.base, a.out_dtype, token * a.ldb + n);
      store_any(a.out, a.out_dtype, token * a.ldo + n, y);
    }
  } else {
    const int n = n0 + (l >> 2) + 8 * (i >> 1);
    if (token < a.T && n < a.out_n) {
      if (a.base) y += load_any(a.base, a.out_dtype, token * a.ldb + n);
      store_any(a.out, a.out_dtype, token * a.ldo + n, y);
    }
  }
}

}  // namespace

cudaError_t launch_fp8_rows(const Fp8LinearArgs& a, cudaStream_t s) {
  const size_t es = a.x_dtype == MOE_DT_F32 ? 4 : 2;
  const bool pair = a.out_n != a.N, wide = (uintptr_t)a.x % 16 == 0 && a.ldx * es % 16 == 0;
  note_launches(1);
  const dim3 grid((a.out_n + (pair ? 7 : 15)) / (pair ? 8 : 16));
  if (a.T <= kPass)
    return pair ? launch_pdl(fp8_rows_kernel<true, 1>, grid, dim3(kThreads), 0, s, a, wide)
                : launch_pdl(fp8_rows_kernel<false, 1>, grid, dim3(kThreads), 0, s, a, wide);
  return pair ? launch_pdl(fp8_rows_kernel<true, 2>, grid, dim3(kThreads), 0, s, a, wide)
              : launch_pdl(fp8_rows_kernel<false, 2>, grid, dim3(kThreads), 0, s, a, wide);
}

}  // namespace moe
