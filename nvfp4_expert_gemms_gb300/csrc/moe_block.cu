// The norms before and after a block with its gate and residual scales.
//
//   enter:  y = norm(x)
//   leave:  out = alpha x + beta g(gate) post(block),   y = next(out)
//
// One pass: every row's x and block are read once into registers, the statistics are reduced over
// the threads that share the row, and out and y are written from the same registers.  All arithmetic
// is fp32; y is taken from out's value before it is rounded to the stream's type.  The variance of a
// layer norm is the mean of squared differences from the mean (a second reduction over registers),
// so a row with a large mean keeps its variance.
//
// Bound: HBM bytes (x, block, out, y once each).
#include "moe_block.cuh"

namespace moe {
namespace {

// Sum over the threads of one row: a warp, or the whole block through shared memory.  `red` has two
// buffers used in turn, so that one barrier per sum is enough: a buffer is written again only after
// every thread has passed the barrier of the sum in between, hence has read it.
struct RowSum {
  float (*red)[32];
  int warps, phase = 0;
  __device__ __forceinline__ float operator()(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* r = red[phase];
    phase ^= 1;
    if (lane == 0) r[warp] = v;
    __syncthreads();
    v = lane < warps ? r[lane] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  }
};

__device__ __forceinline__ float gate_value(float g, int act) {
  if (act == MOE_GATE_SIGMOID) return 1.f / (1.f + expf(-g));
  if (act == MOE_GATE_TANH) return tanhf(g);
  return g;
}

// Mean (LAYER only) and 1 / sqrt(mean square + eps) of a row held as v[N][V] by its threads; col(i)
// is the first column of piece i.
template <int V, int N>
__device__ __forceinline__ void row_stats(const float (&v)[N][V], const moe_norm_t& n, int H, int c0, int step,
                                          RowSum& sum, float& mean, float& rstd) {
  mean = 0.f;
  const float inv = 1.f / (float)H;
  if (n.kind == MOE_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c0 + i * step < H)
#pragma unroll
        for (int j = 0; j < V; ++j) s += v[i][j];
    mean = sum(s) * inv;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (c0 + i * step < H)
#pragma unroll
      for (int j = 0; j < V; ++j) q += (v[i][j] - mean) * (v[i][j] - mean);
  rstd = rsqrtf(sum(q) * inv + n.eps);
}

template <int V>
__device__ __forceinline__ void apply_norm(float* v, const moe_norm_t& n, int c, float mean, float rstd) {
  float w[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = (v[j] - mean) * rstd;
  if (n.weight) {
    load_any<V>(n.weight, n.dtype, c, w);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] *= w[j] + n.weight_offset;
  }
  if (n.bias) {
    load_any<V>(n.bias, n.dtype, c, w);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] += w[j];
  }
}

// A row per `tpr` threads (tpr = 32: one warp each; else the whole block), N pieces of V columns per
// thread: tpr * N * V >= H.
template <typename X, typename A, int V, int N, bool LEAVE>
__global__ void __launch_bounds__(1024) block_rows_kernel(const BlockArgs a, int tpr) {
  __shared__ float red[2][32];
  const int lane = threadIdx.x % tpr;
  const int t = blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
  pdl_wait();
  pdl_trigger();
  if (t >= a.T) return;  // whole warps, and only where a row is one warp
  RowSum sum{red, tpr / 32};
  const int H = a.H, c0 = lane * V, step = tpr * V;
  Pack<X, V> xp[N];
  const X* x = (const X*)a.x + (int64_t)t * a.ldx;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (c0 + i * step < H) xp[i] = load_pack<X, V>(x + c0 + i * step);
  float v[N][V], mean, rstd;
  if constexpr (LEAVE) {
    Pack<A, V> bp[N];
    const A* b = (const A*)a.block + (int64_t)t * a.ldb;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c0 + i * step < H) bp[i] = load_pack<A, V>(b + c0 + i * step);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = c0 + i * step < H ? to_f32(bp[i].e[j]) : 0.f;
    if (a.post.kind) row_stats<V, N>(v, a.post, H, c0, step, sum, mean, rstd);
    X* out = (X*)a.out + (int64_t)t * a.ldo;
    float gt = 1.f;
    if (a.gate && a.gate_step == 0) {
      load_any<1>(a.gate, a.gate_dtype, (int64_t)t * a.gate_ld, &gt);
      gt = gate_value(gt, a.gate_act);
    }
    gt *= a.beta;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i * step;
      if (c < H) {
        if (a.post.kind) apply_norm<V>(v[i], a.post, c, mean, rstd);
        if (a.gate && a.gate_step) {
          float g[V];
          load_any<V>(a.gate, a.gate_dtype, (int64_t)t * a.gate_ld + c, g);
#pragma unroll
          for (int j = 0; j < V; ++j) v[i][j] *= gate_value(g[j], a.gate_act);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = a.alpha * to_f32(xp[i].e[j]) + gt * v[i][j];
        store_pack<X, V>(out + c, v[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = c0 + i * step < H ? to_f32(xp[i].e[j]) : 0.f;
  }
  if (a.next.kind) {
    row_stats<V, N>(v, a.next, H, c0, step, sum, mean, rstd);
    A* y = (A*)a.y + (int64_t)t * a.ldy;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i * step;
      if (c < H) {
        apply_norm<V>(v[i], a.next, c, mean, rstd);
        store_pack<A, V>(y + c, v[i]);
      }
    }
  }
}

// Rows too long for one block's registers: the row's values are computed again from x and block (by
// now in L2) for each of its sums.  A thread visits the same columns every time and writes out and y
// only in the last visit, so out may be x and y may be block.
template <typename X, typename A, bool LEAVE>
__global__ void __launch_bounds__(1024) block_long_kernel(const BlockArgs a) {
  __shared__ float red[2][32];
  const int64_t t = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  RowSum sum{red, (int)blockDim.x / 32};
  const int H = a.H;
  const float inv = 1.f / (float)H;
  const X* x = (const X*)a.x + t * a.ldx;
  const A* b = LEAVE ? (const A*)a.block + t * a.ldb : nullptr;
  float pm = 0.f, pr = 1.f, gt = 1.f;
  if constexpr (LEAVE) {
    if (a.post.kind) {
      float s = 0.f;
      if (a.post.kind == MOE_NORM_LAYER) {
        for (int c = threadIdx.x; c < H; c += blockDim.x) s += to_f32(b[c]);
        pm = sum(s) * inv;
      }
      s = 0.f;
      for (int c = threadIdx.x; c < H; c += blockDim.x) s += (to_f32(b[c]) - pm) * (to_f32(b[c]) - pm);
      pr = rsqrtf(sum(s) * inv + a.post.eps);
    }
    if (a.gate && a.gate_step == 0) {
      load_any<1>(a.gate, a.gate_dtype, t * a.gate_ld, &gt);
      gt = gate_value(gt, a.gate_act);
    }
    gt *= a.beta;
  }
  auto value = [&](int c) {
    if constexpr (LEAVE) {
      float v = to_f32(b[c]), g;
      if (a.post.kind) apply_norm<1>(&v, a.post, c, pm, pr);
      if (a.gate && a.gate_step) {
        load_any<1>(a.gate, a.gate_dtype, t * a.gate_ld + c, &g);
        v *= gate_value(g, a.gate_act);
      }
      return a.alpha * to_f32(x[c]) + gt * v;
    } else {
      return to_f32(x[c]);
    }
  };
  float mean = 0.f, rstd = 1.f;
  if (a.next.kind) {
    float s = 0.f;
    if (a.next.kind == MOE_NORM_LAYER) {
      for (int c = threadIdx.x; c < H; c += blockDim.x) s += value(c);
      mean = sum(s) * inv;
    }
    s = 0.f;
    for (int c = threadIdx.x; c < H; c += blockDim.x) {
      const float d = value(c) - mean;
      s += d * d;
    }
    rstd = rsqrtf(sum(s) * inv + a.next.eps);
  }
  for (int c = threadIdx.x; c < H; c += blockDim.x) {
    float v = value(c);
    if constexpr (LEAVE) store_pack<X, 1>((X*)a.out + t * a.ldo + c, &v);
    if (a.next.kind) {
      apply_norm<1>(&v, a.next, c, mean, rstd);
      store_pack<A, 1>((A*)a.y + t * a.ldy + c, &v);
    }
  }
}

template <typename X, typename A, int V, int N, bool LEAVE>
cudaError_t launch_rows(const BlockArgs& a, cudaStream_t s) {
  const int pieces = (a.H + V - 1) / V;
  const int tpr = ((pieces + N - 1) / N + 31) / 32 * 32;
  const int threads = tpr == 32 ? 128 : tpr, rows = threads / tpr;
  return launch_pdl(block_rows_kernel<X, A, V, N, LEAVE>, dim3((a.T + rows - 1) / rows), dim3(threads), 0, s, a, tpr);
}

template <typename X, typename A, bool LEAVE>
cudaError_t launch_typed(const BlockArgs& a, bool wide, cudaStream_t s) {
  if (wide) {
    const int pieces = (a.H + 7) / 8;
    if (pieces <= 1024) return launch_rows<X, A, 8, 1, LEAVE>(a, s);
    if (pieces <= 4096) return launch_rows<X, A, 8, 4, LEAVE>(a, s);
  } else {
    if (a.H <= 1024) return launch_rows<X, A, 1, 2, LEAVE>(a, s);
    if (a.H <= 8192) return launch_rows<X, A, 1, 8, LEAVE>(a, s);
  }
  return launch_pdl(block_long_kernel<X, A, LEAVE>, dim3(a.T), dim3(1024), 0, s, a);
}

bool aligned16(const void* p, int64_t ld, size_t size) {
  return (uintptr_t)p % 16 == 0 && (ld * (int64_t)size) % 16 == 0;
}

}  // namespace

cudaError_t launch_block(const BlockArgs& a, int x_dtype, int act_dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const size_t sx = dtype_size(x_dtype), sa = dtype_size(act_dtype);
  const bool leave = a.block != nullptr;
  // 16-byte pieces of 8 columns (two per piece in fp32) where every tensor's rows allow them
  bool wide = a.H % 8 == 0 && aligned16(a.x, a.ldx, sx);
  if (leave) wide = wide && aligned16(a.block, a.ldb, sa) && aligned16(a.out, a.ldo, sx);
  if (a.next.kind) wide = wide && aligned16(a.y, a.ldy, sa);
  if (leave && a.gate && a.gate_step) wide = wide && aligned16(a.gate, a.gate_ld, dtype_size(a.gate_dtype));
  for (const moe_norm_t* n : {&a.post, &a.next})
    if (n->kind) wide = wide && (uintptr_t)n->weight % 16 == 0 && (uintptr_t)n->bias % 16 == 0;
  note_launches(1);
#define MOE_BLOCK(DX, X, DA, A) \
  if (x_dtype == DX && act_dtype == DA) return leave ? launch_typed<X, A, true>(a, wide, s) : launch_typed<X, A, false>(a, wide, s)
  MOE_BLOCK(MOE_DT_BF16, __nv_bfloat16, MOE_DT_BF16, __nv_bfloat16);
  MOE_BLOCK(MOE_DT_F16, __half, MOE_DT_F16, __half);
  MOE_BLOCK(MOE_DT_F32, float, MOE_DT_F32, float);
  MOE_BLOCK(MOE_DT_F32, float, MOE_DT_BF16, __nv_bfloat16);
  MOE_BLOCK(MOE_DT_F32, float, MOE_DT_F16, __half);
#undef MOE_BLOCK
  return cudaErrorInvalidValue;  // refused by the entry points before
}

namespace {

bool norm_ok(const moe_norm_t* n) {
  if (n->kind != MOE_NORM_RMS && n->kind != MOE_NORM_LAYER) return false;
  if (!(n->eps > 0.f)) return false;  // NaN too
  if (!n->weight && !n->bias) return true;
  return dtype_ok(n->dtype) && (uintptr_t)n->weight % dtype_size(n->dtype) == 0 &&
         (uintptr_t)n->bias % dtype_size(n->dtype) == 0;
}

bool matrix_ok(const void* p, int64_t ld, int dt, int H) { return p && ld >= H && (uintptr_t)p % dtype_size(dt) == 0; }

// The stream's type and the block's: the same, or an fp32 stream.
bool types_ok(int x, int act) { return x == act || x == MOE_DT_F32; }

}  // namespace
}  // namespace moe

extern "C" {

using namespace moe;

moe_status_t moe_block_enter(const void* x, int64_t ldx, int x_dtype, const moe_norm_t* norm, void* y, int64_t ldy,
                             int y_dtype, int T, int H, moe_stream_t stream) {
  if (T < 0 || H < 1 || !norm || !norm_ok(norm) || !dtype_ok(x_dtype) || !dtype_ok(y_dtype)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!matrix_ok(x, ldx, x_dtype, H) || !matrix_ok(y, ldy, y_dtype, H))) return MOE_ERR_INVALID_ARG;
  if (!types_ok(x_dtype, y_dtype)) return MOE_ERR_UNSUPPORTED;
  const moe_status_t dv = device_ok();
  if (dv != MOE_OK) return dv;
  BlockArgs a = {};
  a.x = x;
  a.y = y;
  a.ldx = ldx;
  a.ldy = ldy;
  a.next = *norm;
  a.T = T;
  a.H = H;
  return launch_block(a, x_dtype, y_dtype, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t moe_block_leave(const void* x, int64_t ldx, int x_dtype, const void* block, int64_t ldb, int act_dtype,
                             const moe_norm_t* post, const void* gate, int64_t gate_ld, int gate_step, int gate_dtype,
                             int gate_act, float alpha, float beta, const moe_norm_t* next, void* out, int64_t ldo,
                             void* y, int64_t ldy, int T, int H, moe_stream_t stream) {
  if (T < 0 || H < 1 || !dtype_ok(x_dtype) || !dtype_ok(act_dtype)) return MOE_ERR_INVALID_ARG;
  if ((post && !norm_ok(post)) || (next && !norm_ok(next))) return MOE_ERR_INVALID_ARG;
  if (gate) {
    if (!dtype_ok(gate_dtype) || gate_act < MOE_GATE_LINEAR || gate_act > MOE_GATE_TANH) return MOE_ERR_INVALID_ARG;
    if ((gate_step != 0 && gate_step != 1) || gate_ld < 0 || (uintptr_t)gate % dtype_size(gate_dtype) != 0)
      return MOE_ERR_INVALID_ARG;
  }
  if (T > 0 && (!matrix_ok(x, ldx, x_dtype, H) || !matrix_ok(block, ldb, act_dtype, H) ||
                !matrix_ok(out, ldo, x_dtype, H) || (next && !matrix_ok(y, ldy, act_dtype, H))))
    return MOE_ERR_INVALID_ARG;
  if (!types_ok(x_dtype, act_dtype)) return MOE_ERR_UNSUPPORTED;
  const moe_status_t dv = device_ok();
  if (dv != MOE_OK) return dv;
  BlockArgs a = {};
  a.x = x;
  a.block = block;
  a.gate = gate;
  a.out = out;
  a.y = next ? y : nullptr;
  a.ldx = ldx;
  a.ldb = ldb;
  a.ldo = ldo;
  a.ldy = ldy;
  a.gate_ld = gate_ld;
  if (post) a.post = *post;
  if (next) a.next = *next;
  a.gate_step = gate_step;
  a.gate_dtype = gate_dtype;
  a.gate_act = gate_act;
  a.alpha = alpha;
  a.beta = beta;
  a.T = T;
  a.H = H;
  return launch_block(a, x_dtype, act_dtype, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
