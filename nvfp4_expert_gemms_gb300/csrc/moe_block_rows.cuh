// The norms before and after a block with its gate and residual scales: the kernels.  One source file per
// pair of stream and block types (moe_block_*.cu) instantiates them.
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
// Bound: HBM bytes (x, block, out, y once each).  16384 x 2048, both norms, a gate per channel: fp32 stream and
// bf16 block 67.4 us, 5.97 TB/s (60.2 us at the copy rate), all bf16 46.5 us (40.1); 2000 x 8192 bf16 28.1 us
// (19.6); rows of 1999 fp16 with padded pitches, two layer norms and a tanh per element, 1237 of them: 11.6 us
// (3.7; there 109 instructions per element bound it).
#pragma once
#include <type_traits>

#include "moe_block.cuh"
#include "moe_tc.cuh"

namespace moe {
namespace {

constexpr int64_t kStreamSize = 1216 * 2048;  // elements from which blocks walk over rows (below: a block per row)
// Shared memory and threads of such a block: two per SM (rows of up to 4096 columns), or one.
template <int W, int N>
constexpr int kStreamSmem = (W * N > 16 ? 226 : 113) * 1024;
template <int N>
constexpr int kStreamThreads = N <= 2 ? 512 : 256;

// Sum over the threads of one row: a warp, or the whole block through shared memory.  `red` has two
// buffers used in turn, so that one barrier per sum is enough: a buffer is written again only after
// every thread has passed the barrier of the sum in between, hence has read it.  Entries past the last
// warp's are zero.
struct RowSum {
  float (*red)[32];
  int warps, phase = 0;
  __device__ __forceinline__ RowSum(float (*r)[32], int w) : red(r), warps(w) {
    if (warps > 1 && threadIdx.x < 64) (&red[0][0])[threadIdx.x] = 0.f;
    if (warps > 1) __syncthreads();
  }
  __device__ __forceinline__ float operator()(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (warps == 1) return v;
    float* r = red[phase];
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < warps; w += 8) {
      const float4 a = *(const float4*)(r + w), b = *(const float4*)(r + w + 4);
      s += ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
    }
    return s;
  }
};

__device__ __forceinline__ float gate_value(float g, int act) {
  if (act == MOE_GATE_SIGMOID) return 1.f / (1.f + expf(-g));
  if (act == MOE_GATE_TANH) return tanhf(g);
  return g;
}

// ---- two fp32 values per operation -------------------------------------------------------------
struct F2 {
  float x, y;
};
__device__ __forceinline__ uint64_t bits(F2 a) { return *(const uint64_t*)&a; }
__device__ __forceinline__ F2 from_bits(uint64_t b) { return *(const F2*)&b; }
__device__ __forceinline__ F2 dup(float a) { return F2{a, a}; }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return from_bits(r);
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return from_bits(r);
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return from_bits(r);
}
__device__ __forceinline__ F2 widen2(uint32_t w, __nv_bfloat16) {
  return F2{__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)};
}
__device__ __forceinline__ F2 widen2(uint32_t w, __half) {
  const float2 f = __half22float2(*(const __half2*)&w);
  return F2{f.x, f.y};
}
__device__ __forceinline__ uint32_t narrow2(F2 v, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *(const uint32_t*)&h;
}
__device__ __forceinline__ uint32_t narrow2(F2 v, __half) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *(const uint32_t*)&h;
}

// 8 columns of a row: as 16-byte pieces (one, or two of fp32) and as four pairs of values.
template <typename E>
constexpr int kPieces = sizeof(E) / 2;
template <typename E>
__device__ __forceinline__ void widen8(const uint4 (&q)[kPieces<E>], F2 (&v)[4]) {
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = F2{__uint_as_float(q[i].x), __uint_as_float(q[i].y)};
      v[2 * i + 1] = F2{__uint_as_float(q[i].z), __uint_as_float(q[i].w)};
    }
  } else {
    v[0] = widen2(q[0].x, E());
    v[1] = widen2(q[0].y, E());
    v[2] = widen2(q[0].z, E());
    v[3] = widen2(q[0].w, E());
  }
}
// Eight fp32 columns move in one 32-byte access (p 32-byte aligned): as two of 16 bytes, each would
// touch every 32-byte sector of the warp's kilobyte and use half of it.
__device__ __forceinline__ void load_pieces(const void* p, uint4 (&q)[2]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(q[0].x), "=r"(q[0].y), "=r"(q[0].z), "=r"(q[0].w), "=r"(q[1].x), "=r"(q[1].y), "=r"(q[1].z),
                 "=r"(q[1].w)
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void load_pieces(const void* p, uint4 (&q)[1]) { q[0] = *(const uint4*)p; }
template <typename E>
__device__ __forceinline__ void load8(const E* p, F2 (&v)[4]) {
  uint4 q[kPieces<E>];
  load_pieces(p, q);
  widen8<E>(q, v);
}
template <typename E>
__device__ __forceinline__ void store8(E* p, const F2 (&v)[4]) {
  if constexpr (sizeof(E) == 4) {
    const uint32_t w[8] = {__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                           __float_as_uint(v[1].y), __float_as_uint(v[2].x), __float_as_uint(v[2].y),
                           __float_as_uint(v[3].x), __float_as_uint(v[3].y)};
    tc::st_global_v8(p, w);
  } else {
    *(uint4*)p = make_uint4(narrow2(v[0], E()), narrow2(v[1], E()), narrow2(v[2], E()), narrow2(v[3], E()));
  }
}
__device__ __forceinline__ void gate8(F2 (&g)[4], int act) {
  if (act == MOE_GATE_LINEAR) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) g[j] = F2{gate_value(g[j].x, act), gate_value(g[j].y, act)};
}

// Column factors: what a column is multiplied by in every row.  post: its weight, beta and a gate per
// channel; next: its weight.
template <typename P>
__device__ __forceinline__ void post_factor(const BlockArgs& a, bool channel_gate, int c, F2 (&f)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = dup(1.f);
  if (a.post.kind && a.post.weight) {
    load8((const P*)a.post.weight + c, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = add2(f[j], dup(a.post.weight_offset));
  }
  if (channel_gate) {
    F2 g[4];
    load8((const P*)a.gate + c, g);
    gate8(g, a.gate_act);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = mul2(f[j], g[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = mul2(f[j], dup(a.beta));
}
template <typename P>
__device__ __forceinline__ void next_factor(const BlockArgs& a, int c, F2 (&f)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = dup(1.f);
  if (a.next.kind && a.next.weight) {
    load8((const P*)a.next.weight + c, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = add2(f[j], dup(a.next.weight_offset));
  }
}

// A row v (zero past its end): LAYER subtracts the mean; returns 1 / sqrt(mean square + eps).
template <int N, class Sum>
__device__ __forceinline__ float center_and_scale(F2 (&v)[N][4], const moe_norm_t& n, int H, int c0, int step,
                                                  Sum& sum) {
  const float inv = 1.f / (float)H;
  if (n.kind == MOE_NORM_LAYER) {
    F2 s[4] = {v[0][0], v[0][1], v[0][2], v[0][3]};
#pragma unroll
    for (int i = 1; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = add2(s[j], v[i][j]);
    const F2 all = add2(add2(s[0], s[1]), add2(s[2], s[3]));
    const F2 minus_mean = dup(-sum(all.x + all.y) * inv);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c0 + i * step < H)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = add2(v[i][j], minus_mean);
  }
  F2 q[4] = {mul2(v[0][0], v[0][0]), mul2(v[0][1], v[0][1]), mul2(v[0][2], v[0][2]), mul2(v[0][3], v[0][3])};
#pragma unroll
  for (int i = 1; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = fma2(v[i][j], v[i][j], q[j]);
  const F2 all = add2(add2(q[0], q[1]), add2(q[2], q[3]));
  return rsqrtf(sum(all.x + all.y) * inv + n.eps);
}

// The general form of eight columns' way back: v = rstd f v + beta g bias, times a full gate, times the
// token's gate gt, plus alpha x.  (Without a bias and a full gate it is alpha x + (rstd gt) f v.)
template <typename P>
__device__ __forceinline__ void leave_general(const BlockArgs& a, bool channel_gate, const P* bias, bool full_gate,
                                              F2 (&full)[4], int c, float rstd, float gt, const F2 (&x)[4], F2 (&v)[4]) {
  F2 u[4], g[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], dup(rstd));
  if (bias) {
    load8(bias + c, u);
    if (channel_gate) {
      load8((const P*)a.gate + c, g);
      gate8(g, a.gate_act);
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = mul2(u[j], g[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = fma2(u[j], dup(a.beta), v[j]);
  }
  if (full_gate) {
    gate8(full, a.gate_act);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], full[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = fma2(v[j], dup(gt), mul2(dup(a.alpha), x[j]));
}

// Rows that allow eight columns per access, few of them: a row per block (a thread per 8 columns, rounded up
// to warps).  All of a row's loads, the parameters' too, are issued before its first sum.  Against the kernel
// below: 304 x 2048 fp32 / bf16 3.4 us (4.4), 1216 rows 6.9 (5.7 with four pieces per lane), 16384 rows 74.5 (66.9).
template <typename X, typename A, typename P, bool LEAVE>
__global__ void __launch_bounds__(512) block_row_kernel(const BlockArgs a) {
  constexpr int N = 1;
  __shared__ __align__(16) float red[2][32];
  const int H = a.H, c0 = threadIdx.x * 8, step = blockDim.x * 8;
  const int64_t t = blockIdx.x;
  const P *pb = (const P*)a.post.bias, *nb = (const P*)a.next.bias, *gate = (const P*)a.gate;
  const bool full_gate = LEAVE && gate && a.gate_step && a.gate_ld, token_gate = LEAVE && gate && !a.gate_step;
  const bool channel_gate = LEAVE && gate && a.gate_step && !a.gate_ld;
  pdl_wait();
  pdl_trigger();
  uint4 xq[N][kPieces<X>], bq[N][kPieces<A>], gq[N][kPieces<P>];
  F2 pf[N][4], nf[N][4];
  float gt = 1.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = c0 + i * step;
    if (c < H) {
      load_pieces((const X*)a.x + t * a.ldx + c, xq[i]);
      if constexpr (LEAVE) {
        load_pieces((const A*)a.block + t * a.ldb + c, bq[i]);
        if (full_gate) load_pieces(gate + t * a.gate_ld + c, gq[i]);
      }
    }
  }
  if (token_gate) gt = to_f32(gate[t * a.gate_ld]);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (c0 + i * step < H) {
      if constexpr (LEAVE) post_factor<P>(a, channel_gate, c0 + i * step, pf[i]);
      next_factor<P>(a, c0 + i * step, nf[i]);
    }
  RowSum sum(red, blockDim.x / 32);
  F2 v[N][4];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (c0 + i * step < H) {
      if constexpr (LEAVE) widen8<A>(bq[i], v[i]);
      else widen8<X>(xq[i], v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = dup(0.f);
    }
  }
  if constexpr (LEAVE) {
    float rstd = 1.f;
    if (a.post.kind) rstd = center_and_scale<N>(v, a.post, H, c0, step, sum);
    if (token_gate) gt = gate_value(gt, a.gate_act);
    X* out = (X*)a.out + t * a.ldo;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i * step;
      if (c < H) {
        F2 x[4], g[4];
        widen8<X>(xq[i], x);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = mul2(v[i][j], pf[i][j]);
        if (!pb && !full_gate) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = fma2(v[i][j], dup(rstd * gt), mul2(dup(a.alpha), x[j]));
        } else {
          if (full_gate) widen8<P>(gq[i], g);
          leave_general<P>(a, channel_gate, pb, full_gate, g, c, rstd, gt, x, v[i]);
        }
        store8(out + c, v[i]);
      }
    }
  }
  if (a.next.kind) {
    const F2 rstd = dup(center_and_scale<N>(v, a.next, H, c0, step, sum));
    A* y = (A*)a.y + t * a.ldy;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i * step;
      if (c < H) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = mul2(mul2(v[i][j], rstd), nf[i][j]);
        if (nb) {
          F2 u[4];
          load8(nb + c, u);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = add2(v[i][j], u[j]);
        }
        store8(y + c, v[i]);
      }
    }
  }
}

// Sum over a group of W warps, as RowSum; the group's named barrier is 1 + group.
template <int W>
struct GroupSum {
  float (*red)[W < 4 ? 4 : W];
  int group, phase = 0;
  __device__ __forceinline__ float operator()(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if constexpr (W == 1) return v;
    float* r = red[phase];
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x / 32 % W] = v;
    tc::named_bar_sync(1 + group, 32 * W);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) s += r[k];
    return s;
  }
};

// The same, many rows: a group of W warps per row (N pieces of 8 columns per lane, 256 W N >= H), groups
// walking the rows with the grid's stride.  A warp copies its own columns of the next row's x, block and
// per-element gate into shared memory (cp.async, two slots) while it works on the current one, so the
// bytes in flight cost no registers; x waits there until it is added.  The column factors are in shared
// memory, fp32, one copy per block.
template <typename X, typename A, typename P, int W, int N, bool LEAVE>
__global__ void __launch_bounds__(kStreamThreads<N>, 2) block_stream_kernel(const BlockArgs a) {
  constexpr int G = 32 * W;  // threads of a row; 256 W columns per step of N
  constexpr int kX = kPieces<X>, kA = LEAVE ? kPieces<A> : 0, kG = LEAVE ? kPieces<P> : 0;
  extern __shared__ __align__(16) uint4 smem[];  // column factors [LEAVE ? 4 : 2][N G], then [groups][2][row]
  __shared__ __align__(16) float red[kStreamThreads<N> / G][2][W < 4 ? 4 : W];
  const int lane = threadIdx.x & 31, group = threadIdx.x / G, w = threadIdx.x / 32 % W, H = a.H;
  const P *pb = (const P*)a.post.bias, *nb = (const P*)a.next.bias, *gate = (const P*)a.gate;
  const bool full_gate = LEAVE && gate && a.gate_step && a.gate_ld, token_gate = LEAVE && gate && !a.gate_step;
  const bool channel_gate = LEAVE && gate && a.gate_step && !a.gate_ld;
  // rows are counted in 32 unsigned bits: a row past the last does not wrap for any T
  const uint32_t T = a.T, stride = gridDim.x * (blockDim.x / G);
  uint32_t t = blockIdx.x * (blockDim.x / G) + group;
  pdl_wait();
  pdl_trigger();
  const int slot = N * (kX + kA + (full_gate ? kG : 0)) * G;
  uint4* ring = smem + (LEAVE ? 4 : 2) * G * N + group * 2 * slot;
  auto fetch = [&](uint32_t row, int at) {
    if (row < T) {
      uint32_t dst = (uint32_t)__cvta_generic_to_shared(ring + at * slot);
      // A row's 16-byte pieces in memory order by lane, to shared memory in the same order: a copy whose two
      // halves of a 32-byte sector part would ask for the sector twice.
      auto pieces = [&](const auto* p) {
        constexpr int n = kPieces<std::remove_cv_t<std::remove_reference_t<decltype(*p)>>>;
#pragma unroll
        for (int i = 0; i < N; ++i, dst += 512 * n * W)
#pragma unroll
          for (int k = 0; k < n; ++k) {
            const int e = k * 32 + lane, c = (i * W + w) * 256 + e * (8 / n);
            const uint32_t to = dst + w * 512 * n + e * 16;
            if (c < H) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p + c) : "memory");
          }
      };
      pieces((const X*)a.x + row * a.ldx);
      if constexpr (LEAVE) {
        pieces((const A*)a.block + row * a.ldb);
        if (full_gate) pieces(gate + row * a.gate_ld);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(t, 0);
  float gt_next = 1.f;
  if (token_gate && t < T) gt_next = to_f32(gate[t * a.gate_ld]);
  for (int i = threadIdx.x; i * 8 < H; i += blockDim.x) {  // piece i: columns 8 i .. 8 i + 7
    F2 f[4];
    next_factor<P>(a, i * 8, f);
    ((float4*)smem)[i] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    ((float4*)smem)[G * N + i] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    if constexpr (LEAVE) {
      post_factor<P>(a, channel_gate, i * 8, f);
      ((float4*)smem)[2 * G * N + i] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
      ((float4*)smem)[3 * G * N + i] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    }
  }
  __syncthreads();
  auto factor = [&](int which, int i, F2 (&f)[4]) {
    const float4 p = ((const float4*)smem)[(2 * which) * G * N + (i * W + w) * 32 + lane];
    const float4 q = ((const float4*)smem)[(2 * which + 1) * G * N + (i * W + w) * 32 + lane];
    f[0] = F2{p.x, p.y};
    f[1] = F2{p.z, p.w};
    f[2] = F2{q.x, q.y};
    f[3] = F2{q.z, q.w};
  };
  GroupSum<W> sum{red[group], group};
  for (int at = 0; t < T; t += stride, at ^= 1) {
    __syncwarp();  // every lane has read the slot that is filled now
    fetch(t + stride, at ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();  // every lane's pieces have landed
    const uint4 *xs = ring + at * slot, *bs = xs + N * kX * G, *gs = bs + N * kA * G;
    F2 v[N][4];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if ((i * W + w) * 256 + lane * 8 < H) {
        if constexpr (LEAVE) {
          uint4 q[kPieces<A>];
#pragma unroll
          for (int k = 0; k < kA; ++k) q[k] = bs[((i * W + w) * 32 + lane) * kA + k];
          widen8<A>(q, v[i]);
        } else {
          uint4 q[kX];
#pragma unroll
          for (int k = 0; k < kX; ++k) q[k] = xs[((i * W + w) * 32 + lane) * kX + k];
          widen8<X>(q, v[i]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = dup(0.f);
      }
    }
    if constexpr (LEAVE) {
      float rstd = 1.f, gt = 1.f;
      if (token_gate) {
        gt = gate_value(gt_next, a.gate_act);
        if (t + stride < T) gt_next = to_f32(gate[(t + stride) * a.gate_ld]);
      }
      if (a.post.kind) rstd = center_and_scale<N>(v, a.post, H, w * 256 + lane * 8, 256 * W, sum);
      X* out = (X*)a.out + t * a.ldo;
      const bool plain = !pb && !full_gate;
      const F2 rg = dup(rstd * gt), al = dup(a.alpha);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * W + w) * 256 + lane * 8;
        if (c < H) {
          F2 f[4], x[4];
          uint4 q[kX];
#pragma unroll
          for (int k = 0; k < kX; ++k) q[k] = xs[((i * W + w) * 32 + lane) * kX + k];
          widen8<X>(q, x);
          factor(1, i, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = mul2(v[i][j], f[j]);
          if (plain) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = fma2(v[i][j], rg, mul2(al, x[j]));
          } else {
            F2 g[4];
            if (full_gate) {
              uint4 r[kPieces<P>];
#pragma unroll
              for (int k = 0; k < kG; ++k) r[k] = gs[((i * W + w) * 32 + lane) * kG + k];
              widen8<P>(r, g);
            }
            leave_general<P>(a, channel_gate, pb, full_gate, g, c, rstd, gt, x, v[i]);
          }
          store8(out + c, v[i]);
        }
      }
    }
    if (a.next.kind) {
      const F2 rstd = dup(center_and_scale<N>(v, a.next, H, w * 256 + lane * 8, 256 * W, sum));
      A* y = (A*)a.y + t * a.ldy;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * W + w) * 256 + lane * 8;
        if (c < H) {
          F2 f[4];
          factor(0, i, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = mul2(mul2(v[i][j], rstd), f[j]);
          if (nb) {
            load8(nb + c, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = add2(v[i][j], f[j]);
          }
          store8(y + c, v[i]);
        }
      }
    }
  }
}

// Rows of any length up to TPR * N and any alignment, one element at a time: a row per block of TPR
// threads (TPR = 32: four rows), columns TPR apart, so that addresses are one base and constants.  All of
// a row's loads, the parameters' too, are issued before its first sum.
template <typename X, typename A, typename P, int TPR, int N, bool LEAVE>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR) block_narrow_kernel(const BlockArgs a) {
  __shared__ __align__(16) float red[2][32];
  const int lane = threadIdx.x % TPR;
  const uint32_t t = blockIdx.x * (blockDim.x / TPR) + threadIdx.x / TPR;
  pdl_wait();
  pdl_trigger();
  RowSum sum(red, TPR / 32);
  if (t >= (uint32_t)a.T) return;
  const int H = a.H, n = (H - lane + TPR - 1) / TPR;  // the thread's columns: lane + i * TPR, i < n
  const float inv = 1.f / (float)H;
  const bool wide_gate = LEAVE && a.gate && a.gate_step;
  auto load = [&](auto (&r)[N], const auto* p) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) r[i] = p[i * TPR];
  };
  X x[N];
  load(x, (const X*)a.x + (int64_t)t * a.ldx + lane);
  A b[LEAVE ? N : 1];
  P w[N], g[N];
  float gt = 1.f;
  if constexpr (LEAVE) {
    load(b, (const A*)a.block + (int64_t)t * a.ldb + lane);
    if (wide_gate) load(g, (const P*)a.gate + (int64_t)t * a.gate_ld + lane);
    if (a.gate && !a.gate_step) gt = to_f32(((const P*)a.gate)[(int64_t)t * a.gate_ld]);
    if (a.post.kind && a.post.weight) load(w, (const P*)a.post.weight + lane);
  }
  float v[N];
  // v becomes norm(v); w holds its weight
  auto norm = [&](const moe_norm_t& nm) {
    if (nm.kind == MOE_NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) s += v[i];
      const float mean = sum(s) * inv;
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = i < n ? v[i] - mean : 0.f;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) q += v[i] * v[i];
    const float rstd = rsqrtf(sum(q) * inv + nm.eps);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= rstd;
    if (nm.weight) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < n) v[i] *= to_f32(w[i]) + nm.weight_offset;
    }
    if (nm.bias) {
      load(w, (const P*)nm.bias + lane);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < n) v[i] += to_f32(w[i]);
    }
  };
  if constexpr (LEAVE) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < n ? to_f32(b[i]) : 0.f;
    if (a.post.kind) norm(a.post);
    if (a.next.kind && a.next.weight) load(w, (const P*)a.next.weight + lane);
    if (a.gate && !a.gate_step) gt = gate_value(gt, a.gate_act);
    gt *= a.beta;
    if (wide_gate) {
      if (a.gate_act == MOE_GATE_TANH) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i < n) v[i] *= tanhf(to_f32(g[i]));
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i < n) v[i] *= gate_value(to_f32(g[i]), a.gate_act);
      }
    }
    X* out = (X*)a.out + (int64_t)t * a.ldo + lane;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) {
        v[i] = a.alpha * to_f32(x[i]) + gt * v[i];
        from_f32(v[i], out + i * TPR);
      }
  } else {
    if (a.next.kind && a.next.weight) load(w, (const P*)a.next.weight + lane);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < n ? to_f32(x[i]) : 0.f;
  }
  if (a.next.kind) {
    norm(a.next);
    A* y = (A*)a.y + (int64_t)t * a.ldy + lane;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) from_f32(v[i], y + i * TPR);
  }
}

// Rows that allow eight columns per access, too long for the kernels above: a row per block, its values kept as
// fp32 in shared memory (columns 8 p .. 8 p + 3 at [p], the next four at [H / 8 + p]: neighbours on neighbouring
// banks), so x and block are still read once.  A thread visits the same columns every time, so nothing but the
// sums needs a barrier, and out may be x and y may be block.  Two blocks per SM up to 28000 columns, so that one's
// loads run under the other's sums; one up to 57856.
//
// Both norms, a gate per channel, 4096 rows of bf16: 12288 columns 89.8 us (60.2 by HBM; the kernel below 448),
// 16384 110 us (80.3; 588), 32768, with one block, 316 us (160.5).  One row of 16384 6.3 us (28.5).
constexpr int kSharedThreads = 512, kSharedMost = 226 * 1024;

template <typename X, typename A, typename P, bool LEAVE>
__global__ void __launch_bounds__(kSharedThreads, 2) block_shared_kernel(const BlockArgs a) {
  extern __shared__ __align__(16) float4 row[];
  __shared__ __align__(16) float red[2][32];
  constexpr int U = 2;  // pieces whose loads are in flight together, beside those of the block's other warps
  const int H = a.H, pieces = H / 8;
  const int64_t t = blockIdx.x;
  const P *pb = (const P*)a.post.bias, *nb = (const P*)a.next.bias, *gate = (const P*)a.gate;
  const bool full_gate = LEAVE && gate && a.gate_step && a.gate_ld, token_gate = LEAVE && gate && !a.gate_step;
  const bool channel_gate = LEAVE && gate && a.gate_step && !a.gate_ld;
  pdl_wait();
  pdl_trigger();
  const X* x = (const X*)a.x + t * a.ldx;
  float gt = 1.f;
  if (token_gate) gt = to_f32(gate[t * a.gate_ld]);
  RowSum sum(red, kSharedThreads / 32);
  const float inv = 1.f / (float)H;
  auto get = [&](int p, F2 (&v)[4]) {
    const float4 q = row[p], r = row[pieces + p];
    v[0] = F2{q.x, q.y};
    v[1] = F2{q.z, q.w};
    v[2] = F2{r.x, r.y};
    v[3] = F2{r.z, r.w};
  };
  auto put = [&](int p, const F2 (&v)[4]) {
    row[p] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    row[pieces + p] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  };
  // A norm's sums over the row: `part` holds what the pass that wrote the row added up, of the values (LAYER) or
  // of their squares.  Returns -mean (0 without one) and 1 / sqrt(mean square + eps).
  F2 part[4];
  auto clear = [&] {
#pragma unroll
    for (int j = 0; j < 4; ++j) part[j] = dup(0.f);
  };
  auto add = [&](const moe_norm_t& n, const F2 (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) part[j] = n.kind == MOE_NORM_LAYER ? add2(part[j], v[j]) : fma2(v[j], v[j], part[j]);
  };
  auto total = [&] {
    const F2 all = add2(add2(part[0], part[1]), add2(part[2], part[3]));
    return sum(all.x + all.y) * inv;
  };
  auto stats = [&](const moe_norm_t& n, float& minus_mean) {
    minus_mean = 0.f;
    float q = total();
    if (n.kind == MOE_NORM_LAYER) {
      minus_mean = -q;
      clear();
      for (int p = threadIdx.x; p < pieces; p += kSharedThreads) {
        F2 v[4];
        get(p, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const F2 d = add2(v[j], dup(minus_mean));
          part[j] = fma2(d, d, part[j]);
        }
      }
      q = total();
    }
    return rsqrtf(q + n.eps);
  };
  float minus_mean = 0.f, rstd = 1.f;
  if constexpr (LEAVE) {
    if (token_gate) gt = gate_value(gt, a.gate_act);
    const A* b = (const A*)a.block + t * a.ldb;
    clear();
    for (int p0 = threadIdx.x; p0 < pieces; p0 += 2 * U * kSharedThreads) {
      uint4 q[2 * U][kPieces<A>];
#pragma unroll
      for (int u = 0; u < 2 * U; ++u)
        if (p0 + u * kSharedThreads < pieces) load_pieces(b + 8 * (p0 + u * kSharedThreads), q[u]);
#pragma unroll
      for (int u = 0; u < 2 * U; ++u) {
        const int p = p0 + u * kSharedThreads;
        if (p < pieces) {  // x is wanted after the sums
          asm volatile("prefetch.global.L2 [%0];" ::"l"(x + 8 * p));
          F2 v[4];
          widen8<A>(q[u], v);
          put(p, v);
          add(a.post, v);
        }
      }
    }
    if (a.post.kind) rstd = stats(a.post, minus_mean);
  }
  clear();
  for (int p0 = threadIdx.x; p0 < pieces; p0 += U * kSharedThreads) {
    uint4 q[U][kPieces<X>];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (p0 + u * kSharedThreads < pieces) load_pieces(x + 8 * (p0 + u * kSharedThreads), q[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = p0 + u * kSharedThreads;
      if (p >= pieces) continue;
      F2 v[4];
      if constexpr (LEAVE) {
        F2 xs[4], f[4];
        widen8<X>(q[u], xs);
        get(p, v);
        post_factor<P>(a, channel_gate, 8 * p, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = mul2(add2(v[j], dup(minus_mean)), f[j]);
        if (!pb && !full_gate) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = fma2(v[j], dup(rstd * gt), mul2(dup(a.alpha), xs[j]));
        } else {
          F2 g[4];
          if (full_gate) load8(gate + t * a.gate_ld + 8 * p, g);
          leave_general<P>(a, channel_gate, pb, full_gate, g, 8 * p, rstd, gt, xs, v);
        }
        store8((X*)a.out + t * a.ldo + 8 * p, v);
      } else {
        widen8<X>(q[u], v);
      }
      put(p, v);
      add(a.next, v);
    }
  }
  if (a.next.kind) {
    rstd = stats(a.next, minus_mean);
    A* y = (A*)a.y + t * a.ldy;
    for (int p = threadIdx.x; p < pieces; p += kSharedThreads) {
      F2 v[4], f[4];
      get(p, v);
      next_factor<P>(a, 8 * p, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = mul2(mul2(add2(v[j], dup(minus_mean)), dup(rstd)), f[j]);
      if (nb) {
        F2 u[4];
        load8(nb + 8 * p, u);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = add2(v[j], u[j]);
      }
      store8(y + 8 * p, v);
    }
  }
}

__device__ __forceinline__ void apply_norm(float* v, const moe_norm_t& n, int c, float mean, float rstd) {
  *v = (*v - mean) * rstd;
  if (n.weight) *v *= load_any(n.weight, n.dtype, c) + n.weight_offset;
  if (n.bias) *v += load_any(n.bias, n.dtype, c);
}

// Long rows that allow no eight columns per access, and calls whose parameters differ in type: one element at a
// time.  `keep`: the row's values stay in shared memory as fp32 between its sums; longer rows are computed again
// from x and block (by then in L2) each time.  A thread visits the same columns every time and writes out and y
// only in the last visit, so out may be x and y may be block.  Bound: instructions (types looked up per element).
// 4096 x 16385 bf16, both norms, a gate per channel: 433 us (80.3 by HBM; computed again 597; four elements in
// flight but one block per SM 628).
template <typename X, typename A, bool LEAVE>
__global__ void __launch_bounds__(1024, 2) block_long_kernel(const BlockArgs a, const bool keep) {
  extern __shared__ __align__(16) float4 row[];
  __shared__ __align__(16) float red[2][32];
  float* kept = (float*)row;
  const int64_t t = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  RowSum sum(red, (int)blockDim.x / 32);
  const int H = a.H;
  const float inv = 1.f / (float)H;
  const X* x = (const X*)a.x + t * a.ldx;
  const A* b = LEAVE ? (const A*)a.block + t * a.ldb : nullptr;
  float pm = 0.f, pr = 1.f, gt = 1.f;
  // The mean of f(c) over the row's columns.
  auto over = [&](auto f) {
    float s = 0.f;
#pragma unroll 2
    for (int c = threadIdx.x; c < H; c += 1024) s += f(c);
    return sum(s) * inv;
  };
  auto square = [](float v) { return v * v; };
  auto first = [&](int c, float v) {  // the first of a value's visits
    if (keep) kept[c] = v;
    return v;
  };
  if constexpr (LEAVE) {
    if (a.post.kind) {
      auto again = [&](int c) { return keep ? kept[c] : to_f32(b[c]); };
      float q;
      if (a.post.kind == MOE_NORM_LAYER) {
        pm = over([&](int c) { return first(c, to_f32(b[c])); });
        q = over([&](int c) { return square(again(c) - pm); });
      } else {
        q = over([&](int c) { return square(first(c, to_f32(b[c]))); });
      }
      pr = rsqrtf(q + a.post.eps);
    }
    if (a.gate && a.gate_step == 0) gt = gate_value(load_any(a.gate, a.gate_dtype, t * a.gate_ld), a.gate_act);
    gt *= a.beta;
  }
  auto value = [&](int c) {
    if constexpr (LEAVE) {
      float v = keep && a.post.kind ? kept[c] : to_f32(b[c]);
      if (a.post.kind) apply_norm(&v, a.post, c, pm, pr);
      if (a.gate && a.gate_step) v *= gate_value(load_any(a.gate, a.gate_dtype, t * a.gate_ld + c), a.gate_act);
      return a.alpha * to_f32(x[c]) + gt * v;
    } else {
      return to_f32(x[c]);
    }
  };
  auto again = [&](int c) { return keep && a.next.kind ? kept[c] : value(c); };
  float mean = 0.f, rstd = 1.f;
  if (a.next.kind) {
    float q;
    if (a.next.kind == MOE_NORM_LAYER) {
      mean = over([&](int c) { return first(c, value(c)); });
      q = over([&](int c) { return square(again(c) - mean); });
    } else {
      q = over([&](int c) { return square(first(c, value(c))); });
    }
    rstd = rsqrtf(q + a.next.eps);
  }
#pragma unroll 2
  for (int c = threadIdx.x; c < H; c += 1024) {
    float v = again(c);
    if constexpr (LEAVE) from_f32(v, (X*)a.out + t * a.ldo + c);
    if (a.next.kind) {
      apply_norm(&v, a.next, c, mean, rstd);
      from_f32(v, (A*)a.y + t * a.ldy + c);
    }
  }
}

template <typename X, typename A, typename P, bool LEAVE>
cudaError_t launch_row(const BlockArgs& a, cudaStream_t s) {
  return launch_pdl(block_row_kernel<X, A, P, LEAVE>, dim3(a.T), dim3((a.H / 8 + 31) / 32 * 32), 0, s, a);
}

template <typename X, typename A, bool LEAVE>
cudaError_t launch_long(const BlockArgs& a, cudaStream_t s) {
  static SmemOptIn opt_in;
  const auto kernel = block_long_kernel<X, A, LEAVE>;
  if (const cudaError_t e = opt_in(kernel, kSharedMost); e != cudaSuccess) return e;
  const bool keep = a.H <= kSharedMost / 4;
  return launch_pdl(kernel, dim3(a.T), dim3(1024), keep ? a.H * 4 : 0, s, a, keep);
}

// Rows of whole pieces, of any length.
template <typename X, typename A, typename P, bool LEAVE>
cudaError_t launch_shared(const BlockArgs& a, cudaStream_t s) {
  if (a.H > kSharedMost / 4) return launch_long<X, A, LEAVE>(a, s);
  static SmemOptIn opt_in;
  const auto kernel = block_shared_kernel<X, A, P, LEAVE>;
  if (const cudaError_t e = opt_in(kernel, kSharedMost); e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(a.T), dim3(kSharedThreads), a.H * 4, s, a);
}

template <typename X, typename A, typename P, int W, int N, bool LEAVE>
cudaError_t launch_stream(const BlockArgs& a, cudaStream_t s) {
  const bool full_gate = LEAVE && a.gate && a.gate_step && a.gate_ld;
  const int slot = N * (kPieces<X> + (LEAVE ? kPieces<A> : 0) + (full_gate ? kPieces<P> : 0)) * 512 * W;
  const int factors = (LEAVE ? 4 : 2) * 512 * W * N;
  constexpr int most_groups = kStreamThreads<N> / (32 * W), most_smem = kStreamSmem<W, N>;
  const int fits = (most_smem - factors) / (2 * slot), groups = fits < most_groups ? fits : most_groups;
  if (groups < 1) return launch_shared<X, A, P, LEAVE>(a, s);
  const int smem = factors + groups * 2 * slot;
  const auto kernel = block_stream_kernel<X, A, P, W, N, LEAVE>;
  static SmemOptIn opt_in;
  if (const cudaError_t e = opt_in(kernel, most_smem); e != cudaSuccess) return e;
  static PerDevice fit[2];  // resident blocks per SM of this kernel
  std::atomic<int>* known;
  if (const cudaError_t e = fit[full_gate].here(&known); e != cudaSuccess) return e;
  int per_sm = known ? known->load(std::memory_order_relaxed) : 0;
  if (per_sm == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, 32 * W * groups, smem);
    if (e != cudaSuccess) return e;
    if (known) known->store(per_sm, std::memory_order_relaxed);
  }
  const int all = (int)(((int64_t)a.T + groups - 1) / groups), most = tc_num_sms() * per_sm;
  return launch_pdl(kernel, dim3(all < most ? all : most), dim3(32 * W * groups), smem, s, a);
}

template <typename X, typename A, typename P, int TPR, int N, bool LEAVE>
cudaError_t launch_narrow(const BlockArgs& a, cudaStream_t s) {
  constexpr int threads = TPR == 32 ? 128 : TPR, rows = threads / TPR;
  return launch_pdl(block_narrow_kernel<X, A, P, TPR, N, LEAVE>, dim3((unsigned)(((int64_t)a.T + rows - 1) / rows)), dim3(threads), 0, s, a);
}

template <typename X, typename A, typename P, bool LEAVE>
cudaError_t launch_typed(const BlockArgs& a, bool wide, cudaStream_t s) {
  if (a.H <= 128) return launch_narrow<X, A, P, 32, 4, LEAVE>(a, s);
  if (wide) {
    if ((int64_t)a.T * a.H >= kStreamSize || a.H > 4096) {
      // four pieces per lane: fewer instructions per row's sums than two, more warps than eight (16384 x 2048
      // fp32 / bf16: 67.4, 66.9, 68.6 us with 2, 4, 8; bf16 50.7, 46.5, 47.5; 4096 x 2048: 21.5, 18.3, 20.0)
      if (a.H <= 512) return launch_stream<X, A, P, 1, 2, LEAVE>(a, s);
      if (a.H <= 1024) return launch_stream<X, A, P, 1, 4, LEAVE>(a, s);
      if (a.H <= 2048) return launch_stream<X, A, P, 2, 4, LEAVE>(a, s);
      if (a.H <= 4096) return launch_stream<X, A, P, 4, 4, LEAVE>(a, s);
      if (a.H <= 8192) return launch_stream<X, A, P, 8, 4, LEAVE>(a, s);
      return launch_shared<X, A, P, LEAVE>(a, s);
    } else {
      return launch_row<X, A, P, LEAVE>(a, s);
    }
  } else {
    if (a.H <= 512) return launch_narrow<X, A, P, 32, 16, LEAVE>(a, s);
    if (a.H <= 1024) return launch_narrow<X, A, P, 128, 8, LEAVE>(a, s);
    if (a.H <= 2048) return launch_narrow<X, A, P, 256, 8, LEAVE>(a, s);
    if (a.H <= 4096) return launch_narrow<X, A, P, 512, 8, LEAVE>(a, s);
    if (a.H <= 8192) return launch_narrow<X, A, P, 1024, 8, LEAVE>(a, s);
  }
  return launch_long<X, A, LEAVE>(a, s);
}

// The one type of the call's parameters and gate (0: they differ) picks the kernel.
template <typename X, typename A, bool LEAVE>
cudaError_t launch_params(const BlockArgs& a, int act_dtype, int param_dtype, bool wide, cudaStream_t s) {
  if (param_dtype == act_dtype) return launch_typed<X, A, A, LEAVE>(a, wide, s);
  if constexpr (sizeof(A) < 4)
    if (param_dtype == MOE_DT_F32) return launch_typed<X, A, float, LEAVE>(a, wide, s);
  return launch_long<X, A, LEAVE>(a, s);
}

}  // namespace

#define MOE_BLOCK_TYPES(name, X, A, act_dtype)                                                      \
  cudaError_t name(const BlockArgs& a, int param_dtype, bool wide, cudaStream_t s) {                \
    return a.block ? launch_params<X, A, true>(a, act_dtype, param_dtype, wide, s)                  \
                   : launch_params<X, A, false>(a, act_dtype, param_dtype, wide, s);                \
  }

}  // namespace moe
