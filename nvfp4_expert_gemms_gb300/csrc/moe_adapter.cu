// The low-rank adapters of many requests beside a shared projection:
//
//   out[t] = base[t] + scale[a] * B[a] (A[a] x[t]),   a = the adapter of t's request.
//
// A tile is up to BM consecutive tokens of one request, so one adapter.  v = X A^T (BM x r, K = H) and
// out = base + v B^T (BM x N, K = r) run as bf16 m16n8k16 MMAs whose operands go straight from global
// memory into registers: which k of the sum sits in which of the MMA's k slots is free as long as both
// operands agree, so a lane takes 8 consecutive columns (16 bytes) of its two rows of x and of its rows
// of A.  In the same way the columns of v are dealt to the two MMA tiles of a rank step so that a lane's
// sums are the A operand of the second product as they stand (and 4 consecutive ranks, 8 bytes, of its
// rows of B its B operand), and the 32 columns of an output group so that a lane holds 8 consecutive
// ones (16 bytes of base and out).  No shared memory but for v's partial sums where warps share K.
//
// v enters the second product as two bf16 terms, hi = bf16(v) and lo = bf16(v - hi): 16 bits of
// significand, so that an adapter as large as base costs the sum no precision that shows in out's own
// bf16 rounding.  The extra MMAs are hidden: HBM bytes of x, base and out bound large batches, the
// reads of A and B (L2) small ones.
#include "moe_block.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *(const uint32_t*)&v;
}
__device__ __forceinline__ float lo_f32(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float hi_f32(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }

struct Tile {
  int slot, t0, rows;
};

// The tile of this block: requests are cut into tiles of bm tokens in order; tile `want` of all.
// slot = -1: no adapter; rows = 0: past the last tile.  Every thread of the block calls it.
__device__ __forceinline__ Tile find_tile(const AdapterArgs& a, int want, int bm) {
  __shared__ int wsum[kWarps];
  __shared__ Tile found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) found = Tile{-1, 0, 0};
  int before = 0;  // tiles of the requests in front of this chunk
  for (int q0 = 0; q0 < a.R; q0 += kWarps * 32) {
    const int q = q0 + tid;
    int s = 0, e = 0;
    if (q < a.R) {
      s = min(max(a.starts[q], 0), a.T);
      e = min(max(a.starts[q + 1], s), a.T);
    }
    const int n = (e - s + bm - 1) / bm;
    int run = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, run, off);
      if (lane >= off) run += o;
    }
    if (lane == 31) wsum[warp] = run;
    __syncthreads();
    int base = before, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      base += w < warp ? wsum[w] : 0;
      all += wsum[w];
    }
    const int first = base + run - n;
    if (want >= first && want < first + n) {
      int sl = a.slot[q];
      sl = sl >= 0 && sl < a.n ? sl : -1;
      const int t0 = s + (want - first) * bm;
      found = Tile{sl, t0, min(bm, e - t0)};
    }
    before += all;
    __syncthreads();
    if (want < before) break;
  }
  __syncthreads();
  return found;
}

// One tile per blockIdx.x, output columns in gridDim.y parts.  WM warps along the tokens (16 each),
// kWarps / WM along K (first product) and along N (second).  RT: rank steps of 16 (r <= 16 RT).
template <int RT, int WM>
__global__ void __launch_bounds__(32 * kWarps) adapter_kernel(const AdapterArgs a) {
  constexpr int WK = kWarps / WM, BM = 16 * WM;
  extern __shared__ float vpart[];  // [WK][WM][RT * 2][32][4], only with WK > 1
  pdl_wait();
  pdl_trigger();
  const Tile tile = find_tile(a, blockIdx.x, BM);
  if (tile.rows == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wm = warp / WK, wk = warp % WK;
  const int g = lane >> 2, t = lane & 3;
  const int r0 = 16 * wm + g, r1 = r0 + 8;  // the lane's two rows of the tile
  const bool ok0 = r0 < tile.rows, ok1 = r1 < tile.rows;
  const int64_t t0 = tile.t0 + (ok0 ? r0 : 0), t1 = tile.t0 + (ok1 ? r1 : 0);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  int rk = 0;
  float sc = 1.f;
  if (tile.slot >= 0) {
    rk = a.rank ? min(max(a.rank[tile.slot], 0), a.r) : a.r;
    if (a.scale) sc = a.scale[tile.slot];
  }
  float v[2 * RT][4];
#pragma unroll
  for (int j = 0; j < 2 * RT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[j][i] = 0.f;
  if (rk > 0 && 16 * wm < tile.rows) {
    const __nv_bfloat16* A = a.A + (int64_t)tile.slot * a.r * a.H;
    const __nv_bfloat16 *x0 = a.x + t0 * a.ldx, *x1 = a.x + t1 * a.ldx;
#pragma unroll 2
    for (int k = 32 * wk + 8 * t; k - 8 * t < a.H; k += 32 * WK) {
      const bool in = k < a.H;
      const uint4 p0 = in && ok0 ? *(const uint4*)(x0 + k) : zero, p1 = in && ok1 ? *(const uint4*)(x1 + k) : zero;
#pragma unroll
      for (int j = 0; j < 2 * RT; ++j) {
        if (16 * (j >> 1) >= rk) break;
        const int row = 16 * (j >> 1) + 4 * (g >> 1) + 2 * (j & 1) + (g & 1);
        const uint4 q = in && row < rk ? *(const uint4*)(A + (int64_t)row * a.H + k) : zero;
        mma_bf16(v[j], p0.x, p1.x, p0.y, p1.y, q.x, q.y);
        mma_bf16(v[j], p0.z, p1.z, p0.w, p1.w, q.z, q.w);
      }
    }
  }
  if constexpr (WK > 1) {  // v's partial sums over the warps' parts of K meet in every warp
    float4* part = (float4*)vpart;
#pragma unroll
    for (int j = 0; j < 2 * RT; ++j) part[((wk * WM + wm) * 2 * RT + j) * 32 + lane] = *(float4*)v[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2 * RT; ++j) {
      float4 s = part[(wm * 2 * RT + j) * 32 + lane];
#pragma unroll
      for (int w = 1; w < WK; ++w) {
        const float4 o = part[((w * WM + wm) * 2 * RT + j) * 32 + lane];
        s.x += o.x;
        s.y += o.y;
        s.z += o.z;
        s.w += o.w;
      }
      *(float4*)v[j] = s;
    }
  }
  if (16 * wm >= tile.rows) return;
  // the second product's A operand: rank step s, rows r0 / r1, first and second k pair
  uint32_t hi[RT][4], lo[RT][4];
#pragma unroll
  for (int s = 0; s < RT; ++s)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int row = 0; row < 2; ++row) {
        const float c0 = v[2 * s + h][2 * row] * sc, c1 = v[2 * s + h][2 * row + 1] * sc;
        const uint32_t p = pack_bf16(c0, c1);
        hi[s][2 * h + row] = p;
        lo[s][2 * h + row] = pack_bf16(c0 - lo_f32(p), c1 - hi_f32(p));
      }
  const __nv_bfloat16* B = a.B + (int64_t)max(tile.slot, 0) * a.N * a.r;
  const __nv_bfloat16 *b0 = a.base + t0 * a.ldb, *b1 = a.base + t1 * a.ldb;
  __nv_bfloat16 *o0 = a.out + t0 * a.ldo, *o1 = a.out + t1 * a.ldo;
  if (rk == 0 && a.out == a.base) return;
  for (int c = 32 * (blockIdx.y * WK + wk); c < a.N; c += 32 * WK * gridDim.y) {
    const int col = c + 8 * t;
    const uint4 y0 = ok0 && col < a.N ? *(const uint4*)(b0 + col) : zero;
    const uint4 y1 = ok1 && col < a.N ? *(const uint4*)(b1 + col) : zero;
    const uint32_t w0[4] = {y0.x, y0.y, y0.z, y0.w}, w1[4] = {y1.x, y1.y, y1.z, y1.w};
    uint32_t q0[4], q1[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float d[4] = {lo_f32(w0[j]), hi_f32(w0[j]), lo_f32(w1[j]), hi_f32(w1[j])};
      const int n = c + 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
      for (int s = 0; s < RT; ++s) {
        if (16 * s >= rk) break;
        const int k = 16 * s + 4 * t;
        uint2 b = make_uint2(0, 0);
        if (n < a.N && k < rk) {
          b = *(const uint2*)(B + (int64_t)n * a.r + k);
          if (k + 4 > rk) {  // what stands past the adapter's rank is not used
            b.x = k + 1 < rk ? b.x : b.x & 0xFFFFu;
            b.y = k + 2 < rk ? (k + 3 < rk ? b.y : b.y & 0xFFFFu) : 0u;
          }
        }
        mma_bf16(d, lo[s][0], lo[s][1], lo[s][2], lo[s][3], b.x, b.y);
        mma_bf16(d, hi[s][0], hi[s][1], hi[s][2], hi[s][3], b.x, b.y);
      }
      q0[j] = pack_bf16(d[0], d[1]);
      q1[j] = pack_bf16(d[2], d[3]);
    }
    if (ok0 && col < a.N) *(uint4*)(o0 + col) = make_uint4(q0[0], q0[1], q0[2], q0[3]);
    if (ok1 && col < a.N) *(uint4*)(o1 + col) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
  }
}

template <int RT, int WM>
cudaError_t launch_tiles(const AdapterArgs& a, int parts, cudaStream_t s) {
  constexpr int BM = 16 * WM, WK = kWarps / WM;
  const int64_t tiles = (int64_t)a.T / BM + (a.R < a.T ? a.R : a.T);  // at most one partial tile per request
  const size_t smem = WK > 1 ? (size_t)WK * WM * RT * 2 * 32 * 16 : 0;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(adapter_kernel<RT, WM>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  note_launches(1);
  return launch_pdl(adapter_kernel<RT, WM>, dim3((unsigned)tiles, parts), dim3(32 * kWarps), smem, s, a);
}

template <int RT>
cudaError_t launch_rank(const AdapterArgs& a, cudaStream_t s) {
  if (a.T / (a.R > 0 ? a.R : 1) >= 512) return launch_tiles<RT, 8>(a, 1, s);
  const int64_t tiles = (int64_t)a.T / 16 + (a.R < a.T ? a.R : a.T);
  const int parts = tiles >= 152 ? 1 : tiles >= 32 ? 4 : 8;
  return launch_tiles<RT, 1>(a, parts, s);
}

}  // namespace

cudaError_t launch_adapters(const AdapterArgs& a, cudaStream_t s) {
  if (a.T == 0 || a.R == 0 || a.N == 0) return cudaSuccess;
  if (a.r <= 16) return launch_rank<1>(a, s);
  if (a.r <= 32) return launch_rank<2>(a, s);
  if (a.r <= 64) return launch_rank<4>(a, s);
  return launch_rank<8>(a, s);
}

}  // namespace moe

extern "C" moe_status_t moe_adapters_add(const void* x, int64_t ldx, const void* base, int64_t ldb, const void* A,
                                         const void* B, const float* scale, const int32_t* rank,
                                         const int32_t* starts, const int32_t* slot, void* out, int64_t ldo, int T,
                                         int R, int n, int r, int H, int N, moe_stream_t stream) {
  using namespace moe;
  if (T < 0 || R < 0 || n < 0 || H < 8 || H % 8 != 0 || N < 8 || N % 8 != 0 || r < 8 || r > 128 || r % 8 != 0)
    return MOE_ERR_INVALID_ARG;
  const auto ok = [](const void* p, int64_t ld, int cols) {
    return p && (uintptr_t)p % 16 == 0 && ld >= cols && ld % 8 == 0;
  };
  if (T > 0 && (!ok(x, ldx, H) || !ok(base, ldb, N) || !ok(out, ldo, N) || !starts || (R > 0 && !slot)))
    return MOE_ERR_INVALID_ARG;
  if (n > 0 && (!ok(A, H, H) || !ok(B, N, N))) return MOE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)scale, (const void*)rank, (const void*)starts, (const void*)slot})
    if ((uintptr_t)p % 4 != 0) return MOE_ERR_INVALID_ARG;
  const moe_status_t dv = device_ok();
  if (dv != MOE_OK) return dv;
  const AdapterArgs a = {(const __nv_bfloat16*)x,
                         (const __nv_bfloat16*)base,
                         (const __nv_bfloat16*)A,
                         (const __nv_bfloat16*)B,
                         scale,
                         rank,
                         starts,
                         slot,
                         (__nv_bfloat16*)out,
                         ldx,
                         ldb,
                         ldo,
                         T,
                         R,
                         n,
                         r,
                         H,
                         N};
  return launch_adapters(a, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
