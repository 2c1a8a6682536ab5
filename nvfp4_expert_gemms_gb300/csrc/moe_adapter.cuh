// Shared by the adapter kernels: the tile of a block, and packed bf16 pairs.
#pragma once
#include "moe_block.cuh"

namespace moe {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *(const uint32_t*)&v;
}
__device__ __forceinline__ float lo_f32(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float hi_f32(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }

struct Tile {
  int slot, t0, rows, rk;  // adapter (-1: none), first token, tokens (0: past the last tile), rank in use
  float scale;
};

// Tile `want` of all: requests are cut into tiles of bm tokens in order.  Every thread of the block
// calls it.  A thread also reads its request's rank and scale, whether or not the tile turns out to be
// its own: that way they cost no further trip to memory.
template <int WARPS>
__device__ __forceinline__ Tile find_tile(const AdapterArgs& a, int want, int bm) {
  __shared__ int wsum[WARPS];
  __shared__ Tile found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) found = Tile{-1, 0, 0, 0, 1.f};
  int before = 0;  // tiles of the requests in front of this chunk
  for (int q0 = 0; q0 < a.R; q0 += WARPS * 32) {
    const int q = q0 + tid;
    int s = 0, e = 0, sl = -1, rk = 0;
    float sc = 1.f;
    if (q < a.R) {
      s = a.starts[q];
      e = a.starts[q + 1];
      sl = a.slot[q];
      s = min(max(s, 0), a.T);
      e = min(max(e, s), a.T);
      if (sl >= 0 && sl < a.n) {
        rk = a.rank ? min(max(a.rank[sl], 0), a.r) : a.r;
        if (a.scale) sc = a.scale[sl];
      } else {
        sl = -1;
      }
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
    for (int w = 0; w < WARPS; ++w) {
      base += w < warp ? wsum[w] : 0;
      all += wsum[w];
    }
    const int first = base + run - n;
    if (want >= first && want < first + n) {
      const int t0 = s + (want - first) * bm;
      found = Tile{sl, t0, min(bm, e - t0), rk, sc};
    }
    before += all;
    __syncthreads();
    if (want < before) break;
  }
  __syncthreads();
  return found;
}

// At most one partial tile per request.
inline int64_t tile_bound(const AdapterArgs& a, int bm) { return (int64_t)a.T / bm + (a.R < a.T ? a.R : a.T); }

// Long requests on the 5th-generation tensor cores (moe_adapter_tile.cu): tiles of 128 tokens.
bool adapter_tiles_fit(const AdapterArgs& a);
cudaError_t launch_adapter_tiles(const AdapterArgs& a, cudaStream_t s);

}  // namespace moe
