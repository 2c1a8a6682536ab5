// Which tokens a block's tile has: of one request (find_tile) or of one adapter (gather_tile), and how many
// tiles there may be.  Nothing but AdapterArgs and the warp's own instructions, declared before, is needed
// here, so that the search can be run thread by thread on a CPU as well (tests/adapter_tiles_host.cpp).
#pragma once

namespace moe {

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

// Tiles of one adapter's tokens, whichever short requests they come from: the tokens of an adapter (and those
// without one) are numbered in request order, and 16 in a row make a tile.  Tiles are ordered by their first
// token's request.  rows: the tile's tokens.  R <= kGatherRequests, n <= kGatherSlots.
constexpr int kGatherRequests = 512, kGatherSlots = 1024;

template <int WARPS>
__device__ __forceinline__ Tile gather_tile(const AdapterArgs& a, int want, int (&rows)[16]) {
  __shared__ int count[kGatherSlots + 1];  // tokens of each adapter so far; [n]: without one
  struct Request {
    int start, len, slot, rk, before;  // before: tokens of its adapter in front of it
    float scale;
  };
  __shared__ Request req[kGatherRequests];
  __shared__ Tile found;
  __shared__ int found_at;  // the number of the tile's first token among its adapter's
  const int tid = threadIdx.x, lane = tid & 31;
  for (int i = tid; i <= a.n; i += 32 * WARPS) count[i] = 0;
  if (tid == 0) found = Tile{-1, 0, 0, 0, 1.f};
  for (int q = tid; q < a.R; q += 32 * WARPS) {
    Request r = {min(max(a.starts[q], 0), a.T), 0, a.slot[q], 0, 0, 1.f};
    r.len = min(max(a.starts[q + 1], r.start), a.T) - r.start;
    if (r.slot >= 0 && r.slot < a.n) {
      r.rk = a.rank ? min(max(a.rank[r.slot], 0), a.r) : a.r;
      if (a.scale) r.scale = a.scale[r.slot];
    } else {
      r.slot = a.n;
    }
    req[q] = r;
  }
  __syncthreads();
  if (tid < 32) {
    int tiles = 0;
    for (int q0 = 0; q0 < a.R; q0 += 32) {
      const int q = q0 + lane, len = q < a.R ? req[q].len : 0, slot = q < a.R ? req[q].slot : a.n;
      // Lanes past the last request have no tokens and count for nothing; what req holds for them is not read.
      const uint32_t there = __ballot_sync(0xffffffffu, q < a.R);
      const uint32_t peers = __match_any_sync(0xffffffffu, slot) & there, front = peers & ((1u << lane) - 1);
      int before = count[slot];
      if (__all_sync(0xffffffffu, len == 1 || q >= a.R)) before += __popc(front);
      else
        for (uint32_t m = front; m; m &= m - 1) before += req[q0 + __ffs(m) - 1].len;
      const int n = (before + len + 15) / 16 - (before + 15) / 16;  // tiles that begin in this request
      int run = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, run, off);
        if (lane >= off) run += o;
      }
      const int first = tiles + run - n;
      if (want >= first && want < first + n) {
        found = Tile{slot, 0, 0, req[q].rk, req[q].scale};
        found_at = ((before + 15) / 16 + want - first) * 16;
      }
      __syncwarp();
      if (q < a.R) req[q].before = before;
      if ((peers >> lane) == 1) count[slot] = before + len;  // the last of them (never a lane past the requests)
      __syncwarp();
      tiles += __shfl_sync(0xffffffffu, run, 31);
    }
    if (lane == 0 && found.slot >= 0) found.rows = min(16, count[found.slot] - found_at);
  }
  __syncthreads();
  Tile tile = found;
  if (tile.rows == 0) return tile;
  for (int q = tid; q < a.R; q += 32 * WARPS)
    if (req[q].slot == tile.slot) {
      const int at = req[q].before - found_at;  // where its tokens stand in the tile
      for (int i = max(-at, 0); i < req[q].len && at + i < 16; ++i) rows[at + i] = req[q].start + i;
    }
  __syncthreads();
  if (tile.slot == a.n) tile.slot = -1;
  return tile;
}

// At most one partial tile per request.
inline int64_t tile_bound(const AdapterArgs& a, int bm) { return (int64_t)a.T / bm + (a.R < a.T ? a.R : a.T); }

// At most one partial tile per adapter, and one of tokens without any.
inline int64_t gather_bound(const AdapterArgs& a) { return (int64_t)a.T / 16 + (a.R <= a.n ? a.R : a.n + 1); }

}  // namespace moe
