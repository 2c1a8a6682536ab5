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
// v enters the second product as three bf16 terms, each the rest of the one before: 24 bits of significand, as fp32
// holds, so that the sum keeps its precision also where base and the adapter's part cancel.  The extra MMAs are
// hidden: the register MMAs run at some 597 TFLOP/s here (1.04 ns per m16n8k16 and SM), and what bounds these kernels
// is memory.
#include <cooperative_groups.h>

#include "moe_adapter.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kWarps = 8;  // of a block of the kernel for few

__device__ __forceinline__ void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A rank step's two tiles of v (the lane's ranks are k .. k+3) times the adapter's scale.  Zero past the adapter's rank,
// where an infinite x leaves NaN.
__device__ __forceinline__ void scale_v(float (&v0)[4], float (&v1)[4], float sc, int k, int rk) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v0[i] = k + (i & 1) < rk ? v0[i] * sc : 0.f;
    v1[i] = k + 2 + (i & 1) < rk ? v1[i] * sc : 0.f;
  }
}

// The same as the second product's A operand: [2 h + row] of the three terms.
__device__ __forceinline__ void split_v(const float (&v0)[4], const float (&v1)[4], Terms (&w)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int row = 0; row < 2; ++row) w[2 * h + row] = split_pair((h ? v1 : v0)[2 * row], (h ? v1 : v0)[2 * row + 1]);
}

// d += v B^T of one rank step, the smallest terms first.
__device__ __forceinline__ void mma_terms(float* d, const Terms (&w)[4], uint2 b) {
  mma_bf16(d, w[0].lo, w[1].lo, w[2].lo, w[3].lo, b.x, b.y);
  mma_bf16(d, w[0].mid, w[1].mid, w[2].mid, w[3].mid, b.x, b.y);
  mma_bf16(d, w[0].hi, w[1].hi, w[2].hi, w[3].hi, b.x, b.y);
}

// Clears what stands past the adapter's rank in a lane's ranks k .. k+3 of a row of B.
__device__ __forceinline__ uint2 cut_rank(uint2 b, int k, int rk) {
  if (k + 4 > rk) {
    b.x = k + 1 < rk ? b.x : k < rk ? b.x & 0xFFFFu : 0u;
    b.y = k + 3 < rk ? b.y : k + 2 < rk ? b.y & 0xFFFFu : 0u;
  }
  return b;
}

// ---- few tokens per request ------------------------------------------------------------------
// One tile of up to 16 MT tokens of a request, or (GATHER) 16 of an adapter's, per cluster of blocks.  The blocks' warps
// share K (each lane's loads of x and A are independent and all issued at once), v's parts are summed warp by warp in
// shared memory and block by block in a fixed order (each block writes its own into every block's shared memory: one
// barrier and no remote read to wait for), and the blocks share N.  B and base of a warp's first 32 columns are loaded
// before the sums meet.
//
// Times in a CUDA graph, as those of the other rules below.  One token, 2048 -> 2048 at rank 16: 3.2 us on eight blocks,
// 6.3 on one (a launch alone takes 1.6); by a clock trace with two terms of v 0.7 of it are the requests, 0.8 x and A,
// 0.9 the sums, 0.4 the second product.  64 requests at rank 32: 5.9 us on four blocks each, 8.4 on one.  4001 tokens of
// 37 requests at rank 16, 2048 -> 1536: 12.1 us in tiles of 32, two blocks each (13.2 in tiles of 16), against 6.0 by HBM.
// Latency bounds it: 324 blocks are one wave, 23% of the warps, issue slots 38% (with two terms of v the L1 was 32% busy,
// the L2 17%, and sixteen warps per block in place of eight 3% slower in tiles of 16, up to 1.7 times at rank 32; 2%
// faster in tiles of 32, but 11% slower past one wave).
//
// Tiles of 32 (ranks up to 16) read A and B half as often: they are for batches whose tiles of 16 leave no four
// blocks to a tile.  2048 -> 2048: 5000 ragged tokens 20.2 us against 25.4, 7000 21.6 against 27.6, 4096 of 16 even
// requests 13.9 against 15.5, 1024 of them 6.7 against 5.3.  At rank 32 they take 19.6 us against 17.6 at 4096 tokens.
template <int RT, int MT, bool GATHER>
__global__ void __launch_bounds__(32 * kWarps, RT <= 4 ? 2 : 1) adapter_few_kernel(const AdapterArgs a) {
  extern __shared__ __align__(128) unsigned char few_smem[];
  float4(*part)[2 * RT * MT][32] = (float4(*)[2 * RT * MT][32])few_smem;  // [kWarps]
  float4(*got)[2 * RT * MT][32] = part + kWarps;  // [C]: the blocks' sums
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), crank = cluster.block_rank();
  pdl_wait();
  pdl_trigger();
  static_assert(!GATHER || MT == 1);
  __shared__ int from[16];  // GATHER: the tile's tokens
  Tile tile;
  if constexpr (GATHER) tile = gather_tile<kWarps>(a, blockIdx.x / C, from);
  else tile = find_tile<kWarps>(a, blockIdx.x / C, 16 * MT);
  if (tile.rows == 0) return;
  const int rk = tile.rk;
  if (rk == 0 && a.out == a.base) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  bool ok[MT][2];
  int64_t tok[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      ok[m][h] = 16 * m + 8 * h + g < tile.rows;
      const int i = ok[m][h] ? 16 * m + 8 * h + g : 0;
      tok[m][h] = GATHER ? from[i] : tile.t0 + i;
    }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int part_w = crank * kWarps + warp, parts = C * kWarps;
  float v[MT][2 * RT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 2 * RT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[m][j][i] = 0.f;
  const __nv_bfloat16* A = a.A + (int64_t)max(tile.slot, 0) * a.r * a.H;
  const __nv_bfloat16* B = a.B + (int64_t)max(tile.slot, 0) * a.N * a.r;
  struct Cols {
    uint2 bq[4][RT];
    uint4 y[MT][2];
  };
  auto load_cols = [&](Cols& f, int c) {  // B and base of columns c .. c+31
    const int col = c + 8 * t;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        f.y[m][h] = ok[m][h] && col < a.N ? *(const uint4*)(a.base + tok[m][h] * a.ldb + col) : zero;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = c + 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
      for (int s = 0; s < RT; ++s) {
        const int k = 16 * s + 4 * t;
        f.bq[j][s] = n < a.N && k < rk ? *(const uint2*)(B + (int64_t)n * a.r + k) : make_uint2(0, 0);
      }
    }
  };
  if (rk > 0) {
    // This block runs: its memory may be written.  Relaxed, nothing of its own is handed over yet (the default
    // orders the accesses before it and holds up the loads below by 0.4 us).
    if (C > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    constexpr int U = RT == 1 ? 4 / MT : RT == 2 && MT == 1 ? 2 : 1;  // steps whose loads are in flight together
    for (int kb = 32 * part_w; kb < a.H; kb += 32 * parts * U) {
      uint4 p[U][MT][2], q[U][2 * RT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = kb + 32 * parts * u + 8 * t;
        const bool in = k < a.H;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            p[u][m][h] = in && ok[m][h] ? *(const uint4*)(a.x + tok[m][h] * a.ldx + k) : zero;
#pragma unroll
        for (int j = 0; j < 2 * RT; ++j) {
          const int row = 16 * (j >> 1) + 4 * (g >> 1) + 2 * (j & 1) + (g & 1);
          q[u][j] = in && row < rk ? *(const uint4*)(A + (int64_t)row * a.H + k) : zero;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2 * RT; ++j)
          if (16 * (j >> 1) < rk)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma_bf16(v[m][j], p[u][m][0].x, p[u][m][1].x, p[u][m][0].y, p[u][m][1].y, q[u][j].x, q[u][j].y);
              mma_bf16(v[m][j], p[u][m][0].z, p[u][m][1].z, p[u][m][0].w, p[u][m][1].w, q[u][j].z, q[u][j].w);
            }
    }
  }
  Cols now;
  load_cols(now, 32 * part_w);
  if (rk > 0) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 2 * RT; ++j)
        if (ok[m][0]) part[warp][2 * RT * m + j][lane] = make_float4(v[m][j][0], v[m][j][1], v[m][j][2], v[m][j][3]);
    __syncthreads();
    if (C > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
    for (int e = threadIdx.x; e < 2 * RT * MT * 32; e += 32 * kWarps) {
      const int j = e >> 5, l = e & 31;
      if (16 * (j / (2 * RT)) + (l >> 2) >= tile.rows) continue;
      float4 s = part[0][j][l];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float4 o = part[w][j][l];
        s.x += o.x;
        s.y += o.y;
        s.z += o.z;
        s.w += o.w;
      }
      if (C == 1) {
        got[0][j][l] = s;
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < C) *cluster.map_shared_rank(&got[crank][j][l], c) = s;
      }
    }
    const float4(*all)[32] = got[0];
    if (C > 1) {
      cluster.sync();  // the only accesses to another block's memory are behind it
      float4(*sum)[32] = part[0];
      for (int e = threadIdx.x; e < 2 * RT * MT * 32; e += 32 * kWarps) {
        const int j = e >> 5, l = e & 31;
        if (16 * (j / (2 * RT)) + (l >> 2) >= tile.rows) continue;
        float4 o[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < C) o[c] = got[c][j][l];
        float4 s = o[0];
#pragma unroll
        for (int c = 1; c < 8; ++c)
          if (c < C) {
            s.x += o[c].x;
            s.y += o[c].y;
            s.z += o[c].z;
            s.w += o[c].w;
          }
        sum[j][l] = s;
      }
      all = part[0];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 2 * RT; ++j) {
        const float4 s = ok[m][0] ? all[2 * RT * m + j][lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        v[m][j][0] = s.x;
        v[m][j][1] = s.y;
        v[m][j][2] = s.z;
        v[m][j][3] = s.w;
      }
  }
  constexpr bool HELD = RT * MT <= 2;  // v's terms are held; else made again for each group of columns (registers)
  Terms held[HELD ? MT : 1][HELD ? RT : 1][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int s = 0; s < RT; ++s) {
      scale_v(v[m][2 * s], v[m][2 * s + 1], tile.scale, 16 * s + 4 * t, rk);
      if constexpr (HELD) split_v(v[m][2 * s], v[m][2 * s + 1], held[m][s]);
    }
  for (int c = 32 * part_w; c < a.N; c += 32 * parts) {
    constexpr bool AHEAD = RT * MT <= 2;  // the next columns are loaded under these ones (registers allowing)
    Cols next;
    if (AHEAD && c + 32 * parts < a.N) load_cols(next, c + 32 * parts);
    if (!AHEAD && c != 32 * part_w) load_cols(now, c);
    const int col = c + 8 * t;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint32_t w0[4] = {now.y[m][0].x, now.y[m][0].y, now.y[m][0].z, now.y[m][0].w};
      const uint32_t w1[4] = {now.y[m][1].x, now.y[m][1].y, now.y[m][1].z, now.y[m][1].w};
      float d[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[j][0] = lo_f32(w0[j]);
        d[j][1] = hi_f32(w0[j]);
        d[j][2] = lo_f32(w1[j]);
        d[j][3] = hi_f32(w1[j]);
      }
#pragma unroll
      for (int s = 0; s < RT; ++s)
        if (16 * s < rk) {
          Terms made[4];
          if constexpr (!HELD) split_v(v[m][2 * s], v[m][2 * s + 1], made);
          const Terms(&w)[4] = HELD ? held[HELD ? m : 0][HELD ? s : 0] : made;
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_terms(d[j], w, cut_rank(now.bq[j][s], 16 * s + 4 * t, rk));
        }
      uint32_t q0[4], q1[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        q0[j] = pack_bf16(d[j][0], d[j][1]);
        q1[j] = pack_bf16(d[j][2], d[j][3]);
      }
      if (ok[m][0] && col < a.N) *(uint4*)(a.out + tok[m][0] * a.ldo + col) = make_uint4(q0[0], q0[1], q0[2], q0[3]);
      if (ok[m][1] && col < a.N) *(uint4*)(a.out + tok[m][1] * a.ldo + col) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
    }
    if (AHEAD) now = next;
  }
}

// ---- many tokens per request, ranks up to 16 ---------------------------------------------------
// One tile of 16 WM tokens per block, WM x WK warps: WM along the tokens, WK along K (first product)
// and N (second).  x and A, then base and B, stream through a ring of NS shared-memory stages filled
// by cp.async NS - 1 stages ahead, so the bytes in flight do not depend on registers or warps.
//   K stage  kKC columns of x ([BM][kKC]) and of A ([16][kKC]); row i's 16-byte piece p sits at
//            piece p ^ 4 (i & 1), so the 8 lanes that one 16-byte shared load serves at a time (two
//            rows, four pieces) hit all banks once
//   N stage  kNC columns of base ([BM][kNC], same placement) and kNC rows of B, row order (n-tile, lane
//            group), 32 bytes each (16 lanes of an 8-byte load: four rows, all banks once)
// Tiles of 32 tokens, four to six blocks per SM: 16384 tokens, 2048 -> 2048 at rank 16 in 42.0 us (30.4 by
// HBM), 100 ragged requests of them 41.7 (with two terms of v 40.2 and 39.8, in tiles of 64 39.6 and 60.3: more empty
// rows).
constexpr int kKC = 128, kNC = 128;

struct Many {
  static constexpr int RT = 1, WM = 2, WK = 2, NS = 4;
  static constexpr int BM = 16 * WM, threads = 32 * WM * WK, pitch = 32;  // bytes of a row of B
  static constexpr int xbytes = BM * kKC * 2, ybytes = BM * kNC * 2;
  static constexpr int stage = xbytes + 16 * kKC * 2;  // of K; an N stage takes as much
  static constexpr int smem = NS * stage;
  static_assert(ybytes + kNC * pitch <= stage && WM * 2 * RT * 32 * 16 <= stage, "v's sums meet in one stage");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

__global__ void __launch_bounds__(Many::threads) adapter_many_kernel(const AdapterArgs a) {
  using G = Many;
  constexpr int RT = G::RT, WM = G::WM, WK = G::WK, BM = G::BM, NT = G::threads, NS = G::NS;
  extern __shared__ __align__(128) unsigned char ring[];
  pdl_wait();
  pdl_trigger();
  const Tile tile = find_tile<WM * WK>(a, blockIdx.x, BM);
  if (tile.rows == 0) return;
  const int rk = tile.rk;
  if (rk == 0 && a.out == a.base) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wm = warp % WM, wk = warp / WM;
  const int g = lane >> 2, t = lane & 3, r0 = 16 * wm + g, r1 = r0 + 8;
  const uint32_t ring_u = (uint32_t)__cvta_generic_to_shared(ring);
  const __nv_bfloat16* A = a.A + (int64_t)max(tile.slot, 0) * a.r * a.H;
  const __nv_bfloat16* B = a.B + (int64_t)max(tile.slot, 0) * a.N * a.r;
  const __nv_bfloat16* x = a.x + (int64_t)tile.t0 * a.ldx;
  const __nv_bfloat16* base = a.base + (int64_t)tile.t0 * a.ldb;
  const int steps = (rk + 15) / 16;  // rank steps in use
  const int kst = rk > 0 ? (a.H + kKC - 1) / kKC : 0, nst = (a.N + kNC - 1) / kNC;

  auto fill_k = [&](int st, int at) {
    const uint32_t xs = ring_u + at * G::stage, as = xs + G::xbytes;
    constexpr int P = kKC / 8;  // pieces per row
    const int k0 = st * kKC;
#pragma unroll
    for (int i = 0; i < BM * P / NT; ++i) {
      const int e = tid + i * NT, row = e / P, p = e % P;
      const bool in = row < tile.rows && k0 + 8 * p < a.H;
      cp16(xs + row * (kKC * 2) + ((p ^ ((row & 1) << 2)) << 4), in ? x + (int64_t)row * a.ldx + k0 + 8 * p : x, in);
    }
    for (int e = tid; e < 16 * steps * P; e += NT) {
      const int row = e / P, p = e % P;
      const bool in = row < rk && k0 + 8 * p < a.H;
      cp16(as + row * (kKC * 2) + ((p ^ ((row & 1) << 2)) << 4), in ? A + (int64_t)row * a.H + k0 + 8 * p : A, in);
    }
  };
  auto fill_n = [&](int st, int at) {
    const uint32_t ys = ring_u + at * G::stage, bs = ys + G::ybytes;
    constexpr int P = kNC / 8;
    const int c0 = st * kNC;
#pragma unroll
    for (int i = 0; i < BM * P / NT; ++i) {
      const int e = tid + i * NT, row = e / P, p = e % P;
      const bool in = row < tile.rows && c0 + 8 * p < a.N;
      cp16(ys + row * (kNC * 2) + ((p ^ ((row & 1) << 2)) << 4), in ? base + (int64_t)row * a.ldb + c0 + 8 * p : base, in);
    }
    for (int e = tid; e < kNC * 2 * steps; e += NT) {
      const int n = e / (2 * steps), p = e % (2 * steps), q = n & 31;
      const int row = (n & ~31) + ((q & 6) << 2) + 2 * (q >> 3) + (q & 1);  // 8 (n-tile) + lane group
      const bool in = c0 + n < a.N && 8 * p < a.r;
      cp16(bs + row * G::pitch + 16 * p, in ? B + (int64_t)(c0 + n) * a.r + 8 * p : B, in);
    }
  };
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
  auto wait = [] { asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory"); };

  float v[2 * RT][4];
#pragma unroll
  for (int j = 0; j < 2 * RT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[j][i] = 0.f;
  if (kst > 0) {
    for (int s = 0; s < NS - 1; ++s) {
      if (s < kst) fill_k(s, s);
      commit();
    }
    for (int st = 0; st < kst; ++st) {
      wait();
      __syncthreads();  // the stage has landed for every thread, and the one refilled below is read
      if (st + NS - 1 < kst) fill_k(st + NS - 1, (st + NS - 1) % NS);
      commit();
      const unsigned char* xs = ring + (st % NS) * G::stage;
      const unsigned char* as = xs + G::xbytes;
      if (16 * wm < tile.rows)
#pragma unroll
        for (int i = 0; i < kKC / 32 / WK; ++i) {
          const int p = (4 * (i * WK + wk) + t) ^ ((g & 1) << 2);
          const uint4 p0 = *(const uint4*)(xs + r0 * (kKC * 2) + 16 * p), p1 = *(const uint4*)(xs + r1 * (kKC * 2) + 16 * p);
#pragma unroll
          for (int j = 0; j < 2 * RT; ++j)
            if ((j >> 1) < steps) {
              const int row = 16 * (j >> 1) + 4 * (g >> 1) + 2 * (j & 1) + (g & 1);
              const uint4 q = *(const uint4*)(as + row * (kKC * 2) + 16 * p);
              mma_bf16(v[j], p0.x, p1.x, p0.y, p1.y, q.x, q.y);
              mma_bf16(v[j], p0.z, p1.z, p0.w, p1.w, q.z, q.w);
            }
        }
    }
    __syncthreads();
  }
  // the first N stages are on their way (from stage 1 of the ring on) while the sums meet in stage 0
  for (int s = 0; s < NS - 1; ++s) {
    if (s < nst) fill_n(s, (s + 1) % NS);
    commit();
  }
  if (rk > 0) {
    float4* sum = (float4*)ring + wm * 2 * RT * 32 + lane;
    if (wk == 1)
#pragma unroll
      for (int j = 0; j < 2 * RT; ++j) sum[32 * j] = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
    __syncthreads();
    if (wk == 0)
#pragma unroll
      for (int j = 0; j < 2 * RT; ++j) {
        const float4 o = sum[32 * j];
        v[j][0] += o.x;
        v[j][1] += o.y;
        v[j][2] += o.z;
        v[j][3] += o.w;
        sum[32 * j] = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
      }
    __syncthreads();
    if (wk == 1)
#pragma unroll
      for (int j = 0; j < 2 * RT; ++j) {
        const float4 o = sum[32 * j];
        v[j][0] = o.x;
        v[j][1] = o.y;
        v[j][2] = o.z;
        v[j][3] = o.w;
      }
  }
  Terms w[RT][4];
#pragma unroll
  for (int s = 0; s < RT; ++s) {
    scale_v(v[2 * s], v[2 * s + 1], tile.scale, 16 * s + 4 * t, rk);
    split_v(v[2 * s], v[2 * s + 1], w[s]);
  }
  const bool ok0 = r0 < tile.rows, ok1 = r1 < tile.rows;
  __nv_bfloat16 *o0 = a.out + (int64_t)(tile.t0 + r0) * a.ldo, *o1 = o0 + 8 * a.ldo;
  for (int st = 0; st < nst; ++st) {
    wait();
    __syncthreads();
    if (st + NS - 1 < nst) fill_n(st + NS - 1, (st + NS) % NS);
    commit();
    const unsigned char* ys = ring + ((st + 1) % NS) * G::stage;
    const unsigned char* bs = ys + G::ybytes;
    if (16 * wm >= tile.rows) continue;
#pragma unroll
    for (int i = 0; i < kNC / 32 / WK; ++i) {
      const int c = 32 * (i * WK + wk), col = st * kNC + c + 8 * t;
      if (st * kNC + c >= a.N) break;
      const int p = (c / 8 + t) ^ ((g & 1) << 2);
      const uint4 y0 = *(const uint4*)(ys + r0 * (kNC * 2) + 16 * p), y1 = *(const uint4*)(ys + r1 * (kNC * 2) + 16 * p);
      const uint32_t w0[4] = {y0.x, y0.y, y0.z, y0.w}, w1[4] = {y1.x, y1.y, y1.z, y1.w};
      uint32_t q0[4], q1[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float d[4] = {lo_f32(w0[j]), hi_f32(w0[j]), lo_f32(w1[j]), hi_f32(w1[j])};
#pragma unroll
        for (int s = 0; s < RT; ++s)
          if (s < steps) {
            uint2 b = *(const uint2*)(bs + (c + 8 * j + g) * G::pitch + 32 * s + 8 * t);
            if (16 * s + 16 > rk) b = cut_rank(b, 16 * s + 4 * t, rk);
            mma_terms(d, w[s], b);
          }
        q0[j] = pack_bf16(d[0], d[1]);
        q1[j] = pack_bf16(d[2], d[3]);
      }
      if (ok0 && col < a.N) *(uint4*)(o0 + col) = make_uint4(q0[0], q0[1], q0[2], q0[3]);
      if (ok1 && col < a.N) *(uint4*)(o1 + col) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
    }
  }
}

cudaError_t launch_many(const AdapterArgs& a, cudaStream_t s) {
  static SmemOptIn opt_in;
  if (const cudaError_t e = opt_in(adapter_many_kernel, Many::smem); e != cudaSuccess) return e;
  note_launches(1);
  return launch_pdl(adapter_many_kernel, dim3((unsigned)tile_bound(a, Many::BM)), dim3(Many::threads), Many::smem, s, a);
}

template <int RT, int MT, bool GATHER>
cudaError_t launch_few(const AdapterArgs& a, int cluster, cudaStream_t s) {
  constexpr int per = 2 * RT * MT * 32 * 16, most = (kWarps + 8) * per;
  static SmemOptIn opt_in;
  if (const cudaError_t e = opt_in(adapter_few_kernel<RT, MT, GATHER>, most); e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((GATHER ? gather_bound(a) : tile_bound(a, 16 * MT)) * cluster));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = (kWarps + cluster) * per;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  note_launches(1);
  return cudaLaunchKernelEx(&cfg, adapter_few_kernel<RT, MT, GATHER>, a);
}

template <int RT>
cudaError_t launch_rank(const AdapterArgs& a, cudaStream_t s) {
  const int64_t requests = a.R < a.T ? a.R : a.T, mean = a.T / requests;
  const int64_t room = (int64_t)tc_num_sms() * (RT <= 4 ? 2 : 1);  // blocks that the device takes at once
  // Tiles, with requests of mean > the tile's height half a tile over each.
  const int64_t likely16 = a.T / 16 + requests / 2, likely32 = a.T / 32 + requests / 2;
  // Blocks of a cluster share a tile as long as the grid fits the device at once.  By eight only up to 80% of it
  // (512 tokens of one request, 32 tiles, at rank 16: 4.6 us by eight, 4.2 by four; at rank 128, a block per SM, 25.8 and
  // 12.3), but for ranks 33 to 64, where the work outweighs it (32 requests of 16 tokens at rank 64: 8.7 and 10.3, though
  // one request 8.6 and 8.0).
  const auto blocks = [&](int64_t tiles) {
    return 80 * tiles <= room * (RT == 4 ? 10 : 8) ? 8 : 4 * tiles <= room ? 4 : 2 * tiles <= room ? 2 : 1;
  };
  if constexpr (RT == 1) {
    // Long requests past one wave of tiles of 32: 16384 tokens, 2048 -> 2048, the ring 42.0 us, those tiles 43.5
    // (tcgen05 tiles 40.0, 60.9 ragged); 10000 ragged 36.2 and 38.5; 7000, within a wave, 27.6 and 21.6.
    if (mean >= 32 && likely32 > room) return launch_many(a, s);
    if (mean > 16 && 4 * likely16 > room) return launch_few<1, 2, false>(a, blocks(likely32), s);
  } else if (mean >= 16) {
    // The tcgen05 tiles or the kernel for few, by their waves over the SMs (a part of one where clusters share a
    // tile), a wave of the tiles in units of the other's: 1.95, 0.85 and 1.1 at ranks up to 32, 64 and 128.  Times
    // with the tiles and without, 2048 -> 2048, ragged requests: rank 32, 4096 tokens of 4 requests 19.2 and 17.5 us, 6000
    // of 40 24.6 and 30.3; rank 64, 2048 of 32 33.4 and 19.0, 4096 of 64 25.3 and 31.9, 16384 of 300 88 and 118, of 1000
    // 200 and 165; rank 128, 2048 of 32 50.5 and 40.2, of 128 43.7 and 72.7, 8192 of 128 45.8 and 143, 16384 of 300 123 and
    // 280.  Even requests may fill the tiles otherwise than guessed (6000 of 40, rank 32, 41.3 and 30.6; 2048 of 32, rank
    // 128, 29.2 and 40.2).  The tiles' fixed cost wants some work against it: 2048 of 100, 256 -> 256, rank 64, 20.5 and
    // 6.4; 16384 of 16, 512 -> 512, rank 32, 15.3 and 20.9, rank 64 15.9 and 35.6 (3000 of 20, 1024 -> 1024, near the
    // bound, 14.4 and 16.3 ragged, 25.9 and 16.0 even).
    const int64_t sms = tc_num_sms(), likely128 = a.T / 128 + (mean >= 128 ? requests / 2 : requests);
    const double full = likely128 > sms ? (double)likely128 / sms : 1.;
    const double tiles = (RT == 2 ? 1.95 : RT == 4 ? 0.85 : 1.1) *
                         (mean < 128 || 20 * likely128 > sms * 9 ? full : 40 * likely128 > sms * 9 ? 0.75 : 0.55);
    const double few = blocks(likely16) == 1 ? (double)((likely16 + room - 1) / room) : blocks(likely16) == 2 ? 0.58 : 0.3;
    const double work = few * (16 * RT) * (a.H + a.N);
    if (tiles < few && work >= (RT == 2 ? 1.0e5 : 1.5e5) && adapter_tiles_fit(a)) return launch_adapter_tiles(a, s);
  }
  // Short requests that share adapters, enough of them to pay for the longer search (0.4 to 1 us): one token each,
  // 2048 -> 2048, 256 requests over 16 adapters: rank 16 6.7 us against 9.0, rank 64 10.8 against 26.0, rank 128 14.9
  // against 61.1; over 64 adapters: rank 16 9.1 against 8.9, rank 32 10.4 against 13.4, rank 64 20.0 against 29.4.
  if (a.R >= 32 && a.R <= kGatherRequests && a.n <= kGatherSlots && a.T <= 8 * (int64_t)a.R &&
      (int64_t)a.R * (RT < 4 ? RT : 4) >= 8 * (int64_t)a.n)
    return launch_few<RT, 1, true>(a, blocks(gather_bound(a)), s);
  return launch_few<RT, 1, false>(a, blocks(mean > 16 ? likely16 : tile_bound(a, 16)), s);
}

}  // namespace

cudaError_t launch_adapters(const AdapterArgs& a, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
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
  if (T > 0 && (R < 1 || !ok(x, ldx, H) || !ok(base, ldb, N) || !ok(out, ldo, N) || !starts || !slot))
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
