// Request adapters for long requests: tiles of 128 tokens of one request, both products on the
// 5th-generation tensor cores.
//
//   v = X A^T        M = 128 tokens, N = the adapter's rank (in steps of 16), K = H
//   out = base + (scale v) B^T   M = 128, N = 128 columns at a time, K = rank, three times: v enters as three
//                                bf16 terms, each the rest of the one before (24 bits of significand)
//
// X and A, then B and base, arrive by TMA in the 128-byte swizzle that the MMA reads, through one ring of
// shared memory that is cut into K stages for the first product and two stages of column blocks for the
// second.  v goes from tensor memory through registers (scaled, split, zero past the adapter's rank) back
// into tensor memory as the second product's A operand.  The accumulator of the second product has two
// 128-column buffers (the first one lies where v's sums were), so the epilogue of one column block runs
// under the MMAs of the next.  A 5-D tensor map deals B's rows so that a lane's accumulator fragment is 16
// consecutive output columns: out is then written in whole lines straight from registers (natural order,
// with a way through shared memory, where N or out's rows do not allow it: 55.0 us for 41.3, with two terms of v).
// Where there are few tiles, the blocks of a cluster share one: each takes a part of K, the parts of v are
// summed in block order through distributed shared memory, and each takes a part of N.
//
// 16384 tokens of 16 requests, 2048 -> 2048: 40.8 us at rank 64, 50.8 at 128, against 31.4 and 32.6 by HBM (in a CUDA
// graph; with two terms of v, in shared memory, 40.2 and 49.3; register MMAs in tiles of 64: 76 and 133).  By a clock
// trace at rank 64, of the form with two terms, the first product takes 16 us, the second 17.  With two K stages the
// first took 20: 19 without A's copies, 12 without x's, 19 without the MMAs.  So the copies pace it, at about 2.6 ns per
// 128-byte row and SM, and neither the MMAs nor HBM alone.
// 4096 tokens at rank 64: 21.7 us with four blocks per tile (31.4 with one, and two terms).
//
// Every wait gives up after about a second (moe_tc.cuh); the block then waits, with the same limit, for
// its own copies and MMAs, frees its tensor memory, leaves its rows unfinished and records a timeout that
// moe_get_adapter_error reads.
#include <cooperative_groups.h>
#include <cudaTypedefs.h>
#include <string.h>

#include <atomic>

#include "moe_adapter.cuh"
#include "moe_tc.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

using namespace tc;

__device__ int g_adapter_error;  // kDevOk or the first failure

constexpr int kBM = 128, kEpiWarps = 8, kTileWarps = kEpiWarps + 3, kMaxSlots = 8;
constexpr int kAtom = 128 * 128;  // bytes: 128 rows of 64 bf16 columns in the 128-byte swizzle
// Columns of tensor memory: two accumulators of 128, then v's terms, 64 each (128 ranks, two to a column).
constexpr int kTermCol = 256, kTermCols = 64, kTmemCols = 512;
constexpr int kSmem = 225 * 1024;  // most that a block takes (one per SM): 1 KB alignment, v's parts, two N stages

struct TileArgs {
  CUtensorMap x, a, b, y;
  AdapterArgs g;
  int r16, katoms;    // rank in steps of 16 (all adapters), 64-column atoms of B
  int ka, kslot;      // 64-column atoms and bytes of a K stage
  int bps, nslot;     // 128-column blocks and bytes of an N stage
  int nk;             // K stages
  bool dealt;         // B's rows dealt for a direct epilogue (whole 64-column groups, 32-byte rows of out)
};

struct Bars {
  uint64_t full_k[kMaxSlots], empty_k[kMaxSlots], full_n[2], cut_n[2], empty_n[2];
  uint64_t v_sums, v_ready, acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort;
};

// Byte of column chunk j (8 bf16) of row `row` in an operand of 64-column atoms.
__device__ __forceinline__ uint32_t swz(int row, int j) {
  return (j >> 3) * kAtom + row * 128 + (((j & 7) ^ (row & 7)) << 4);
}

// 16 tensor-memory lanes x 64 columns as fragments: v[4 j + 2 u + i] is row (lane / 4) + 8 u, column
// 8 j + 2 (lane % 4) + i.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
// B's rows, 256 from row 64 g on, dealt as the epilogue wants them (rows_map).
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int g) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %4, %4, "
      "%5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(m), "r"(smem_u32(bar)), "r"(c0), "r"(0), "r"(g)
      : "memory");
}

// A wait of the clean-up: with the limit, whatever the block's state.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  int never = 0;
  mbar_wait(bar, parity, &never);
}

__global__ void __launch_bounds__(32 * kTileWarps) adapter_tile_kernel(const __grid_constant__ TileArgs p) {
  extern __shared__ unsigned char dyn[];
  __shared__ Bars bars;
  const AdapterArgs& a = p.g;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), crank = cluster.block_rank();
  const Tile tile = find_tile<kTileWarps>(a, blockIdx.x / C, kBM);
  if (tile.rows == 0) return;  // the whole cluster
  const int rk = tile.rk, steps = (rk + 15) / 16;
  if (rk == 0) {  // no adapter: base as it is
    if (a.out == a.base) return;
    const int chunks = a.N / 8;
    for (int64_t e = crank * 32 * kTileWarps + tid; e < (int64_t)tile.rows * chunks; e += C * 32 * kTileWarps) {
      const int64_t t = tile.t0 + e / chunks;
      const int c = (int)(e % chunks) * 8;
      *(uint4*)(a.out + t * a.ldo + c) = *(const uint4*)(a.base + t * a.ldb + c);
    }
    return;
  }
  // in a cluster this block's part of v's sums, [4 steps][128 rows]; then the K stages, whose memory is the two N
  // stages' later
  float4* parts = (float4*)(((uintptr_t)dyn + 1023) & ~(uintptr_t)1023);
  unsigned char* ring = (unsigned char*)parts + 2 * p.katoms * kAtom;
  const int natom = p.bps * kAtom, ybytes = p.katoms * natom;  // an atom of a stage's B; where its base begins
  // this block's part of the K stages and of the N stages (column blocks)
  const int atoms = (a.H + 63) / 64, kall = (atoms + p.ka - 1) / p.ka, kper = (kall + C - 1) / C;
  const int k0 = min(crank * kper, kall), kst = min(kper, kall - k0);
  const int ball = (a.N + 127) / 128, nall = (ball + p.bps - 1) / p.bps, nper = (nall + C - 1) / C;
  const int n0 = min(crank * nper, nall), nst = min(nper, nall - n0);
  const int b0 = n0 * p.bps, nblk = max(0, min(nst * p.bps, ball - b0));
  const bool partial = rk % 16 != 0;  // the last rank step of B holds columns that are not the adapter's
  if (tid == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(&bars.full_k[i], 1);
      mbar_init(&bars.empty_k[i], 1);
    }
    mbar_init(&bars.v_sums, 1);
    mbar_init(&bars.v_ready, 32 * kEpiWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.full_n[i], 1);
      mbar_init(&bars.cut_n[i], 1);
      mbar_init(&bars.empty_n[i], 1 + kEpiWarps);
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], kEpiWarps);
    }
    mbar_init(&bars.done, 1);
    bars.abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(&bars.tmem, kTmemCols);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = bars.tmem;
  volatile int* abort = &bars.abort;

  const int quarter = warp & 3, half = warp >> 2;  // of the epilogue's warps: tensor-memory lanes, columns
  int kdone = 0, n = 0;                            // copies issued: K stages, N stages
  bool ok = true;
  auto load_n = [&] {  // N stage n
    unsigned char* at = ring + (1 - (n & 1)) * p.nslot;
    uint64_t* full = &bars.full_n[n & 1];
    const int c0 = 128 * p.bps * (n0 + n);
    mbar_arrive_expect_tx(full, p.nslot);
    for (int i = 0; i < p.katoms; ++i)
      if (p.dealt) tma_load_5d(at + i * natom, &p.b, full, 64 * i, (tile.slot * a.N + c0) / 64);
      else tma_load_2d(at + i * natom, &p.b, full, 64 * i, tile.slot * a.N + c0);
    if (p.dealt) tma_load_3d(at + ybytes, &p.y, full, 0, tile.t0, c0 / 64);
    else
      for (int i = 0; i < 2 * p.bps; ++i) tma_load_2d(at + ybytes + i * kAtom, &p.y, full, c0 + 64 * i, tile.t0);
    ++n;
  };

  // ---- the first product
  if (warp == kEpiWarps) {  // copies
    if (lane == 0) {
      prefetch_tmap(&p.x);
      prefetch_tmap(&p.a);
      prefetch_tmap(&p.b);
      prefetch_tmap(&p.y);
      for (; kdone < kst; ++kdone) {
        const int s = kdone % p.nk, u = kdone / p.nk, k = k0 + kdone;
        if (u > 0 && !mbar_wait(&bars.empty_k[s], (u - 1) & 1, abort)) break;
        unsigned char* at = ring + s * p.kslot;
        mbar_arrive_expect_tx(&bars.full_k[s], p.kslot);
        if (p.ka == 1) {
          tma_load_2d(at, &p.x, &bars.full_k[s], 64 * k, tile.t0);
          tma_load_2d(at + kAtom, &p.a, &bars.full_k[s], 64 * k, tile.slot * a.r);
        } else {  // atoms past H arrive as zeros
          tma_load_3d(at, &p.x, &bars.full_k[s], 0, tile.t0, p.ka * k);
          tma_load_3d(at + p.ka * kAtom, &p.a, &bars.full_k[s], 0, tile.slot * a.r, p.ka * k);
        }
      }
      ok = kdone == kst && mbar_wait(&bars.v_sums, 0, abort);  // every K stage has been read
      while (ok && n < nst && n < 2) load_n();
    }
  } else if (warp == kEpiWarps + 1) {  // MMAs
    if (lane == 0) {
      const uint32_t id1 = idesc_bf16_f32(128, 16 * steps);
      for (int k = 0; ok && k < kst; ++k) {
        const int s = k % p.nk;
        ok = mbar_wait(&bars.full_k[s], (k / p.nk) & 1, abort);
        if (!ok) break;
        fence_after_sync();
        const uint32_t xs = smem_u32(ring + s * p.kslot), as = xs + p.ka * kAtom;
        const int here = min(atoms - p.ka * (k0 + k), p.ka);
        for (int i = 0; i < 4 * here; ++i)
          mma_f16_ss(tmem, sdesc_k_sw128(xs + (i >> 2) * kAtom + (i & 3) * 32),
                     sdesc_k_sw128(as + (i >> 2) * p.r16 * 128 + (i & 3) * 32), id1, (k | i) != 0);
        mma_commit(&bars.empty_k[s]);
      }
      if (ok) mma_commit(&bars.v_sums);
    }
  } else if (warp < kEpiWarps) {
    ok = __all_sync(0xffffffffu, mbar_wait(&bars.v_sums, 0, abort));
    fence_after_sync();
  }
  __syncwarp();

  // ---- v: from tensor memory (in a cluster: every block's part of K, summed in block order) back to it, scaled, in
  // three terms, zero past the rank.  A thread has one row and every second rank step.
  const int row = 32 * quarter + lane;
  auto split = [&](int i, const float* f) {  // rank step half + 2 i
    const int s = half + 2 * i;
    uint32_t w[3][8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const Terms t = split_pair(16 * s + 2 * c < rk ? f[2 * c] * tile.scale : 0.f,
                                 16 * s + 2 * c + 1 < rk ? f[2 * c + 1] * tile.scale : 0.f);
      w[0][c] = t.lo;
      w[1][c] = t.mid;
      w[2][c] = t.hi;
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) tmem_st_32x8(taddr(tmem, 32 * quarter, kTermCol + j * kTermCols + 8 * s), w[j]);
  };
  if (warp < kEpiWarps && ok) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (half + 2 * i < steps) {
        uint32_t w[16];
        tmem_ld_32x16(taddr(tmem, 32 * quarter, 16 * (half + 2 * i)), w);
        tmem_ld_wait();
        if (C == 1) {
          split(i, (const float*)w);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            parts[(4 * (half + 2 * i) + c) * 128 + row] =
                kst > 0 ? make_float4(__uint_as_float(w[4 * c]), __uint_as_float(w[4 * c + 1]),
                                      __uint_as_float(w[4 * c + 2]), __uint_as_float(w[4 * c + 3]))
                        : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
  }
  if (C > 1) {
    cluster.sync();
    if (warp < kEpiWarps) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (half + 2 * i < steps) {
          float f[16];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float4* at = &parts[(4 * (half + 2 * i) + c) * 128 + row];
            float4 q = *cluster.map_shared_rank(at, 0);
            for (int b = 1; b < C; ++b) {
              const float4 o = *cluster.map_shared_rank(at, b);
              q.x += o.x;
              q.y += o.y;
              q.z += o.z;
              q.w += o.w;
            }
            f[4 * c] = q.x;
            f[4 * c + 1] = q.y;
            f[4 * c + 2] = q.z;
            f[4 * c + 3] = q.w;
          }
          split(i, f);
        }
    }
    cluster.sync();  // every block has read every part: a block may leave
  }

  // ---- the second product
  if (warp == kEpiWarps) {  // copies
    if (lane == 0) {
      while (ok && n < nst) {
        ok = mbar_wait(&bars.empty_n[n & 1], ((n >> 1) - 1) & 1, abort);
        if (ok) load_n();
      }
      if (*abort) {  // copies in flight land before the block leaves
        for (int i = kdone > p.nk ? kdone - p.nk : 0; i < kdone; ++i) drain(&bars.full_k[i % p.nk], (i / p.nk) & 1);
        for (int i = n > 2 ? n - 2 : 0; i < n; ++i) drain(&bars.full_n[i & 1], (i >> 1) & 1);
      }
    }
  } else if (warp == kEpiWarps + 1) {  // MMAs
    if (lane == 0) {
      const uint32_t id2 = idesc_bf16_f32(128, 128);
      if (ok) ok = mbar_wait(&bars.v_ready, 0, abort);
      fence_after_sync();
      for (int b = 0; ok && b < nblk; ++b) {
        const int st = b / p.bps, sub = b % p.bps, s = st & 1, buf = b & 1;
        if (b > 1) ok = mbar_wait(&bars.acc_empty[buf], ((b >> 1) - 1) & 1, abort);
        if (ok && sub == 0) ok = mbar_wait(partial ? &bars.cut_n[s] : &bars.full_n[s], (st >> 1) & 1, abort);
        if (!ok) break;
        fence_after_sync();
        const uint32_t bs = smem_u32(ring + (1 - s) * p.nslot) + sub * kAtom, acc = tmem + 128 * buf;
        for (int i = 0; i < steps; ++i) {
          const uint64_t d = sdesc_k_sw128(bs + (i >> 2) * natom + (i & 3) * 32);
#pragma unroll
          for (int j = 0; j < 3; ++j) mma_f16_ts(acc, tmem + kTermCol + j * kTermCols + 8 * i, d, id2, (i | j) != 0);
        }
        if (sub == p.bps - 1 || b == nblk - 1) mma_commit(&bars.empty_n[s]);
        mma_commit(&bars.acc_full[buf]);
      }
      mma_commit(&bars.done);  // no arrival is on its way into this block's barriers when it leaves
      drain(&bars.done, 0);
    }
  } else if (warp == kEpiWarps + 2) {  // columns of B past the adapter's rank, where a step has some
    if (partial) {
      const int c0 = rk / 8, c1 = 2 * steps;  // 8-column chunks from the partial one on
      for (int i = 0; i < nst; ++i) {
        const int s = i & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&bars.full_n[s], (i >> 1) & 1, abort))) break;
        unsigned char* bs = ring + (1 - s) * p.nslot;
        for (int r = lane; r < 128 * p.bps; r += 32)
          for (int c = c0; c < c1; ++c) {
            uint4* q = (uint4*)(bs + (c >> 3) * natom + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            const int keep = rk - 8 * c;  // columns of the chunk that stay
            uint4 w = keep > 0 ? *q : make_uint4(0, 0, 0, 0);
            uint32_t* e = (uint32_t*)&w;
#pragma unroll
            for (int j = 0; j < 4; ++j) e[j] = keep >= 2 * j + 2 ? e[j] : keep == 2 * j + 1 ? e[j] & 0xFFFFu : 0u;
            *q = w;
          }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.cut_n[s]);
      }
    }
  } else {  // epilogue
    tmem_st_wait();
    if (ok) {
      fence_before_sync();
      mbar_arrive(&bars.v_ready);
    }
    // The accumulator's fragments: with B's rows dealt, a lane holds 16 consecutive columns of four rows of
    // the tile and four lanes a row's 128 bytes, which go out as they are.  Else it holds pairs of columns,
    // which are added in place to base in shared memory, from where the warp writes whole rows.
    const int g = lane >> 2, t = lane & 3, r0 = 32 * quarter;
    for (int b = 0; ok && b < nblk; ++b) {
      const int st = b / p.bps, sub = b % p.bps, s = st & 1, buf = b & 1, col = 128 * (b0 + b) + 64 * half;
      const bool last = sub == p.bps - 1 || b == nblk - 1;
      if (sub == 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars.full_n[s], (st >> 1) & 1, abort));
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars.acc_full[buf], (b >> 1) & 1, abort));
      if (!ok) break;
      fence_after_sync();
      uint32_t w[2][32];
      tmem_ld_16x64(taddr(tmem, r0, 128 * buf + 64 * half), w[0]);
      tmem_ld_16x64(taddr(tmem, r0 + 16, 128 * buf + 64 * half), w[1]);
      unsigned char* ys = ring + (1 - s) * p.nslot + ybytes + (2 * sub + half) * kAtom;  // base of this half
      if (p.dealt) {
        uint4 y[4][2];  // a row's pieces 2 t and 2 t + 1 (eight lanes: all banks once)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) y[i][h] = *(const uint4*)(ys + swz(r0 + g + 8 * i, 2 * t + h));
        tmem_ld_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars.acc_empty[buf]);
          if (last) mbar_arrive(&bars.empty_n[s]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + g + 8 * i;
          if (r < tile.rows && col < a.N) {
            const uint32_t* yb = (const uint32_t*)y[i];
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              o[j] = pack_bf16(lo_f32(yb[j]) + __uint_as_float(w[i >> 1][4 * j + 2 * (i & 1)]),
                               hi_f32(yb[j]) + __uint_as_float(w[i >> 1][4 * j + 2 * (i & 1) + 1]));
            st_global_v8(a.out + (int64_t)(tile.t0 + r) * a.ldo + col + 16 * t, o);
          }
        }
      } else {
        tmem_ld_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.acc_empty[buf]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {  // columns 8 j + 2 t and the next: 32 lanes on 32 banks
            uint32_t* q = (uint32_t*)(ys + swz(r0 + g + 8 * i, j)) + t;
            *q = pack_bf16(lo_f32(*q) + __uint_as_float(w[i >> 1][4 * j + 2 * (i & 1)]),
                           hi_f32(*q) + __uint_as_float(w[i >> 1][4 * j + 2 * (i & 1) + 1]));
          }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = r0 + 4 * i + (lane >> 3), c = col + 8 * (lane & 7);
          const uint4 q = *(const uint4*)(ys + swz(r, lane & 7));
          if (r < tile.rows && c < a.N) *(uint4*)(a.out + (int64_t)(tile.t0 + r) * a.ldo + c) = q;
        }
        fence_proxy_async_smem();  // the next copy into this memory comes after these accesses
        __syncwarp();
        if (lane == 0 && last) mbar_arrive(&bars.empty_n[s]);
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 0) {
    tmem_relinquish();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && bars.abort) set_dev_error(&g_adapter_error, kDevTimeout);
}

}  // namespace

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 fn = known.load(std::memory_order_relaxed);
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess)
      fn = (PFN_cuTensorMapEncodeTiled_v12000)f;
    known.store(fn, std::memory_order_relaxed);
  }
  return fn;
}

static bool bf16_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                     const cuuint32_t* box) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a [rows, cols] bf16 matrix as [cols / 64 atoms][rows][64]: one copy brings `height` rows x ka atoms.
static bool atoms_map(CUtensorMap* m, const void* base, uint64_t rows, int cols, int64_t ld, int height, int ka) {
  const cuuint64_t dims[3] = {64, rows, (cuuint64_t)cols / 64}, strides[2] = {(cuuint64_t)ld * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)height, (cuuint32_t)ka};
  return bf16_map(m, base, 3, dims, strides, box);
}

// Rows of B [rows, r], `groups` times 64, each in the order (j, a, b) of row 16 a + 2 j + b (a < 4, j < 8, b < 2): the
// accumulator's column 8 j + 2 a + b is then output column 16 a + 2 j + b, and a lane's fragment (a = lane % 4)
// 16 consecutive ones.  rows is a multiple of 64.
static bool rows_map(CUtensorMap* m, const void* base, uint64_t rows, int r, int groups) {
  const cuuint64_t one = (cuuint64_t)r * 2;
  const cuuint64_t dims[5] = {(cuuint64_t)r, 2, 4, 8, rows / 64}, strides[4] = {one, 16 * one, 2 * one, 64 * one};
  const cuuint32_t box[5] = {64, 2, 4, 8, (cuuint32_t)groups};
  return bf16_map(m, base, 5, dims, strides, box);
}

bool adapter_tiles_fit(const AdapterArgs& a) {  // rows of A and B by 32-bit coordinates; a map has some
  return a.n > 0 && (int64_t)a.n * a.N < INT32_MAX && (int64_t)a.n * a.r < INT32_MAX;
}

cudaError_t launch_adapter_tiles(const AdapterArgs& g, cudaStream_t s) {
  TileArgs p;
  memset(&p, 0, sizeof(p));
  p.g = g;
  p.r16 = (g.r + 15) / 16 * 16;
  p.katoms = (g.r + 63) / 64;
  p.bps = p.katoms == 1 ? 2 : 1;
  p.nslot = p.bps * (p.katoms + 2) * kAtom;  // B's rows and base's columns of the stage's blocks
  // K stages: four at least in the memory of the N stages, two atoms wide where that leaves as many (H in
  // whole atoms then: the 3-D maps count columns by atoms)
  const int64_t tiles = tile_bound(g, kBM);
  const int katom = kAtom + p.r16 * 128;
  p.ka = g.H % 64 == 0 && 2 * p.nslot / (2 * katom) >= 4 ? 2 : 1;
  p.kslot = p.ka * katom;
  p.nk = 2 * p.nslot / p.kslot < kMaxSlots ? 2 * p.nslot / p.kslot : kMaxSlots;
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const bool maps =
      p.ka == 1 ? tc_make_map(&p.x, bf16, g.x, g.H, g.T, (uint64_t)g.ldx * 2, 64, kBM, sw) &&
                      tc_make_map(&p.a, bf16, g.A, g.H, (uint64_t)g.n * g.r, (uint64_t)g.H * 2, 64, p.r16, sw)
                : atoms_map(&p.x, g.x, g.T, g.H, g.ldx, kBM, p.ka) &&
                      atoms_map(&p.a, g.A, (uint64_t)g.n * g.r, g.H, g.H, p.r16, p.ka);
  p.dealt = g.N % 64 == 0 && g.ldo % 16 == 0 && (uintptr_t)g.out % 32 == 0;
  const uint64_t brows = (uint64_t)g.n * g.N;
  const bool nmaps = p.dealt ? rows_map(&p.b, g.B, brows, g.r, 2 * p.bps) && atoms_map(&p.y, g.base, g.T, g.N, g.ldb, kBM, 2 * p.bps)
                             : tc_make_map(&p.b, bf16, g.B, g.r, brows, (uint64_t)g.r * 2, 64, 128 * p.bps, sw) &&
                                   tc_make_map(&p.y, bf16, g.base, g.N, g.T, (uint64_t)g.ldb * 2, 64, kBM, sw);
  if (!maps || !nmaps) return cudaErrorInvalidValue;
  static SmemOptIn opt_in;
  if (const cudaError_t e = opt_in(adapter_tile_kernel, kSmem); e != cudaSuccess) return e;
  // Blocks of a cluster share a tile, each a part of K, then of N, while the device takes the clusters at once
  // (half a tile over per request; a tenth of the SMs may not form clusters: 37 tiles by four 38 us, by two 25).
  const int64_t likely = (int64_t)g.T / kBM + (g.R < g.T ? g.R : g.T) / 2, room = tc_num_sms() * 9 / 10;
  const int cluster = 4 * likely <= room ? 4 : 2 * likely <= room ? 2 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * cluster));
  cfg.blockDim = dim3(32 * kTileWarps);
  cfg.dynamicSmemBytes = kSmem;
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
  return cudaLaunchKernelEx(&cfg, adapter_tile_kernel, p);
}

}  // namespace moe

extern "C" moe_status_t moe_get_adapter_error(moe_stream_t stream, int32_t* code) {
  using namespace moe;
  if (!code) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  int32_t v = 0;
  const int zero = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_adapter_error, sizeof(v), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess ||
      cudaMemcpyToSymbolAsync(g_adapter_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return MOE_ERR_CUDA;
  *code = v;
  return MOE_OK;
}
