// moe_fp8_linear in tiles of 128 rows on tcgen05.
//
// Both operands go to the tensor cores as stored codes (kind::f8f6f4, M = 128 rows of x, N = BN weight rows, K = 32; TMA tiles in
// the 128-byte swizzle).  Their scales change every 128 columns, so each group's partial sum goes to a tensor-memory
// buffer of its own, and promoting warps read it back, scale it and add it to sums that they keep in registers, while the MMAs
// of the next groups fill the other buffers.  16384 x 2048 x 4096 takes 147 us (1.87 PFLOP/s), x 4096 267 us (2.06 PFLOP/s), the tensor
// pipe busy for 40% of it: what paces the tiles is the promotion, 64 sums a thread and group, and the L2's rate (48 KB per 8.4 MFLOP).
#include <cudaTypedefs.h>

#include "moe_dec.cuh"
#include "moe_fp8.cuh"
#include "moe_tc.cuh"

namespace moe {

using namespace tc;

namespace {

__device__ int g_fp8_error;  // kDevOk or the first failure: the call has no workspace of its own to keep one in

constexpr int kM = 128, kTileA = kM * 128;  // rows of x per tile; bytes of its group of 128 columns

template <int BN>
struct Shape {
  static constexpr int kPromote = BN / 16;  // warps: a row per thread, 64 columns per warp
  // A warp of its own brings the groups' scales where 96 registers a thread leave nothing for it (as it is they spill 20 bytes, 28 with pairs, 56
  // with pairs that cross blocks; each promoting thread loading its
  // row's, each from a line of its own: 16384 x 4096 x 4096 359 us).  For BN = 64 a seventh warp would cost the others 40 registers.
  static constexpr bool kScaleWarp = BN == 256;
  static constexpr int kThreads = 32 * (kPromote + 2 + kScaleWarp);
  static constexpr int kStage = kTileA + BN * 128;
  // A stage comes back thousands of cycles after it was freed, a group's MMAs take 640: the more stages the better, and the outputs make
  // do with 2 KB per warp.
  static constexpr int kStages = BN == 256 ? 4 : 3;
  static constexpr int kBuffers = BN == 256 ? 2 : 4;
  static constexpr int kBox = BN == 256 ? 2048 : 4096;  // per promoting warp: outputs on their way
  static constexpr int kSmem = 1024 + kStages * kStage + kPromote * kBox;
};

struct Args {
  CUtensorMap x, w, out, base;
  Fp8LinearArgs l;
  int tiles_m, tiles_n;
  int box_m;   // rows of x that a tile's copies ask for
  bool boxed;  // outputs leave (and base comes) by TMA, 32 rows of a warp's columns at a time
};

// 32 lanes x 8 columns
__device__ __forceinline__ void tmem_ld_32x8(uint32_t taddr, uint32_t* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr)
               : "memory");
}
// Two sums at once: a += p f, b += q g.
__device__ __forceinline__ void fma2(float& a, float& b, uint32_t p, uint32_t q, float f, float g) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n mov.b64 z, {%4, %5};\n fma.rn.f32x2 x, y, z, x;\n"
      " mov.b64 {%0, %1}, x;\n}"
      : "+f"(a), "+f"(b)
      : "r"(p), "r"(q), "f"(f), "f"(g));
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void store_remote4(uint32_t addr, uint32_t rank, const float* v) {
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n st.shared::cluster.v4.f32 [a], {%2, %3, %4, %5};\n}" ::"r"(addr),
               "r"(rank), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
               : "memory");
}

// A warp's W outputs of each of its 32 rows (lane r holds row r's, from column c0 on) with base added, through the warp's box of
// shared memory, so that lanes write side by side: columns of any alignment (a lane's own row at a time, 1237 x 1111 fp32 outputs took
// 20 us).  Element (r, c) stands at column c ^ r: neither a row nor a column meets a bank twice.
template <class T, int W>
__device__ __forceinline__ void store_columns(const Fp8LinearArgs& l, float* box, int64_t row0, int c0, const float* y, int lane) {
  constexpr int kRows = 32 / W;  // rows written at a time
  __syncwarp();
#pragma unroll
  for (int j = 0; j < W; ++j) box[lane * W + (j ^ (lane % W))] = y[j];
  __syncwarp();
  const int c = c0 + lane % W;
  T* out = (T*)l.out + c;
  const T* base = (const T*)l.base + c;
  const bool in = c < l.out_n;
  constexpr int kAtOnce = W == 32 ? 32 : 8;  // rows (or sets of them) whose base is loaded first
#pragma unroll 1
  for (int i0 = 0; i0 < 32; i0 += kAtOnce * kRows) {
    float v[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int r = i0 + i * kRows + lane / W;
      v[i] = l.base && in && r < 32 && row0 + r < l.T ? to_f32(base[(row0 + r) * l.ldb]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int r = i0 + i * kRows + lane / W;
      if (in && r < 32 && row0 + r < l.T) from_f32(box[r * W + (lane % W ^ (r % W))] + v[i], out + (row0 + r) * l.ldo);
    }
  }
}
template <int n, int most>
__device__ __forceinline__ void store_any_columns(const Fp8LinearArgs& l, float* box, int64_t row0, int c0, const float* y, int lane) {
  constexpr int W = n < most ? n : most;
#pragma unroll
  for (int j = 0; j < n; j += W) {
    if (l.out_dtype == MOE_DT_F32) store_columns<float, W>(l, box, row0, c0 + j, y + j, lane);
    else if (l.out_dtype == MOE_DT_F16) store_columns<__half, W>(l, box, row0, c0 + j, y + j, lane);
    else store_columns<__nv_bfloat16, W>(l, box, row0, c0 + j, y + j, lane);
  }
}

// The same for 16-bit outputs whose rows TMA can store: 32 of them per lane into the box, 64-byte rows whose 16-byte parts are
// XORed with half the row, where base already stands if there is one.
__device__ __forceinline__ void fill_box(char* box, int out_dtype, bool base, const float* y, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4* at = (uint4*)(box + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4));
    uint32_t w[4];
    if (base) {
      const uint4 u = *at;
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = y[8 * j + 2 * i], b = y[8 * j + 2 * i + 1];
      if (out_dtype == MOE_DT_F16) {
        const float2 v = base ? __half22float2(*(const __half2*)&w[i]) : make_float2(0.f, 0.f);
        const __half2 h = __floats2half2_rn(a + v.x, b + v.y);
        w[i] = *(const uint32_t*)&h;
      } else {
        const float2 v = base ? make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)) : make_float2(0.f, 0.f);
        const __nv_bfloat162 h = __floats2bfloat162_rn(a + v.x, b + v.y);
        w[i] = *(const uint32_t*)&h;
      }
    }
    *at = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(m), "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// A tile per cluster of SPLIT blocks, which share its groups of columns and join their sums through each other's shared memory;
// SPLIT = 1: blocks walk the tiles.  MODE 1, 2 (PAIR): the tile's weight rows are BN / 2 gates and the same features' ups; a thread's sums
// are then 32 of each (alternating, so that a factor had to be chosen for each, 1024 x 2048 x 6000 took twice as long).
template <int BN, int MODE, int SPLIT>
__global__ void __launch_bounds__(Shape<BN>::kThreads, BN == 256 ? 1 : 2) fp8_tile_kernel(const __grid_constant__ Args a) {
  using S = Shape<BN>;
  constexpr bool PAIR = MODE != 0, CROSS = MODE == 2;
  constexpr int kBufs = S::kBuffers, kStages = S::kStages;
  extern __shared__ __align__(1024) char smem_raw[];
  char* ring = (char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t full[kStages], empty[kStages], pfull[kBufs], pempty[kBufs], bfull[S::kPromote], drain;
  __shared__ float s_x[kBufs][kM], s_w[kBufs][4];  // a group's scales: of the rows; of the blocks of weight rows, and 1 where some may not meet
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const Fp8LinearArgs& l = a.l;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kProd = S::kPromote, kMma = S::kPromote + 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&pfull[i], S::kScaleWarp ? 2 : 1);
      mbar_init(&pempty[i], S::kPromote);
    }
    for (int i = 0; i < S::kPromote; ++i) mbar_init(&bfull[i], 1);
    mbar_init(&drain, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == kMma) {
    tmem_alloc(&s_tmem, kBufs * BN);
    tmem_relinquish();
  }
  if (warp == kProd && lane == 0) {
    prefetch_tmap(&a.x);
    prefetch_tmap(&a.w);
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = s_tmem;
  const int rank = SPLIT > 1 ? (int)cluster_rank() : 0;
  const int tiles = a.tiles_m * a.tiles_n, first = blockIdx.x / SPLIT, stride = gridDim.x / SPLIT;
  // kHigh tiles along the rows, then the next along the outputs: those that are worked on at a time, 152 or 304, share x and w in L2
  // (all rows first: 16384 x 4096 x 4096 took 406 us for 341)
  constexpr int kHigh = BN == 256 ? 12 : 24;
  auto place = [&](int i, int& row, int& col) {
    const int band = i / (kHigh * a.tiles_n), j = i - band * kHigh * a.tiles_n, h = min(kHigh, a.tiles_m - kHigh * band);
    row = kM * (kHigh * band + j % h);
    col = (PAIR ? BN / 2 : BN) * (j / h);
  };
  // this block's groups of columns
  const int g0 = SPLIT > 1 ? l.groups * rank / SPLIT : 0, g1 = SPLIT > 1 ? l.groups * (rank + 1) / SPLIT : l.groups;
  pdl_wait();
  pdl_trigger();

  if (warp == kProd) {
    int armed = 0;
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int i = first; ok && i < tiles; i += stride) {
        int row, n0;
        place(i, row, n0);
        const int n1 = PAIR ? l.out_n + n0 : n0 + BN / 2;
        for (int g = g0; g < g1; ++g, ++it) {
          const int st = it % kStages;
          ok = mbar_wait(&empty[st], ((it / kStages) & 1) ^ 1, &s_abort);
          if (!ok) break;
          char* to = ring + st * S::kStage;
          mbar_arrive_expect_tx(&full[st], 128 * (a.box_m + BN));
          armed = it + 1;
          tma_load_2d(to, &a.x, &full[st], 128 * g, row);
          tma_load_2d(to + kTileA, &a.w, &full[st], 128 * g, n0);
          tma_load_2d(to + kTileA + BN * 64, &a.w, &full[st], 128 * g, n1);
        }
      }
      if (s_abort) {  // let every issued copy land before shared memory goes away
        volatile int no_abort = 0;
        for (int n = armed > kStages ? armed - kStages : 0; n < armed; ++n) mbar_wait(&full[n % kStages], (n / kStages) & 1, &no_abort);
      }
    }
    __syncwarp();
  } else if (warp == kMma) {
    const uint32_t idesc = dec::idesc_e4m3_f32(kM, BN);
    int it = 0;
    bool ok = true;
    for (int i = first; ok && i < tiles; i += stride)
      for (int g = g0; ok && g < g1; ++g, ++it) {
        const int st = it % kStages, b = it % kBufs;
        ok = mbar_wait(&pempty[b], ((it / kBufs) & 1) ^ 1, &s_abort) && mbar_wait(&full[st], (it / kStages) & 1, &s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        fence_after_sync();
        if (lane == 0) {
          const uint32_t xa = smem_u32(ring + st * S::kStage), wa = xa + kTileA;
#pragma unroll
          for (int k = 0; k < 4; ++k) dec::mma_f8_ss(tmem + b * BN, sdesc_k_sw128(xa + 32 * k), sdesc_k_sw128(wa + 32 * k), idesc, k != 0);
          mma_commit(&empty[st]);
          mma_commit(&pfull[b]);
        }
        __syncwarp();
      }
    if (lane == 0) mma_commit(&drain);
    __syncwarp();
  } else if (S::kScaleWarp && warp == kMma + 1) {
    // The scales of a group's 128 rows and of its blocks of weight rows, loaded a group ahead.
    int it = 0;
    bool ok = true;
    for (int i = first; ok && i < tiles; i += stride) {
      int row0, n0;
      place(i, row0, n0);
      const int block = lane == 0 ? n0 / 128 : PAIR ? (l.out_n + n0) / 128 + lane - 1 : n0 / 128 + 1;
      const float *w = l.ws + (int64_t)min(block, (l.N - 1) / 128) * l.groups, *x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = l.qs + min((int64_t)row0 + 32 * j + lane, (int64_t)l.T - 1) * l.groups;
      float sx[4], sw = 0.f;
      auto load = [&](int g) {
#pragma unroll
        for (int j = 0; j < 4; ++j) sx[j] = x[j][g];
        if (lane < 3) sw = w[g];
      };
      load(g0);
      for (int g = g0; g < g1; ++g, ++it) {
        const int b = it % kBufs;
        ok = __all_sync(0xffffffffu, mbar_wait(&pempty[b], ((it / kBufs) & 1) ^ 1, &s_abort));
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) s_x[b][32 * j + lane] = sx[j];
        const bool moderate = scale_moderate(sx[0]) && scale_moderate(sx[1]) && scale_moderate(sx[2]) && scale_moderate(sx[3]) && (lane >= 3 || scale_moderate(sw));
        const bool apart = !__all_sync(0xffffffffu, moderate);
        if (lane < 4) s_w[b][lane] = lane < 3 ? sw : apart ? 1.f : 0.f;
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[b]);
        if (g + 1 < g1) load(g + 1);
      }
    }
  } else {
    const int q = warp & 3, grp = warp >> 2;  // tensor-memory lanes of this warp; its columns
    int it = 0;
    uint32_t box_phase = 0;
    bool ok = true;
    char* box = ring + kStages * S::kStage + warp * S::kBox;
    for (int i = first; ok && i < tiles; i += stride) {
      int row0, n0;
      place(i, row0, n0);
      row0 += 32 * q;
      // the weight rows of the thread's columns: 64 from c on, or (PAIR) 32 gates from c on and 32 ups.  CROSS: ups may get into another
      // block of rows, `cross` columns from their first.
      const int c = n0 + (PAIR ? 32 : 64) * grp, up = l.out_n + c, cross = CROSS ? 128 - up % 128 : 128;
      const int block = PAIR ? 1 + up / 128 - (l.out_n + n0) / 128 : c / 128 - n0 / 128;  // whose scale, of s_w
      const int last = (l.N - 1) / 128;
      const float *sx = l.qs + min((int64_t)row0 + lane, (int64_t)l.T - 1) * l.groups, *sa = l.ws + (int64_t)min(c / 128, last) * l.groups;
      const float *sb = PAIR ? l.ws + (int64_t)min(up / 128, last) * l.groups : sa, *sc = CROSS ? l.ws + (int64_t)min(up / 128 + 1, last) * l.groups : sa;
      const bool some = row0 < l.T && c < l.out_n;  // the warp has outputs
      // the box, free again, and base's 32 columns from c0 on into it (lane 0)
      auto open_box = [&](int c0) {
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        if (l.base && c0 < l.out_n) {
          mbar_arrive_expect_tx(&bfull[warp], 32 * 64);
          tma_load_2d(box, &a.base, &bfull[warp], c0, row0);
        }
      };
      if (SPLIT == 1 && a.boxed && some && lane == 0) open_box(c);
      __syncwarp();
      float acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0.f;
      for (int g = g0; g < g1; ++g, ++it) {
        const int b = it % kBufs;
        float s, wa, wb = 0.f, wc = 0.f;
        if (!S::kScaleWarp) {
          s = sx[g], wa = __ldg(sa + g);
          if (PAIR) wb = __ldg(sb + g);
          if (CROSS && cross < 32) wc = __ldg(sc + g);
        }
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&pfull[b], (it / kBufs) & 1, &s_abort));
        if (!ok) break;
        fence_after_sync();
        if (S::kScaleWarp) {
          s = s_x[b][32 * q + lane], wa = s_w[b][PAIR ? 0 : block];
          if (PAIR) wb = s_w[b][block];
          if (CROSS) wc = s_w[b][min(block + 1, 2)];
        }
        const uint32_t at = taddr(tmem, 32 * q, b * BN);
        auto columns = [&](int h) { return at + (PAIR ? (h < 32 ? h : BN / 2 + h - 32) + 32 * grp : h + 64 * grp); };
        auto release = [&]() {
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pempty[b]);
        };
        constexpr int kAtOnce = CROSS ? 16 : 32;  // sums per wait, as registers allow (16384 x 2048 x 4096: 32 143 us, 16 148; CROSS: 16 45, 32 59)
        uint32_t p[kAtOnce];
        if (!S::kScaleWarp) {  // (the scales come meanwhile)
#pragma unroll
          for (int j = 0; j < kAtOnce; j += 16) tmem_ld_32x16(columns(0) + j, p + j);
        }
        const bool apart = S::kScaleWarp ? s_w[b][3] != 0.f
                                         : !__all_sync(0xffffffffu, scale_moderate(s) && scale_moderate(wa) && (!PAIR || scale_moderate(wb)) &&
                                                                        (!CROSS || cross >= 32 || scale_moderate(wc)));
        // Rare, and eight sums at a time, so that it asks for no more registers than the other way.  (To have it at all takes 147 us for 143 at
        // 16384 x 2048 x 4096.)
        if (apart) {
          if (!S::kScaleWarp) tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 64; h += 8) {
            const bool ups = PAIR && h >= 32;
            tmem_ld_32x8(columns(h), p);
            if (S::kScaleWarp) {  // (read again, for the same reason)
              s = ((volatile float*)s_x[b])[32 * q + lane], wa = ((volatile float*)s_w[b])[PAIR && !ups ? 0 : block];
              if (CROSS && ups) wc = ((volatile float*)s_w[b])[min(block + 1, 2)];
            } else if (ups) {
              wa = wb;
            }
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float w = CROSS && ups && h - 32 + j >= cross ? wc : wa;
              acc[h + j] = fmaf(__uint_as_float(p[j]) * scale_before(w, s), scale_after(w, s), acc[h + j]);
            }
          }
          release();
          continue;
        }
        const float fa = s * wa, fb = PAIR ? s * wb : fa, fc = CROSS ? s * wc : fb;
#pragma unroll
        for (int h = 0; h < 64; h += kAtOnce) {
          if (h > 0 || S::kScaleWarp) {
#pragma unroll
            for (int j = 0; j < kAtOnce; j += 16) tmem_ld_32x16(columns(h) + j, p + j);
          }
          tmem_ld_wait();
          if (h + kAtOnce == 64) release();
          const float f = PAIR && h >= 32 ? fb : fa;
          if (CROSS && h >= 32 && cross < 32) {
#pragma unroll
            for (int j = 0; j < kAtOnce; j += 2)
              fma2(acc[h + j], acc[h + j + 1], p[j], p[j + 1], h - 32 + j < cross ? fb : fc, h - 31 + j < cross ? fb : fc);
          } else {
#pragma unroll
            for (int j = 0; j < kAtOnce; j += 2) fma2(acc[h + j], acc[h + j + 1], p[j], p[j + 1], f, f);
          }
        }
      }
      if constexpr (SPLIT == 1) {
        constexpr int kMine = PAIR ? 32 : 64;
        if constexpr (PAIR) {
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[j] = silu_mul(acc[j], acc[32 + j]);
        }
        if (a.boxed && some) {
#pragma unroll
          for (int h = 0; h < kMine; h += 32) {
            if (c + h >= l.out_n) break;
            if (h > 0) {
              if (lane == 0) open_box(c + h);
              __syncwarp();
            }
            if (l.base) {  // (whoever has given up: nothing is in flight into the box when the block ends)
              volatile int alone = 0;
              const bool came = mbar_wait(&bfull[warp], box_phase, &alone);
              box_phase ^= 1;
              if (!came) s_abort = 1;
              ok = __all_sync(0xffffffffu, ok && came);
            }
            if (ok) {
              fill_box(box, l.out_dtype, l.base != nullptr, acc + h, lane);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) tma_store_2d(&a.out, box, c + h, row0);
            }
          }
        } else if (ok && some) {
          store_any_columns<kMine, S::kBox / 128>(l, (float*)box, row0, c, acc, lane);
        }
      } else {
        // Every block takes 64 / SPLIT of a thread's sums from all of them.  Its ring is free: the MMAs that read it are done.
        constexpr int kMine = 64 / SPLIT;
        float* meet = (float*)ring;  // [from][sum / 4][thread][4]
        constexpr int kThr = 32 * S::kPromote;
        __syncwarp();
        cluster_arrive();
        cluster_wait();
#pragma unroll
        for (int to = 0; to < SPLIT; ++to)
#pragma unroll
          for (int j = 0; j < kMine; j += 4) {
            const int from = !PAIR ? kMine * to + j : j < kMine / 2 ? kMine / 2 * to + j : 32 + kMine / 2 * (to - 1) + j;
            store_remote4(smem_u32(meet + ((rank * (kMine / 4) + j / 4) * kThr + threadIdx.x) * 4), to, acc + from);
          }
        cluster_arrive();
        cluster_wait();
        float y[kMine];
#pragma unroll
        for (int j = 0; j < kMine; ++j) y[j] = 0.f;
        for (int from = 0; from < SPLIT; ++from)
#pragma unroll
          for (int j = 0; j < kMine; j += 4) {
            const float4 v = *(const float4*)(meet + ((from * (kMine / 4) + j / 4) * kThr + threadIdx.x) * 4);
            y[j] += v.x, y[j + 1] += v.y, y[j + 2] += v.z, y[j + 3] += v.w;
          }
        constexpr int kOut = PAIR ? kMine / 2 : kMine;
        if constexpr (PAIR) {
#pragma unroll
          for (int j = 0; j < kOut; ++j) y[j] = silu_mul(y[j], y[kOut + j]);
        }
        if (ok && some) store_any_columns<kOut, S::kBox / 128>(l, (float*)(ring + kStages * S::kStage + warp * S::kBox), row0, c + kOut * rank, y, lane);
      }
    }
  }
  if (SPLIT > 1 && warp >= kProd) {  // the promoters' two meetings
    __syncwarp();
    for (int i = 0; i < 2; ++i) {
      cluster_arrive();
      cluster_wait();
    }
  }
  if (warp < kProd && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // outputs have left
  {
    volatile int no_abort = 0;
    if (!mbar_wait(&drain, 0, &no_abort)) s_abort = 1;  // bounded; every MMA of this block has completed
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (threadIdx.x == 0 && s_abort) set_dev_error(&g_fp8_error, kDevTimeout);
  if (warp == kMma) tmem_dealloc(tmem, kBufs * BN);
}

template <int BN, int MODE, int SPLIT>
cudaError_t launch(const Fp8LinearArgs& l, cudaStream_t s) {
  using S = Shape<BN>;
  constexpr bool PAIR = MODE != 0;
  static SmemOptIn opt_in;
  if (const cudaError_t e = opt_in(fp8_tile_kernel<BN, MODE, SPLIT>, S::kSmem); e != cudaSuccess) return e;
  Args a;
  a.l = l;
  a.tiles_m = (l.T + kM - 1) / kM;
  a.tiles_n = (l.out_n + (PAIR ? BN / 2 : BN) - 1) / (PAIR ? BN / 2 : BN);
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  // No more rows than there are, in 32s: what is left of a single tile multiplies whatever stands in shared memory, into rows that
  // are not stored.  (Copies of 128 rows of a matrix of fewer than 32 took almost twice as long: 20 x 4096 x 14336 34.8 us, 32 rows 20.6.)
  a.box_m = l.T < kM ? (l.T + 31) / 32 * 32 : kM;
  if (!tc_make_map(&a.x, u8, l.x, l.K, l.T, l.ldx, 128, a.box_m, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc_make_map(&a.w, u8, l.w, l.K, l.N, l.K, 128, BN / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  a.boxed = false;
  // (a TMA store clips a row of odd length at 16 bytes, not at the element: such rows are stored by the lanes)
  if (SPLIT == 1 && l.out_dtype != MOE_DT_F32 && l.out_n % 8 == 0 && (uintptr_t)l.out % 16 == 0 && (uintptr_t)l.base % 16 == 0 && l.ldo % 8 == 0 &&
      (!l.base || l.ldb % 8 == 0)) {
    const auto type = CU_TENSOR_MAP_DATA_TYPE_UINT16;
    const auto sw = CU_TENSOR_MAP_SWIZZLE_64B;
    if (!tc_make_map(&a.out, type, l.out, l.out_n, l.T, 2 * l.ldo, 32, 32, sw) ||
        (l.base && !tc_make_map(&a.base, type, l.base, l.out_n, l.T, 2 * l.ldb, 32, 32, sw)))
      return cudaErrorInvalidValue;
    a.boxed = true;
  }
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = SPLIT;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT > 1 ? 2 : 1;
  const int64_t most = SPLIT > 1 ? tiles : (int64_t)tc_num_sms() * (BN == 256 ? 1 : 2);
  cfg.gridDim = dim3((unsigned)((tiles < most ? tiles : most) * SPLIT));
  note_launches(1);
  return cudaLaunchKernelEx(&cfg, fp8_tile_kernel<BN, MODE, SPLIT>, a);
}

template <int MODE>
cudaError_t choose(const Fp8LinearArgs& l, cudaStream_t s) {
  constexpr bool PAIR = MODE != 0;
  const int64_t rows = (l.T + kM - 1) / kM, sms = tc_num_sms();
  auto tiles = [&](int bn) { return rows * ((l.out_n + (PAIR ? bn / 2 : bn) - 1) / (PAIR ? bn / 2 : bn)); };
  // Tiles of 256 columns from half of one wave on (us, 64 and 256: 512 x 2048 x 4096, 64 tiles, 10.9 and 13; 600 x 4096 x 4096, 80 tiles,
  // 31.4 and 29.6; 1024 x 2048 x 4096 18.5 and 13.3); a single row of tiles streams weights, and more and smaller tiles do that better
  // (128 x 2048 x 40960 27.7 and 30.4).
  if (rows > 1 && tiles(256) * 2 >= sms) return launch<256, MODE, 1>(l, s);
  const int64_t n = tiles(64);
  // K split where that leaves every block an SM of its own and each share two groups or more: the blocks' meetings cost over a
  // microsecond (us, SPLIT 1, 2 and 4: 64 x 2048 x 1024, 16 tiles, 9.8, 8.9 and 7.1; 32 x 2048 x 4096, 64 tiles, 11.3, 11.0 and 12.1;
  // 256 x 2048 x 4096, 128 tiles, 10.1, 10.4 and 17.3; 128 x 512 x 2048, 32 tiles of 4 groups, 4.4, 6.1 and 5.6).
  if (n * 2 > sms || l.groups < 8) return launch<64, MODE, 1>(l, s);
  return n * 4 > sms ? launch<64, MODE, 2>(l, s) : launch<64, MODE, 4>(l, s);
}

}  // namespace

cudaError_t launch_fp8_tiles(const Fp8LinearArgs& l, cudaStream_t s) {
  if (l.out_n == l.N) return choose<0>(l, s);
  return l.out_n % 32 == 0 ? choose<1>(l, s) : choose<2>(l, s);
}

}  // namespace moe

extern "C" moe_status_t moe_get_fp8_linear_error(moe_stream_t stream, int32_t* code) {
  using namespace moe;
  if (!code) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  int32_t v = 0;
  const int zero = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_fp8_error, sizeof(v), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess ||
      cudaMemcpyToSymbolAsync(g_fp8_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return MOE_ERR_CUDA;
  *code = v;
  return MOE_OK;
}
