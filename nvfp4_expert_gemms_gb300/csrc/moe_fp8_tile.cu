// moe_fp8_linear in tiles of 128 rows on tcgen05.
//
// Both operands go to the tensor cores as stored codes (kind::f8f6f4, M = 128 rows of x, N = BN weight rows, K = 32; TMA tiles in
// the 128-byte swizzle).  Their scales change every 128 columns, so each group's partial sum goes to a tensor-memory
// buffer of its own, and promoting warps read it back, scale it and add it to sums that they keep in registers, while the MMAs
// of the next groups fill the other buffers.
#include <cudaTypedefs.h>

#include "moe_dec.cuh"
#include "moe_fp8.cuh"
#include "moe_tc.cuh"

namespace moe {

using namespace tc;

namespace {

constexpr int kM = 128, kTileA = kM * 128;  // rows of x per tile; bytes of its group of 128 columns

template <int BN>
struct Shape {
  static constexpr int kPromote = BN / 16;  // warps: a row per thread, 64 columns per warp
  static constexpr int kThreads = 32 * (kPromote + 2);
  static constexpr int kStage = kTileA + BN * 128;
  static constexpr int kStages = BN == 256 ? 4 : 4;
  static constexpr int kBuffers = BN == 256 ? 2 : 4;
  static constexpr int kSmem = 1024 + kStages * kStage;
};

struct Args {
  CUtensorMap x, w;
  Fp8LinearArgs l;
  int tiles_m, tiles_n;
};

// 32 lanes x 8 columns of 32-bit words.
__device__ __forceinline__ void tmem_ld_32x8(uint32_t taddr, uint32_t* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr)
               : "memory");
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

// The first n of y as consecutive outputs of a row from column c0 on, with base added.
template <class T, int n>
__device__ __forceinline__ void store_row(const Fp8LinearArgs& l, int64_t row, int c0, const float* y) {
  T* out = (T*)l.out + row * l.ldo + c0;
  const T* base = l.base ? (const T*)l.base + row * l.ldb + c0 : nullptr;
  constexpr int kVec = 16 / sizeof(T);
  if (n % kVec == 0 && c0 + n <= l.out_n && (uintptr_t)out % 16 == 0 && (uintptr_t)base % 16 == 0) {
#pragma unroll
    for (int i = 0; i < n; i += kVec) {
      uint4 u;
      T* e = (T*)&u;
      float b[kVec];
      if (base) {
        u = *(const uint4*)(base + i);
#pragma unroll
        for (int j = 0; j < kVec; ++j) b[j] = to_f32(e[j]);
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) from_f32(base ? y[i + j] + b[j] : y[i + j], e + j);
      *(uint4*)(out + i) = u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (c0 + i < l.out_n) from_f32(base ? y[i] + to_f32(base[i]) : y[i], out + i);
  }
}
template <int n>
__device__ __forceinline__ void store_typed(const Fp8LinearArgs& l, int64_t row, int c0, const float* y) {
  if (l.out_dtype == MOE_DT_F32) store_row<float, n>(l, row, c0, y);
  else if (l.out_dtype == MOE_DT_F16) store_row<__half, n>(l, row, c0, y);
  else store_row<__nv_bfloat16, n>(l, row, c0, y);
}

// A tile per cluster of SPLIT blocks, which share its groups of columns and join their sums through each other's shared memory; SPLIT = 1:
// blocks walk the tiles.  PAIR: the tile's weight rows are BN / 2 gates and the same features' ups; a thread's sums
// then alternate gate, up.
template <int BN, bool PAIR, int SPLIT>
__global__ void __launch_bounds__(Shape<BN>::kThreads, 1) fp8_tile_kernel(const __grid_constant__ Args a) {
  using S = Shape<BN>;
  constexpr int kBufs = S::kBuffers, kStages = S::kStages;
  extern __shared__ __align__(1024) char smem_raw[];
  char* ring = (char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t full[kStages], empty[kStages], pfull[kBufs], pempty[kBufs], drain;
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
      mbar_init(&pfull[i], 1);
      mbar_init(&pempty[i], S::kPromote);
    }
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
  // this block's groups of columns
  const int g0 = l.groups * rank / SPLIT, g1 = l.groups * (rank + 1) / SPLIT;
  pdl_wait();
  pdl_trigger();
  // tile i: rows 128 (i % tiles_m), outputs from (BN or BN / 2) (i / tiles_m) on
  constexpr int kOut = PAIR ? BN / 2 : BN;

  if (warp == kProd) {
    int armed = 0;
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int i = first; ok && i < tiles; i += stride) {
        const int row = kM * (i % a.tiles_m), n0 = kOut * (i / a.tiles_m), n1 = PAIR ? l.out_n + n0 : n0 + BN / 2;
        for (int g = g0; g < g1; ++g, ++it) {
          const int st = it % kStages;
          ok = mbar_wait(&empty[st], ((it / kStages) & 1) ^ 1, &s_abort);
          if (!ok) break;
          char* to = ring + st * S::kStage;
          mbar_arrive_expect_tx(&full[st], S::kStage);
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
  } else {
    const int q = warp & 3, grp = warp >> 2, r = 32 * q + lane;  // tensor-memory lanes of this warp; its columns
    int it = 0;
    bool ok = true;
    for (int i = first; ok && i < tiles; i += stride) {
      const int64_t row = (int64_t)kM * (i % a.tiles_m) + r;
      const int n0 = kOut * (i / a.tiles_m);
      const float* sx = l.qs + min(row, (int64_t)l.T - 1) * l.groups;
      // the weight rows of the thread's columns: 64 from c on, or (PAIR) 32 gates from c on and 32 ups.  Ups may cross into another
      // block of rows, `cross` columns from their first.
      const int c = n0 + (PAIR ? 32 : 64) * grp, last = (l.N - 1) / 128;
      const int up = l.out_n + c, cross = PAIR ? 128 - up % 128 : 128;
      const float* sa = l.ws + (int64_t)min(c / 128, last) * l.groups;
      const float* sb = PAIR ? l.ws + (int64_t)min(up / 128, last) * l.groups : sa;
      const float* sc = PAIR ? l.ws + (int64_t)min(up / 128 + 1, last) * l.groups : sa;
      float acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0.f;
      for (int g = g0; g < g1; ++g, ++it) {
        const int b = it % kBufs;
        const float s = sx[g], fa = s * __ldg(sa + g), fb = PAIR ? s * __ldg(sb + g) : fa, fc = PAIR && cross < 32 ? s * __ldg(sc + g) : fb;
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&pfull[b], (it / kBufs) & 1, &s_abort));
        if (!ok) break;
        fence_after_sync();
        const uint32_t at = taddr(tmem, 32 * q, b * BN);
        constexpr int kAtOnce = BN == 256 ? 16 : 32;  // sums per wait: as registers allow
#pragma unroll
        for (int h = 0; h < 64; h += kAtOnce) {
          uint32_t p[kAtOnce];
          if (PAIR) {
            uint32_t e[kAtOnce];
            static_assert(kAtOnce % 16 == 0, "");
#pragma unroll
            for (int j = 0; j < kAtOnce / 2; j += 8) {
              tmem_ld_32x8(at + 32 * grp + h / 2 + j, e + j);
              tmem_ld_32x8(at + BN / 2 + 32 * grp + h / 2 + j, e + kAtOnce / 2 + j);
            }
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) p[j] = e[j / 2 + j % 2 * (kAtOnce / 2)];
          } else {
#pragma unroll
            for (int j = 0; j < kAtOnce; j += 16) tmem_ld_32x16(at + 64 * grp + h + j, p + j);
            tmem_ld_wait();
          }
          if (h + kAtOnce == 64) {
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pempty[b]);
          }
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j)
            acc[h + j] = fmaf(__uint_as_float(p[j]), !PAIR || j % 2 == 0 ? fa : (h + j) / 2 < cross ? fb : fc, acc[h + j]);
        }
      }
      if constexpr (SPLIT == 1) {
        if (ok && row < l.T) {
          if constexpr (PAIR) {
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[j] = silu_mul(acc[2 * j], acc[2 * j + 1]);
          }
          store_typed<PAIR ? 32 : 64>(l, row, c, acc);
        }
      } else {
        // Every block takes 64 / SPLIT of a thread's sums from all of them.  Its ring is free: the MMAs that read it are done.
        constexpr int kMine = 64 / SPLIT;
        float* box = (float*)ring;  // [from][sum / 4][thread][4]
        constexpr int kThr = 32 * S::kPromote;
        __syncwarp();
        cluster_arrive();
        cluster_wait();
#pragma unroll
        for (int to = 0; to < SPLIT; ++to)
#pragma unroll
          for (int j = 0; j < kMine; j += 4)
            store_remote4(smem_u32(box + ((rank * (kMine / 4) + j / 4) * kThr + threadIdx.x) * 4), to, acc + kMine * to + j);
        cluster_arrive();
        cluster_wait();
        float y[kMine];
#pragma unroll
        for (int j = 0; j < kMine; ++j) y[j] = 0.f;
        for (int from = 0; from < SPLIT; ++from)
#pragma unroll
          for (int j = 0; j < kMine; j += 4) {
            const float4 v = *(const float4*)(box + ((from * (kMine / 4) + j / 4) * kThr + threadIdx.x) * 4);
            y[j] += v.x, y[j + 1] += v.y, y[j + 2] += v.z, y[j + 3] += v.w;
          }
        if (ok && row < l.T) {
          constexpr int n = PAIR ? kMine / 2 : kMine;
          if constexpr (PAIR) {
#pragma unroll
            for (int j = 0; j < n; ++j) y[j] = silu_mul(y[2 * j], y[2 * j + 1]);
          }
          store_typed<n>(l, row, c + n * rank, y);
        }
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
  {
    volatile int no_abort = 0;
    mbar_wait(&drain, 0, &no_abort);  // bounded; every MMA of this block has completed
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == kMma) tmem_dealloc(tmem, kBufs * BN);
}

template <int BN, bool PAIR, int SPLIT>
cudaError_t launch(const Fp8LinearArgs& l, cudaStream_t s) {
  using S = Shape<BN>;
  static SmemOptIn opt_in;
  if (const cudaError_t e = opt_in(fp8_tile_kernel<BN, PAIR, SPLIT>, S::kSmem); e != cudaSuccess) return e;
  Args a;
  a.l = l;
  a.tiles_m = (l.T + kM - 1) / kM;
  a.tiles_n = (l.out_n + (PAIR ? BN / 2 : BN) - 1) / (PAIR ? BN / 2 : BN);
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!tc_make_map(&a.x, u8, l.x, l.K, l.T, l.ldx, 128, kM, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc_make_map(&a.w, u8, l.w, l.K, l.N, l.K, 128, BN / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
  const int64_t most = SPLIT > 1 ? tiles : (int64_t)tc_num_sms() * (BN == 256 ? 1 : 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tiles < most ? tiles : most) * SPLIT));
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
  note_launches(1);
  return cudaLaunchKernelEx(&cfg, fp8_tile_kernel<BN, PAIR, SPLIT>, a);
}

template <bool PAIR>
cudaError_t choose(const Fp8LinearArgs& l, cudaStream_t s) {
  const int64_t rows = (l.T + kM - 1) / kM, sms = tc_num_sms();
  auto tiles = [&](int bn) { return rows * ((l.out_n + (PAIR ? bn / 2 : bn) - 1) / (PAIR ? bn / 2 : bn)); };
  if (tiles(256) >= sms) return launch<256, PAIR, 1>(l, s);
  const int64_t n = tiles(64);
  if (n >= sms || l.groups < 2) return launch<64, PAIR, 1>(l, s);
  if (n * 2 >= sms || l.groups < 4) return launch<64, PAIR, 2>(l, s);
  return launch<64, PAIR, 4>(l, s);
}

}  // namespace

cudaError_t launch_fp8_tiles(const Fp8LinearArgs& l, cudaStream_t s) {
  return l.out_n != l.N ? choose<true>(l, s) : choose<false>(l, s);
}

}  // namespace moe
