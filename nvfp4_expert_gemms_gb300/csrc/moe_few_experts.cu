// The experts of moe_layer_few in one kernel: routing, gate/up, down and the combine.
//
// Work is cut into units of some weight rows of one expert, whole along K: first every unit of the gate/up matrices, in
// the order of the active experts, then those of the down matrices.  Blocks take them by ticket in that order, so whoever
// waits (a down unit for its expert's h) waits for units that running blocks hold and that wait for nothing: no two blocks
// have to be resident together, and calls on other streams cannot stand in the way.
//
// In a block, one warp keeps a ring of shared memory full by TMA (in flight per SM: 144 to 160 KB; weights need about
// 45 KB at HBM's rate and latency) and runs ahead of everyone, into the down matrices while h is not there yet.  Sixteen
// warps each take a piece of 128 columns (64 of bf16) of 16 rows, decode it into MMA operands and multiply it with up to
// eight tokens; four more add the pieces up, four units in flight, and finish them: h = silu(gate) up, or the weighted row
// of y.  The block that finishes the last expert's rows of some output columns sums them over each token's experts,
// in their order.
#include "moe_few.cuh"
#include "moe_formats.cuh"
#include "moe_tc.cuh"

namespace moe {

using namespace tc;

namespace {

constexpr int kMulWarps = 16, kEndWarps = 4, kProdWarp = kMulWarps + kEndWarps;
constexpr int kWarps = kProdWarp + 1, kThreads = 32 * kWarps;
constexpr int kMaxStages = 8;
constexpr int kColumns = 16;  // pieces of K per slab at most: one per multiplying warp
constexpr size_t kSmemMax = 227 * 1024 - 14 * 1024;  // beside the tables below

template <int FMT>
struct Format {
  static constexpr int kPiece = FMT == MOE_FMT_BF16 ? 64 : 128;  // columns of a piece
  static constexpr int kRowBytes = FMT == MOE_FMT_NVFP4_W4A16 || FMT == MOE_FMT_INT4_G128_W4A16 ? 64 : 128;  // of a piece
  static constexpr int kTiles = kRowBytes == 64 ? 2 : 1;         // 16-row tiles a warp multiplies per piece
  static constexpr int kRegs = kPiece / 8;                       // registers of a piece's activations
};

// One of the two matrices: how its rows and columns are cut.
struct Cut {
  int K, rows;       // columns; features (gate/up) or outputs (down)
  int pieces;        // pieces of K
  int columns;       // pieces per slab
  int slabs;         // slabs of a unit
  int groups;        // warps along the rows per piece of K
  int mt;            // 16-row tiles per unit
  int step;          // features or outputs per unit: 8 mt or 16 mt
  int units;         // per expert
  int run;           // consecutive units per ticket
  uint32_t bytes;    // codes of a slab
  const char* scales;
  const float* gs;
};

struct Args {
  CUtensorMap map[2], smap[2];
  FewArgs f;
  ScoreGeom geom;
  Cut cut[2];
  int stages, stage_bytes;
};

struct Tables {  // what routing leaves in shared memory
  int idx[kFewSlots];
  float wt[kFewSlots];
  uint8_t rows[kMaxE][kFewTokens];  // slots of an active expert
  uint8_t expert[kMaxE], count[kMaxE], active_of[kMaxE];
  int leaders[kFewSlots / 32 + 1];
  int nactive, down_passes;         // passes over all active experts
};

__device__ __forceinline__ int passes(int kind, int count) { return kind ? (count + 3) / 4 : (count + 7) / 8; }

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1, bool bf) {
  if (bf)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t c) {  // the two codes in c's low half
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xFFFFu), __NV_E4M3);
  return *(const uint32_t*)&h;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*(const __half2*)&a, *(const __half2*)&b);
  return *(const uint32_t*)&r;
}
// Eight E2M1 codes -> four pairs of fp16.
__device__ __forceinline__ void e2m1x8_f16(uint32_t c, uint32_t (&o)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(c));
}

// Where the q-th eight elements of a lane's share of a piece stand in the piece (t: lane % 4).  The MMA's K order is free as
// long as both operands use the same one, so a lane takes what it can read in wide, conflict-free accesses.
template <int FMT>
__device__ __forceinline__ int element(int t, int q) {
  if (FMT == MOE_FMT_INT4_G128_W4A16) return 8 * (t + 4 * q);
  return Format<FMT>::kPiece / 4 * t + 8 * q;
}

// INT4 words decode into pairs of elements (j, j + 4): the same order for the activations.
template <int FMT>
__device__ __forceinline__ void order_pairs(uint32_t* b) {
  if (FMT != MOE_FMT_INT4_G128_W4A16) return;
  const uint32_t r0 = b[0], r1 = b[1], r2 = b[2], r3 = b[3];
  b[0] = __byte_perm(r0, r2, 0x5410);
  b[1] = __byte_perm(r0, r2, 0x7632);
  b[2] = __byte_perm(r1, r3, 0x5410);
  b[3] = __byte_perm(r1, r3, 0x7632);
}

// A piece of the activations as the MMA's column operand: x of up to eight tokens, ...
template <int FMT>
__device__ __forceinline__ void load_x(const FewArgs& f, const Tables& s, int ai, int pass, int col, int lane, uint32_t (&b)[Format<FMT>::kRegs]) {
  const int g = lane >> 2, t = lane & 3, r = 8 * pass + g;
  const bool live = r < s.count[ai];
  const int token = s.rows[ai][live ? r : 0] / f.k;
  const uint16_t* row = FMT == MOE_FMT_BF16 ? (const uint16_t*)(f.x + token * f.ldx) : (const uint16_t*)(f.xs + (size_t)token * f.d.H);
#pragma unroll
  for (int q = 0; q < Format<FMT>::kRegs / 4; ++q) {
    const uint4 u = live ? *(const uint4*)(row + col + element<FMT>(t, q)) : make_uint4(0, 0, 0, 0);
    b[4 * q] = u.x, b[4 * q + 1] = u.y, b[4 * q + 2] = u.z, b[4 * q + 3] = u.w;
    order_pairs<FMT>(b + 4 * q);
  }
}

// ... or h of up to four: the columns 0 .. 3 hold the nearest fp16 (bf16) of each, 4 .. 7 what is left.
template <int FMT>
__device__ __forceinline__ void load_h(const FewArgs& f, const Tables& s, int ai, int pass, int col, int lane, uint32_t (&b)[Format<FMT>::kRegs]) {
  const int g = lane >> 2, t = lane & 3, r = 4 * pass + (g & 3);
  const bool live = r < s.count[ai], low = g >= 4;
  const int slot = s.rows[ai][live ? r : 0];
  const float* row = f.h + (size_t)slot * f.d.I + col;
  const float scale = FMT == MOE_FMT_BF16 ? 1.f : row_scale(__ldcg(f.hmax + slot));
#pragma unroll
  for (int q = 0; q < Format<FMT>::kRegs / 4; ++q) {
    const float4* p = (const float4*)(row + element<FMT>(t, q));
    const float4 u0 = live ? __ldcg(p) : make_float4(0, 0, 0, 0), u1 = live ? __ldcg(p + 1) : make_float4(0, 0, 0, 0);
    const float v[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (FMT == MOE_FMT_BF16) {
        __nv_bfloat162 hi = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        if (low) hi = __floats2bfloat162_rn(v[2 * j] - __low2float(hi), v[2 * j + 1] - __high2float(hi));
        b[4 * q + j] = *(const uint32_t*)&hi;
      } else {
        const float x = v[2 * j] * scale, y = v[2 * j + 1] * scale;
        __half2 hi = __floats2half2_rn(x, y);
        if (low) hi = __floats2half2_rn(x - __low2float(hi), y - __high2float(hi));
        b[4 * q + j] = *(const uint32_t*)&hi;
      }
    }
    order_pairs<FMT>(b + 4 * q);
  }
}

// c += one piece of a 16-row tile times the activations.  sm: the slab's codes; tile m of mt; piece: in the slab.  Rows: gate/up
// holds the 8 mt gate rows and then the ups, a tile's rows 0 .. 7 its gates and 8 .. 15 the same features' ups.
template <int FMT>
__device__ __forceinline__ void multiply(const Cut& cut, int kind, const char* sm, const char* sc, int e, int n0, int m, int slab, int piece,
                                         int lane, const uint32_t (&b)[Format<FMT>::kRegs], float (&c)[4]) {
  const int g = lane >> 2, t = lane & 3, mt = cut.mt;
  // the tile's rows g and g + 8 within the slab
  const int r0 = kind ? 16 * m + g : 8 * m + g, r1 = kind ? r0 + 8 : 8 * mt + r0;
  const char* at = sm + (size_t)piece * (16 * mt * Format<FMT>::kRowBytes);
  float p[4] = {0.f, 0.f, 0.f, 0.f};
  if constexpr (FMT == MOE_FMT_FP8_B128_W8A16) {
    // rows of 128 bytes, 16-byte parts XORed with the row: a lane's two parts of eight lanes lie in different banks
    const int col = cut.columns * slab + piece, f0 = n0 + (kind ? r0 : 8 * m + g), f1 = kind ? n0 + r1 : cut.rows + f0;
    const int per = (kind ? cut.rows : 2 * cut.rows) / 128;  // blocks of rows
    const float* s = (const float*)cut.scales + (size_t)e * per * cut.pieces + col;
    // (a tile past the matrix's end is not stored: any scale will do)
    const float s0 = __ldg(s + (size_t)min(f0 / 128, per - 1) * cut.pieces), s1 = __ldg(s + (size_t)min(f1 / 128, per - 1) * cut.pieces);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int part = (2 * t + q) ^ g;
      const uint4 u = *(const uint4*)(at + 128 * r0 + 16 * part), v = *(const uint4*)(at + 128 * r1 + 16 * part);
      const uint32_t w0[4] = {u.x, u.y, u.z, u.w}, w1[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        mma(p, e4m3x2_f16(w0[j]), e4m3x2_f16(w1[j]), e4m3x2_f16(w0[j] >> 16), e4m3x2_f16(w1[j] >> 16), b[8 * q + 2 * j], b[8 * q + 2 * j + 1], false);
    }
    c[0] = fmaf(p[0], s0, c[0]), c[1] = fmaf(p[1], s0, c[1]), c[2] = fmaf(p[2], s1, c[2]), c[3] = fmaf(p[3], s1, c[3]);
  } else if constexpr (FMT == MOE_FMT_BF16) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int part = (2 * t + q) ^ g;
      const uint4 u = *(const uint4*)(at + 128 * r0 + 16 * part), v = *(const uint4*)(at + 128 * r1 + 16 * part);
      mma(p, u.x, v.x, u.y, v.y, b[4 * q], b[4 * q + 1], true);
      mma(p, u.z, v.z, u.w, v.w, b[4 * q + 2], b[4 * q + 3], true);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] += p[i];
  } else if constexpr (FMT == MOE_FMT_NVFP4_W4A16) {
    // rows of 64 bytes: eight lanes read 128 consecutive ones.  A code times its block's scale has six significant bits: exact in
    // fp16 (2^-10 at the least, 2688 at most).
    const int col = cut.columns * slab + piece, per = cut.K / 16;
    const uint32_t q0 = e4m3x2_f16(*(const uint16_t*)(sc + r0 * per + 8 * col + 2 * t)), q1 = e4m3x2_f16(*(const uint16_t*)(sc + r1 * per + 8 * col + 2 * t));
    const uint4 u = *(const uint4*)(at + 64 * r0 + 16 * t), v = *(const uint4*)(at + 64 * r1 + 16 * t);
    const uint32_t w0[4] = {u.x, u.y, u.z, u.w}, w1[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t s0 = __byte_perm(q0, q0, j < 2 ? 0x1010 : 0x3232), s1 = __byte_perm(q1, q1, j < 2 ? 0x1010 : 0x3232);
      uint32_t x[4], y[4];
      e2m1x8_f16(w0[j], x);
      e2m1x8_f16(w1[j], y);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        mma(p, hmul2(x[2 * i], s0), hmul2(y[2 * i], s1), hmul2(x[2 * i + 1], s0), hmul2(y[2 * i + 1], s1), b[4 * j + 2 * i], b[4 * j + 2 * i + 1], false);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] += p[i];
  } else {
    // a word holds eight columns of one row, and words of a column group lie side by side along the rows: a group of warps has
    // its 32 rows' words (128 bytes, or 64 of gates and 64 of ups; 16-byte parts of these XORed with the column group) to itself.  Half-words of nibbles become
    // 1024 + code in fp16, less 1032 the weight.
    const __half* s = (const __half*)sc + (size_t)piece * 16 * mt;
    const float s0 = __half2float(s[r0]), s1 = __half2float(s[r1]);
    const char* words = sm + (size_t)(m >> 1) * (cut.columns * 2048) + 2048 * piece;
    const int at0 = 4 * (kind ? 16 * (m & 1) + g : 8 * (m & 1) + g), at1 = at0 + (kind ? 32 : 64);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int kr = t + 4 * q, swap = (kr & (kind ? 7 : 3)) << 4;
      const uint32_t w[2] = {*(const uint32_t*)(words + 128 * kr + (at0 ^ swap)), *(const uint32_t*)(words + 128 * kr + (at1 ^ swap))};
      uint32_t x[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t v = ((w[i] >> (4 * j)) & 0x000F000Fu) | 0x64006400u;
          const __half2 d = __hsub2(*(const __half2*)&v, __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408)));
          x[i][j] = *(const uint32_t*)&d;
        }
      mma(p, x[0][0], x[1][0], x[0][1], x[1][1], b[4 * q], b[4 * q + 1], false);
      mma(p, x[0][2], x[1][2], x[0][3], x[1][3], b[4 * q + 2], b[4 * q + 3], false);
    }
    c[0] = fmaf(p[0], s0, c[0]), c[1] = fmaf(p[1], s0, c[1]), c[2] = fmaf(p[2], s1, c[2]), c[3] = fmaf(p[3], s1, c[3]);
  }
}

// Whole warp: wait until *p >= want (bounded).
__device__ __forceinline__ bool wait_count(const int* p, int want, int lane, volatile int* abort) {
  bool ok = true;
  if (lane == 0) {
    const long long t0 = clock64();
    int v;
    for (int i = 0;; ++i) {
      asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
      if (v >= want) break;
      if ((i & 63) == 63 && (*abort || clock64() - t0 > kWaitLimitCycles)) {
        *abort = 1;
        ok = false;
        break;
      }
    }
  }
  return __shfl_sync(0xffffffffu, ok, 0);
}

// The experts and weights of every token, and the active experts' rows, in shared memory.
__device__ __noinline__ void route_tokens(const Args& a, Tables& s, ScoreScratch* scratch) {
  const FewArgs& f = a.f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, R = f.T * f.k;
  for (int t = warp; t < f.T; t += kWarps) {
    if (a.geom.per <= 1) score_token<1>(f.router, a.geom, t, f.k, lane, s.idx, s.wt, scratch[warp]);
    else if (a.geom.per <= 2) score_token<2>(f.router, a.geom, t, f.k, lane, s.idx, s.wt, scratch[warp]);
    else if (a.geom.per <= 4) score_token<4>(f.router, a.geom, t, f.k, lane, s.idx, s.wt, scratch[warp]);
    else if (a.geom.per <= 8) score_token<8>(f.router, a.geom, t, f.k, lane, s.idx, s.wt, scratch[warp]);
    else score_token<16>(f.router, a.geom, t, f.k, lane, s.idx, s.wt, scratch[warp]);
  }
  __syncthreads();
  // an expert is active as of its first slot, in the order of those
  const int i = threadIdx.x, e = i < R ? s.idx[i] : -1;
  int rank = 0, total = 0;
  if (i < R)
    for (int j = 0; j < R; ++j) {
      const bool same = s.idx[j] == e;
      rank += same && j < i;
      total += same;
    }
  const bool leader = i < R && rank == 0;
  const uint32_t ballot = __ballot_sync(0xffffffffu, leader);
  if (lane == 0 && warp < kFewSlots / 32) s.leaders[warp] = __popc(ballot);
  __syncthreads();
  if (leader) {
    int ai = __popc(ballot & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) ai += s.leaders[w];
    s.expert[ai] = (uint8_t)e;
    s.count[ai] = (uint8_t)total;
    s.active_of[e] = (uint8_t)ai;
  }
  if (i == 0) {
    int n = 0;
    for (int w = 0; w < kFewSlots / 32; ++w) n += s.leaders[w];
    s.nactive = n;
    s.down_passes = 0;
  }
  __syncthreads();
  if (i < R) s.rows[s.active_of[e]][rank] = (uint8_t)i;
  if (leader) atomicAdd(&s.down_passes, passes(1, total));
  if (blockIdx.x == 0 && i < R) {
    if (f.topk_idx) f.topk_idx[i] = e;
    if (f.topk_w) f.topk_w[i] = s.wt[i];
  }
  __syncthreads();
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) few_experts_kernel(const __grid_constant__ Args a) {
  constexpr int kRegs = Format<FMT>::kRegs, kTiles = Format<FMT>::kTiles;
  extern __shared__ __align__(1024) char smem_raw[];
  __shared__ Tables s;
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], ufull[kEndWarps], uempty[kEndWarps];
  __shared__ int s_unit[kMaxStages], s_end[kEndWarps][2], s_abort;
  char* ring = (char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  float4* parts = (float4*)(ring + (size_t)a.stages * a.stage_bytes);  // [unit % 4][tile][piece][lane]
  constexpr int kPartsPerUnit = kTiles * kColumns * 32;
  const FewArgs& f = a.f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kMulWarps);
    }
    for (int i = 0; i < kEndWarps; ++i) {
      mbar_init(&ufull[i], kMulWarps);
      mbar_init(&uempty[i], 1);
    }
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == kProdWarp && lane < 2) prefetch_tmap(&a.map[lane]);
  pdl_wait();  // the router's logits and the scaled rows
  pdl_trigger();
  route_tokens(a, s, (ScoreScratch*)parts);
  const int ngu = s.nactive * a.cut[0].units, nunits = ngu + s.nactive * a.cut[1].units;
  // a unit: its matrix, active expert and place there
  auto place = [&](int unit, int& kind, int& ai, int& tile) {
    kind = unit >= ngu;
    const int j = kind ? unit - ngu : unit, per = a.cut[kind].units;
    ai = j / per;
    tile = j % per;
  };

  if (warp == kProdWarp) {
    // ---------------- weights into the ring (lane 0) ----------------
    if (lane == 0) {
      const int run0 = a.cut[0].run, run1 = a.cut[1].run, t0 = (ngu + run0 - 1) / run0;
      int it = 0, armed[kMaxStages];
      for (int i = 0; i < kMaxStages; ++i) armed[i] = 0;
      bool ok = true;
      int ticket = atomicAdd(f.status + 1, 1);
      while (ok) {
        const int lo = ticket < t0 ? ticket * run0 : ngu + (ticket - t0) * run1;
        const int hi = min(lo + (ticket < t0 ? run0 : run1), ticket < t0 ? ngu : nunits);
        const int next = lo < nunits ? atomicAdd(f.status + 1, 1) : 0;
        for (int unit = lo < nunits ? lo : -1; ok && unit < hi; ++unit) {
          int kind = 0, ai = 0, tile = 0;
          if (unit >= 0) place(unit, kind, ai, tile);
          const Cut& cut = a.cut[kind];
          // a unit of several slabs is streamed again for each pass over its tokens
          const int copies = unit < 0 ? 1 : cut.slabs == 1 ? 1 : cut.slabs * passes(kind, s.count[ai]);
          for (int c = 0; ok && c < copies; ++c, ++it) {
            const int st = it % a.stages;
            ok = mbar_wait(&empty[st], ((it / a.stages) & 1) ^ 1, &s_abort);
            if (!ok) break;
            s_unit[st] = unit;
            if (unit < 0) {
              mbar_arrive(&full[st]);
              continue;
            }
            const int slab = c % cut.slabs, e = s.expert[ai], n0 = tile * cut.step, live = min(cut.step, cut.rows - n0);
            char* dst = ring + (size_t)st * a.stage_bytes;
            uint32_t bytes = cut.bytes, sbytes = 0;
            if (FMT == MOE_FMT_NVFP4_W4A16) bytes += 2 * (sbytes = live * (cut.K / 16) / (kind ? 2 : 1));
            if (FMT == MOE_FMT_INT4_G128_W4A16) bytes += cut.columns * 32 * cut.mt;
            mbar_arrive_expect_tx(&full[st], bytes);
            ++armed[st];
            if (FMT == MOE_FMT_INT4_G128_W4A16) {
              for (int i = 0; i < cut.groups; ++i) {
                char* to = dst + (size_t)i * (cut.columns * 2048);
                if (kind == 0) tma_load_4d(to, &a.map[0], &full[st], n0 + 16 * i, 0, 16 * cut.columns * slab, e);
                else tma_load_3d(to, &a.map[1], &full[st], n0 + 32 * i, 16 * cut.columns * slab, e);
              }
              if (kind == 0) tma_load_4d(dst + cut.bytes, &a.smap[0], &full[st], n0, 0, cut.columns * slab, e);
              else tma_load_3d(dst + cut.bytes, &a.smap[1], &full[st], n0, cut.columns * slab, e);
            } else {
              if (kind == 0) tma_load_5d(dst, &a.map[0], &full[st], 0, n0, 0, cut.columns * slab, e);
              else tma_load_4d(dst, &a.map[1], &full[st], 0, n0, cut.columns * slab, e);
              if (FMT == MOE_FMT_NVFP4_W4A16) {
                const size_t row = (size_t)cut.K / 16;
                char* sc = dst + cut.bytes;
                if (kind == 0) {
                  const char* src = cut.scales + ((size_t)e * 2 * cut.rows + n0) * row;
                  bulk_load(sc, src, sbytes, &full[st]);
                  bulk_load(sc + cut.step * row, src + cut.rows * row, sbytes, &full[st]);
                } else {
                  bulk_load(sc, cut.scales + ((size_t)e * cut.rows + n0) * row, 2 * sbytes, &full[st]);
                }
              }
            }
          }
          if (unit < 0) break;
        }
        if (lo >= nunits) break;
        ticket = next;
      }
      if (s_abort) {  // let every issued copy land before shared memory goes away
        volatile int no_abort = 0;
        for (int i = 0; i < a.stages; ++i)
          if (armed[i]) mbar_wait(&full[i], (armed[i] - 1) & 1, &no_abort);
      }
    }
    __syncwarp();
  } else if (warp < kMulWarps) {
    // ---------------- pieces: decode and multiply ----------------
    uint32_t b[kRegs];
    int key = -1, it = 0, u = 0;
    bool ok = true;
    auto acquire = [&](int n) { return __all_sync(0xffffffffu, mbar_wait(&full[n % a.stages], (n / a.stages) & 1, &s_abort)); };
    auto release = [&](int n) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[n % a.stages]);
    };
    // hand over a pass of a unit: this warp's sums, tile by tile
    auto post = [&](int unit, int pass, const float (&c)[kTiles][4], const Cut* cut, int group, int piece) {
      const int q = u % kEndWarps;
      if (!__all_sync(0xffffffffu, mbar_wait(&uempty[q], ((u / kEndWarps) & 1) ^ 1, &s_abort))) return false;
      if (cut) {
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
          parts[q * kPartsPerUnit + ((group * kTiles + m) * cut->columns + piece) * 32 + lane] = make_float4(c[m][0], c[m][1], c[m][2], c[m][3]);
      }
      if (warp == 0 && lane == 0) {
        s_end[q][0] = unit;
        s_end[q][1] = pass;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ufull[q]);
      ++u;
      return true;
    };
    while (ok) {
      ok = acquire(it);
      if (!ok) break;
      const int unit = *(volatile int*)&s_unit[it % a.stages];
      float c[kTiles][4];
      if (unit < 0) {
        for (int i = 0; i < kEndWarps && ok; ++i) ok = post(-1, 0, c, nullptr, 0, 0);
        break;
      }
      int kind, ai, tile;
      place(unit, kind, ai, tile);
      const Cut& cut = a.cut[kind];
      const int e = s.expert[ai], n0 = tile * cut.step, np = passes(kind, s.count[ai]);
      const int piece = warp % cut.columns, group = warp / cut.columns;
      const bool active = group < cut.groups;
      for (int p = 0; ok && p < np; ++p) {
#pragma unroll
        for (int m = 0; m < kTiles; ++m) c[m][0] = c[m][1] = c[m][2] = c[m][3] = 0.f;
        for (int slab = 0; ok && slab < cut.slabs; ++slab) {
          const int col = slab * cut.columns + piece;
          const bool mine = active && col < cut.pieces;
          const int want = cut.slabs == 1 ? (kind * kMaxE + ai) * kFewTokens + p : -2;
          if (want != key || want == -2) {  // the activations are kept from one unit of an expert to the next
            if (kind) ok = wait_count(f.done + ai, a.cut[0].units * passes(0, s.count[ai]), lane, &s_abort);
            if (mine && ok) {
              if (kind) load_h<FMT>(f, s, ai, p, col * Format<FMT>::kPiece, lane, b);
              else load_x<FMT>(f, s, ai, p, col * Format<FMT>::kPiece, lane, b);
            }
            key = want;
          }
          if (ok && (slab > 0 || (cut.slabs > 1 && p > 0))) ok = acquire(it);
          if (mine && ok) {
            const char* sm = ring + (size_t)(it % a.stages) * a.stage_bytes;
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
              multiply<FMT>(cut, kind, sm, sm + cut.bytes, e, n0, group * kTiles + m, slab, piece, lane, b, c[m]);
          }
          if (ok && (cut.slabs > 1 || p == np - 1)) release(it++);
        }
        if (ok) ok = post(unit, p, c, active ? &cut : nullptr, group, piece);
      }
    }
  } else {
    // ---------------- sums over the pieces, h and y, the combine ----------------
    const int q = warp - kMulWarps, g = lane >> 2, t = lane & 3;
    for (int u = 0;; ++u) {
      if (!__all_sync(0xffffffffu, mbar_wait(&ufull[q], u & 1, &s_abort))) break;
      const int unit = *(volatile int*)&s_end[q][0], p = *(volatile int*)&s_end[q][1];
      if (unit < 0) break;
      int kind, ai, tile;
      place(unit, kind, ai, tile);
      const Cut& cut = a.cut[kind];
      const int e = s.expert[ai], n0 = tile * cut.step, count = s.count[ai];
      const int r = (kind ? 4 : 8) * p + 2 * t;  // the lane's columns are the expert's rows r and r + 1
      const bool live[2] = {r < count && (!kind || t < 2), r + 1 < count && (!kind || t < 2)};
      const int slot[2] = {s.rows[ai][live[0] ? r : 0], s.rows[ai][live[1] ? r + 1 : 0]};
      float factor[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        factor[i] = FMT == MOE_FMT_BF16 ? 1.f : kind ? row_scale_inv(__ldcg(f.hmax + slot[i])) : f.xinv[slot[i] / f.k];
        if (kind) factor[i] *= s.wt[slot[i]];
      }
      const float gs = FMT == MOE_FMT_NVFP4_W4A16 ? __ldg(cut.gs + e) : 1.f;
      uint32_t hm[2] = {0, 0};
      for (int m = 0; m < cut.mt; ++m) {
        const float4* v = parts + q * kPartsPerUnit + m * cut.columns * 32 + lane;
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < cut.columns; ++i) {
          const float4 x = v[32 * i];
          c[0] += x.x, c[1] += x.y, c[2] += x.z, c[3] += x.w;
        }
        if (kind) {  // both terms of h
#pragma unroll
          for (int i = 0; i < 4; ++i) c[i] += __shfl_down_sync(0xffffffffu, c[i], 2);
        }
        if (FMT == MOE_FMT_NVFP4_W4A16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) c[i] = c[i] / gs;
        }
        if (kind == 0) {
          const int n = n0 + 8 * m + g;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float gate = c[i] * factor[i], up = c[2 + i] * factor[i], h = gate / (1.f + expf(-gate)) * up;
            if (live[i] && n < cut.rows) {
              f.h[(size_t)slot[i] * cut.rows + n] = h;
              hm[i] = max(hm[i], __float_as_uint(fabsf(h)));
            }
          }
        } else {
          const int n = n0 + 16 * m + g;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (live[i & 1] && n + 8 * (i >> 1) < cut.rows) f.y[(size_t)slot[i & 1] * cut.rows + n + 8 * (i >> 1)] = c[i] * factor[i & 1];
        }
      }
      if (kind == 0 && FMT != MOE_FMT_BF16) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) hm[i] = max(hm[i], __shfl_xor_sync(0xffffffffu, hm[i], off));
          if (g == 0 && live[i]) atomicMax(f.hmax + slot[i], hm[i]);
        }
      }
      __syncwarp();
      bool last = false;
      if (lane == 0) {
        mbar_arrive(&uempty[q]);
        __threadfence();
        if (kind == 0) atomicAdd(f.done + ai, 1);
        else last = atomicAdd(f.tile + tile, 1) == s.down_passes - 1;
      }
      if (!__shfl_sync(0xffffffffu, last, 0)) continue;
      __threadfence();
      const int quads = min(cut.step, cut.rows - n0) / 4;
      for (int i = lane; i < f.T * quads; i += 32) {
        const int token = i / quads, n = n0 + 4 * (i % quads);
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < f.k; ++j) {
          const float4 v = __ldcg((const float4*)(f.y + (size_t)(token * f.k + j) * cut.rows + n));
          o[0] += v.x, o[1] += v.y, o[2] += v.z, o[3] += v.w;
        }
        __nv_bfloat162 w[2] = {__floats2bfloat162_rn(o[0], o[1]), __floats2bfloat162_rn(o[2], o[3])};
        *(uint2*)(f.out + token * f.ldo + n) = *(const uint2*)w;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && s_abort) set_dev_error(f.status, kDevTimeout);
}

template <int FMT>
bool make_cut(Args& a, int kind) {
  const FewArgs& f = a.f;
  const moe_packed_desc_t& d = f.d;
  Cut& c = a.cut[kind];
  const MatView v = mat_view(d, f.packed, kind);
  c.K = kind ? d.I : d.H;
  c.rows = kind ? d.H : d.I;
  c.scales = (const char*)v.b;
  c.gs = v.gs;
  c.pieces = c.K / Format<FMT>::kPiece;
  c.columns = c.pieces < kColumns ? c.pieces : kColumns;
  c.slabs = (c.pieces + c.columns - 1) / c.columns;
  const int R = f.T * f.k, active = R < d.E ? R : d.E, sms = tc_num_sms();
  // As many rows per unit as keep all the warps busy (128 at most), unless there are then fewer than four units for every SM.
  auto size = [&](int groups) {
    c.groups = groups;
    c.mt = groups * Format<FMT>::kTiles;
    c.step = (kind ? 16 : 8) * c.mt;
    c.units = (c.rows + c.step - 1) / c.step;
  };
  size(kColumns / c.columns < 8 / Format<FMT>::kTiles ? kColumns / c.columns : 8 / Format<FMT>::kTiles);
  while (c.groups > 1 && active * c.units < 4 * sms) size(c.groups / 2);
  c.bytes = (uint32_t)c.mt * c.columns * 16 * Format<FMT>::kRowBytes;
  const int per = active * c.units / (8 * sms);
  c.run = per < 1 ? 1 : per > 8 ? 8 : per;

  const uint64_t E = d.E, N = v.N, K = c.K;
  if (FMT == MOE_FMT_INT4_G128_W4A16) {
    const uint32_t w = c.step, cols = c.columns;
    if (kind == 0) {
      const uint64_t dims[4] = {(uint64_t)c.rows, 2, K / 8, E}, strides[3] = {4 * (uint64_t)c.rows, 4 * N, N * K / 2};
      const uint32_t box[4] = {16, 2, 16 * cols, 1};
      const uint64_t sdims[4] = {(uint64_t)c.rows, 2, K / 128, E}, sstrides[3] = {2 * (uint64_t)c.rows, 2 * N, N * K / 64};
      const uint32_t sbox[4] = {w, 2, cols, 1};
      return tc_make_map_nd(&a.map[0], CU_TENSOR_MAP_DATA_TYPE_UINT32, v.a, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B) &&
             tc_make_map_nd(&a.smap[0], CU_TENSOR_MAP_DATA_TYPE_UINT16, v.b, 4, sdims, sstrides, sbox, CU_TENSOR_MAP_SWIZZLE_NONE);
    }
    const uint64_t dims[3] = {N, K / 8, E}, strides[2] = {4 * N, N * K / 2};
    const uint32_t box[3] = {32, 16 * cols, 1};
    const uint64_t sdims[3] = {N, K / 128, E}, sstrides[2] = {2 * N, N * K / 64};
    const uint32_t sbox[3] = {w, cols, 1};
    return tc_make_map_nd(&a.map[1], CU_TENSOR_MAP_DATA_TYPE_UINT32, v.a, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) &&
           tc_make_map_nd(&a.smap[1], CU_TENSOR_MAP_DATA_TYPE_UINT16, v.b, 3, sdims, sstrides, sbox, CU_TENSOR_MAP_SWIZZLE_NONE);
  }
  const uint32_t rb = Format<FMT>::kRowBytes;
  const uint64_t row = (uint64_t)c.pieces * rb;  // bytes of a matrix row
  const CUtensorMapSwizzle sw = rb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE;
  if (kind == 0) {
    const uint64_t dims[5] = {rb, (uint64_t)c.rows, 2, (uint64_t)c.pieces, E}, strides[4] = {row, row * c.rows, rb, row * N};
    const uint32_t box[5] = {rb, (uint32_t)c.step, 2, (uint32_t)c.columns, 1};
    return tc_make_map_nd(&a.map[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, v.a, 5, dims, strides, box, sw);
  }
  const uint64_t dims[4] = {rb, N, (uint64_t)c.pieces, E}, strides[3] = {row, rb, row * N};
  const uint32_t box[4] = {rb, (uint32_t)c.step, (uint32_t)c.columns, 1};
  return tc_make_map_nd(&a.map[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, v.a, 4, dims, strides, box, sw);
}

template <int FMT>
cudaError_t launch(const FewArgs& f, cudaStream_t s) {
  static SmemOptIn opt_in;
  if (const cudaError_t e = opt_in(few_experts_kernel<FMT>, (int)kSmemMax); e != cudaSuccess) return e;
  Args a;
  a.f = f;
  a.geom = score_geom(f.router, f.d.E);
  a.stage_bytes = 0;
  for (int kind = 0; kind < 2; ++kind) {
    if (!make_cut<FMT>(a, kind)) return cudaErrorInvalidValue;
    const Cut& c = a.cut[kind];
    int bytes = (int)c.bytes;
    if (FMT == MOE_FMT_NVFP4_W4A16) bytes += 16 * c.mt * (c.K / 16);
    if (FMT == MOE_FMT_INT4_G128_W4A16) bytes += c.columns * 32 * c.mt;
    bytes = (bytes + 1023) / 1024 * 1024;
    if (bytes > a.stage_bytes) a.stage_bytes = bytes;
  }
  const size_t parts = (size_t)kEndWarps * Format<FMT>::kTiles * kColumns * 512;
  a.stages = (int)((kSmemMax - 1024 - parts) / a.stage_bytes);
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  if (a.stages < 2) return cudaErrorInvalidValue;
  const int R = f.T * f.k, active = R < f.d.E ? R : f.d.E, sms = tc_num_sms();
  const long units = (long)active * (a.cut[0].units + a.cut[1].units);
  note_launches(1);
  return launch_pdl(few_experts_kernel<FMT>, dim3((unsigned)(units < sms ? units : sms)), dim3(kThreads),
                    1024 + parts + (size_t)a.stages * a.stage_bytes, s, a);
}

}  // namespace

cudaError_t launch_few_experts(const FewArgs& a, cudaStream_t s) {
  switch (a.d.fmt) {
    case MOE_FMT_FP8_B128_W8A16:
    case MOE_FMT_FP8_B128_W8A8:
      return launch<MOE_FMT_FP8_B128_W8A16>(a, s);
    case MOE_FMT_INT4_G128_W4A16:
      return launch<MOE_FMT_INT4_G128_W4A16>(a, s);
    case MOE_FMT_BF16:
      return launch<MOE_FMT_BF16>(a, s);
    default:
      return launch<MOE_FMT_NVFP4_W4A16>(a, s);
  }
}

}  // namespace moe
