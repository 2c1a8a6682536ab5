// The experts of moe_layer_few in one kernel: gate/up, down and the combine.
//
// Tokens of one expert go four at a time (an entry: an expert and up to four of its (token, choice) slots).  Work is cut into
// units of an entry's weight rows, whole along K: 16 gates and the same features' ups, or 32 outputs (twice these where K
// is short); first every unit of the gate/up matrices, entry by entry, then those of the down matrices.  Teams of warps
// take runs of units by ticket in that order, so whoever waits (a down unit for its entry's h) waits for units that running
// teams hold and that wait for nothing: no two blocks have to be resident together, and calls on other streams cannot
// stand in the way.  An atomic's answer takes over a microsecond, so a team gets along with one ticket per matrix and asks for
// the next one as it starts a run.
//
// A block holds two teams, each with stages of its own (with stages for both, of which a team skips the other's, a barrier could run
// a lap ahead of who waits on it).  One thread of a team copies by TMA, eight pieces of 128 columns (64 of bf16) by 32 rows to a stage of
// shared memory, 50 to 64 KB ahead (HBM's rate and latency ask for some 45 per block), into the down matrices while h is not there
// yet.  Eight warps take a piece of a stage each, decode it straight into MMA operands, multiply it with the entry's tokens, whose
// operands they keep in shared memory from unit to unit, and leave their sums of 32 rows there too.  A ninth adds them up and
// finishes the rows: h = silu(gate) up, or weighted rows of y.  Who copied sums y over each token's experts at the end,
// in their order.
//
// h and y carry no flags: a value that is not there yet is a NaN that is never written, and who needs it loads until it has
// changed.  With counters behind fences in their place a block's units took up to half as long again (134 us for 90 at 16
// tokens of FP8, 128 experts of 2048 x 768, whichever warp fenced); a fence waits for the SM's traffic.
//
// What it takes (128 experts of 2048 x 768, 8 per token, with the router's kernel): FP8 21.2 us at 1 token and 83 at 16, where HBM alone would
// take 5.6 and 57; NVFP4 42 at 4 tokens (11.5), INT4 80 at 16 (29.6).  Some 7 to 10 us are the router and the entries, 3 to 5 the waits
// for the last h and the last y; the rest is instructions: of a piece's multiplication (130 to 210 per warp) and of what surrounds
// it (some 190, shared by eight warps in part), at six to nine cycles each.  HBM brings a unit of FP8 in 2800 cycles per SM and one of
// four bits in 1500.  Hence teams, each on a unit of its own; one wait per stage, whose description comes with it (a queue of units
// beside the stages, and scales loaded for each: 89 us for 83 at 16 tokens of FP8); as little as possible per stage for the
// copying thread (one warp that copied for both: 91).  And nothing in that chain may wait for L2: no spilled register (with 222 KB of
// shared memory there is next to no L1; the NVFP4 kernel spills 16 bytes), no scale or address that was not asked for early.
#include "moe_few.cuh"
#include "moe_formats.cuh"
#include "moe_tc.cuh"

namespace moe {

using namespace tc;

namespace {

constexpr int kTeams = 2, kTeam = 8, kMulWarps = kTeams * kTeam, kCopyWarp = kMulWarps + kTeams;
constexpr int kWarps = kCopyWarp + kTeams, kThreads = 32 * kWarps;
constexpr int kEntryRows = 4;
constexpr int kStagePieces = kTeam;
constexpr int kParts = 3;   // blocks of 32 rows that a team may be ahead of its ninth warp
constexpr int kMaxStages = 3;
constexpr int kLast = 1 << 16;
constexpr int kTokens = 4;  // per combined piece of 32 columns

template <int FMT>
struct Format {
  static constexpr bool kNvfp4 = FMT == MOE_FMT_NVFP4_W4A16, kInt4 = FMT == MOE_FMT_INT4_G128_W4A16, kBf16 = FMT == MOE_FMT_BF16;
  static constexpr int kPiece = kBf16 ? 64 : 128;                   // columns of a piece
  static constexpr int kRegs = kPiece / 8;                          // registers of a piece's activations
  static constexpr int kRowBytes = kNvfp4 || kInt4 ? 64 : 128;      // of a piece
  static constexpr int kCodes = 32 * kRowBytes;                     // bytes of a piece's codes, 32 rows
  static constexpr int kScales = kNvfp4 ? 256 : kInt4 ? 64 : 0;     // and of the scales that come along
  static constexpr int kStage = kStagePieces * (kCodes + kScales);  // a multiple of 512
  static constexpr int kStages = kNvfp4 || kInt4 ? 3 : 2;           // of each team: whoever waits for a stage has seen all that were in its place
  static constexpr int kOperands = kRegs * 128;                     // bytes of a piece's activations
  static constexpr int kKept = 4096 / kOperands;                    // pieces per unit whose activations a warp keeps
  static constexpr int kSmem = 1024 + kTeams * kStages * ((kStage + 1023) / 1024 * 1024) + kMulWarps * 4096 + kTeams * kParts * kTeam * 512;
};

// One of the two matrices.
struct Cut {
  const char *codes, *scales;
  const float* gs;
  int N, K;          // stored rows and columns per expert
  int rows, pieces;  // features or outputs; pieces of K
  int steps;         // stages along K
  int blocks;        // of 32 weight rows per unit
  int step;          // features or outputs per unit
  int units;         // per entry
  int pairs;         // NVFP4: pieces are copied two by two, 128 bytes of a row, and the scales of eight of them (K % 256 = 0)
};

struct Args {
  CUtensorMap map[2], smap[2];  // codes, and 4-bit formats' scales
  FewArgs f;
  Cut cut[2];
};
__device__ __forceinline__ Cut cut_of(const Args& a, int kind) { return kind ? a.cut[1] : a.cut[0]; }

struct Tables {
  alignas(8) uint8_t slots[kMaxE][kFewSlots / 32];  // an expert's, of each 32
  float wt[kFewSlots];
  uint8_t rows[kFewSlots][kEntryRows];  // an entry's slots
  uint8_t expert[kFewSlots], count[kFewSlots];
  uint16_t first[kMaxE];                // an expert's first entry
  int sums[kWarps];
  float xinv[kFewTokens];
  int entries;
};

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

// Where the j-th eight elements of a lane's share of a piece stand in the piece (t: lane % 4).  The MMA's K order is free as
// long as both operands use the same one, so a lane takes what it can read in whole 16-byte parts without bank conflicts.
template <int FMT>
__device__ __forceinline__ int element(int t, int j) {
  return Format<FMT>::kInt4 ? 8 * t + 32 * j : Format<FMT>::kPiece / 4 * t + 8 * j;
}

// INT4 words decode into pairs of elements (j, j + 4): the same order for the activations.
template <int FMT>
__device__ __forceinline__ void order_pairs(uint32_t* b) {
  if constexpr (Format<FMT>::kInt4) {
    const uint32_t r0 = b[0], r1 = b[1], r2 = b[2], r3 = b[3];
    b[0] = __byte_perm(r0, r2, 0x5410);
    b[1] = __byte_perm(r0, r2, 0x7632);
    b[2] = __byte_perm(r1, r3, 0x5410);
    b[3] = __byte_perm(r1, r3, 0x7632);
  }
}
// The weights code - 8 of two nibbles, one per half-word, at bits 0 .. 3 or (HIGH) 4 .. 7.  Set into the mantissa of 1024 a nibble makes
// 1024 + code, or 1024 + 16 code; both steps from there are exact.
template <bool HIGH>
__device__ __forceinline__ uint32_t int4x2_f16(uint32_t w) {
  const uint32_t v = (w & (HIGH ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u, c = HIGH ? 0xD480D480u : 0xE408E408u, sixteenth = 0x2C002C00u;
  const __half2 h = *(const __half2*)&v, bias = *(const __half2*)&c;  // -72, -1032
  const __half2 r = HIGH ? __hfma2(h, *(const __half2*)&sixteenth, bias) : __hadd2(h, bias);
  return *(const uint32_t*)&r;
}

// A piece of an entry's activations as the MMA's column operand: x in the columns 0 .. 3, ...
template <int FMT>
__device__ __forceinline__ void load_x(const FewArgs& f, const Tables& s, int entry, int col, int lane, uint32_t (&b)[Format<FMT>::kRegs]) {
  const int g = lane >> 2, t = lane & 3;
  const bool live = g < s.count[entry];
  const int token = s.rows[entry][live ? g : 0] / f.k;
  const uint16_t* row = (Format<FMT>::kBf16 ? (const uint16_t*)f.x + token * f.ldx : (const uint16_t*)f.xs + (size_t)token * f.d.H) + col;
#pragma unroll
  for (int j = 0; j < Format<FMT>::kRegs / 4; ++j) {
    const uint4 u = live ? *(const uint4*)(row + element<FMT>(t, j)) : make_uint4(0, 0, 0, 0);
    b[4 * j] = u.x, b[4 * j + 1] = u.y, b[4 * j + 2] = u.z, b[4 * j + 3] = u.w;
    order_pairs<FMT>(b + 4 * j);
  }
}

// Four values that other blocks write, as they are now.
__device__ __forceinline__ uint4 load_now(const float* p) {
  uint4 v;
  asm volatile("ld.relaxed.gpu.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ bool all_set(const uint4& v) { return v.x != kFewUnset && v.y != kFewUnset && v.z != kFewUnset && v.w != kFewUnset; }
__device__ __forceinline__ void store_now(float* p, float v) {
  asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(few_value(v)) : "memory");
}
// mbar_wait in few instructions: a block's roles have to fit the instruction caches together.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  long long since = 0;
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    const long long now = clock64();
    if (since == 0) since = now;
    if (now - since > kWaitLimitCycles) *abort = 1;
    if (*abort) return false;
  }
  return true;
}
// A wait's clock: true once it has run out, or another thread of the block has given up.
struct Patience {
  long long since = 0;
  __device__ __forceinline__ bool over(volatile int* abort) {
    const long long now = clock64();
    if (since == 0) since = now;
    if (now - since > kWaitLimitCycles) *abort = 1;
    __nanosleep(100);
    return *abort;
  }
};

// ... or h, once it is there: the nearest fp16 (bf16) of each in the columns 0 .. 3, what is left in 4 .. 7, after scaling by a power of
// two per row of the piece; inv: its inverse for the rows of the lane's MMA columns 2 t and 2 t + 1.  False if it never came.
template <int FMT>
__device__ __forceinline__ bool load_h(const FewArgs& f, const Tables& s, int entry, int col, int lane, uint32_t (&b)[Format<FMT>::kRegs],
                                       float (&inv)[2], volatile int* abort) {
  const int g = lane >> 2, t = lane & 3, r = g & 3;
  const bool live = r < s.count[entry], low = g >= 4;
  const float* row = f.h + (size_t)s.rows[entry][live ? r : 0] * f.d.I + col;
  uint4 v[Format<FMT>::kRegs / 2];
  for (Patience p;;) {
    bool set = true;
#pragma unroll
    for (int j = 0; j < Format<FMT>::kRegs / 4; ++j) {
      v[2 * j] = load_now(row + element<FMT>(t, j));
      v[2 * j + 1] = load_now(row + element<FMT>(t, j) + 4);
    }
#pragma unroll
    for (int j = 0; j < Format<FMT>::kRegs / 2; ++j) set = set && all_set(v[j]);
    if (__all_sync(0xffffffffu, set)) break;
    if (__any_sync(0xffffffffu, p.over(abort))) return false;
  }
  float scale = 1.f;
  if (!Format<FMT>::kBf16) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < Format<FMT>::kRegs / 2; ++j)
      m = max(m, max(max(v[j].x & 0x7FFFFFFFu, v[j].y & 0x7FFFFFFFu), max(v[j].z & 0x7FFFFFFFu, v[j].w & 0x7FFFFFFFu)));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    scale = row_scale(m);
    const float back = row_scale_inv(m);
#pragma unroll
    for (int i = 0; i < 2; ++i) inv[i] = __shfl_sync(0xffffffffu, back, 4 * ((2 * t + i) & 3));
  }
#pragma unroll
  for (int j = 0; j < Format<FMT>::kRegs / 4; ++j) {
    const uint32_t w[8] = {v[2 * j].x, v[2 * j].y, v[2 * j].z, v[2 * j].w, v[2 * j + 1].x, v[2 * j + 1].y, v[2 * j + 1].z, v[2 * j + 1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = live ? __uint_as_float(w[2 * i]) * scale : 0.f, y = live ? __uint_as_float(w[2 * i + 1]) * scale : 0.f;
      // (an infinity is the largest number and, left over, an infinity: infinity less infinity would be NaN.  So are the fp32 numbers that
      // bf16 rounds to infinity the largest and a rest.)
      constexpr float kMost = Format<FMT>::kBf16 ? 3.38953139e38f : 65504.f;
      const float xm = fminf(fmaxf(x, -kMost), kMost), ym = fminf(fmaxf(y, -kMost), kMost);
      if (Format<FMT>::kBf16) {
        __nv_bfloat162 hi = __floats2bfloat162_rn(xm, ym);
        if (low) hi = __floats2bfloat162_rn(x - __low2float(hi), y - __high2float(hi));
        b[4 * j + i] = *(const uint32_t*)&hi;
      } else {
        __half2 hi = __floats2half2_rn(xm, ym);
        if (low) hi = __floats2half2_rn(x - __low2float(hi), y - __high2float(hi));
        b[4 * j + i] = *(const uint32_t*)&hi;
      }
    }
    order_pairs<FMT>(b + 4 * j);
  }
  return true;
}

// INT4: which four of a unit's 32 stored rows are a lane's.
__device__ __forceinline__ int four_rows(int lane) { return lane >> 3 | (lane >> 2 & 1) << 2; }

// acc += a piece of 32 rows at `sm` (its scales at `sc`) times the activations.  Tile m's MMA rows g and g + 8 are gate and up
// n0 + 8 m + g of the features, or outputs n0 + 16 m + g and 8 further on; INT4: stored rows 2 m and 2 m + 1 of the lane's four.  inv: what the two columns' activations were scaled by.
template <int FMT>
__device__ __forceinline__ void multiply(const char* sm, const char* sc, int pair, int kind, float s0, float s1, const float (&inv)[2], int lane,
                                         const uint4* kept, float (&acc)[2][4]) {
  const int g = lane >> 2, t = lane & 3;
  uint32_t b[Format<FMT>::kRegs];
#pragma unroll
  for (int i = 0; i < Format<FMT>::kRegs / 4; ++i) {
    const uint4 u = kept[32 * i];
    b[4 * i] = u.x, b[4 * i + 1] = u.y, b[4 * i + 2] = u.z, b[4 * i + 3] = u.w;
  }
  if constexpr (Format<FMT>::kInt4) {
    // Words hold eight columns of a row and lie side by side along the rows, 128 bytes per column group: 16-byte parts XORed with
    // the group (gate/up: each half's four parts by the group mod 4).  A lane reads parts, four rows, which are its rows of both
    // tiles; even g take the first half's and odd ones the second's, gates and ups or outputs 16 apart, and eight lanes that
    // read together find different banks.  (With a word of each row at a time, two lanes of four turned about for the
    // banks' sake, 16 tokens took 88 us.)
    const int q = four_rows(lane);
    const uint2 sv = *(const uint2*)(sc + 8 * q);
    const float2 s01 = __half22float2(*(const __half2*)&sv.x), s23 = __half22float2(*(const __half2*)&sv.y);
    const char* part[2] = {sm + 128 * t + ((q ^ t) << 4), sm + 128 * t + ((q ^ t ^ (kind ? 4 : 0)) << 4)};
    float p[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 u = *(const uint4*)(part[j & 1] + 512 * j);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      // (Codes multiplied as they are, as subnormals, and 8 times the activations' sum subtracted afterwards take 69 us for 80 at 16
      // tokens, but leave errors that go by 8 |x| and not by |code - 8| |x|: a weight of zero did not take its activation out.)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint32_t v0 = w[2 * m] >> (8 * n), v1 = w[2 * m + 1] >> (8 * n);
          mma(p[m], int4x2_f16<false>(v0), int4x2_f16<false>(v1), int4x2_f16<true>(v0), int4x2_f16<true>(v1), b[4 * j + 2 * n], b[4 * j + 2 * n + 1], false);
        }
    }
    const float scale[4] = {s01.x, s01.y, s23.x, s23.y};
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = fmaf(p[m][i] * scale[2 * m + i / 2], inv[i & 1], acc[m][i]);
  } else {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float p[4] = {0.f, 0.f, 0.f, 0.f};
      auto step = [&](uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, int i) { mma(p, a0, a1, a2, a3, b[i], b[i + 1], Format<FMT>::kBf16); };
      const int r0 = kind ? 16 * m + g : 8 * m + g, r1 = kind ? r0 + 8 : r0 + 16;
      if constexpr (Format<FMT>::kNvfp4) {
        // a code times its block's scale has six significant bits: exact in fp16 (2^-10 at the least, 2688 at most)
        // pair < 0: rows of 64 bytes and of 8 scales; else the pair-th half of rows of 128 bytes, 16-byte parts XORed with the row, and
        // rows of 64 scales
        const int srow = pair < 0 ? 8 : 64, row = pair < 0 ? 64 : 128, part = (pair < 0 ? t : (4 * pair + t) ^ g) << 4;
        const uint32_t q0 = e4m3x2_f16(*(const uint16_t*)(sc + srow * r0 + 2 * t)), q1 = e4m3x2_f16(*(const uint16_t*)(sc + srow * r1 + 2 * t));
        const uint4 u = *(const uint4*)(sm + row * r0 + part), v = *(const uint4*)(sm + row * r1 + part);
        const uint32_t w0[4] = {u.x, u.y, u.z, u.w}, w1[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t z0 = __byte_perm(q0, q0, j < 2 ? 0x1010 : 0x3232), z1 = __byte_perm(q1, q1, j < 2 ? 0x1010 : 0x3232);
          uint32_t x[4], y[4];
          e2m1x8_f16(w0[j], x);
          e2m1x8_f16(w1[j], y);
#pragma unroll
          for (int i = 0; i < 2; ++i) step(hmul2(x[2 * i], z0), hmul2(y[2 * i], z1), hmul2(x[2 * i + 1], z0), hmul2(y[2 * i + 1], z1), 4 * j + 2 * i);
        }
      } else {
        // rows of 128 bytes, 16-byte parts XORed with the row
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int part = ((2 * t + q) ^ g) << 4;
          const uint4 u = *(const uint4*)(sm + 128 * r0 + part), v = *(const uint4*)(sm + 128 * r1 + part);
          if constexpr (Format<FMT>::kBf16) {
            step(u.x, v.x, u.y, v.y, 4 * q);
            step(u.z, v.z, u.w, v.w, 4 * q + 2);
          } else {
            const uint32_t w0[4] = {u.x, u.y, u.z, u.w}, w1[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              step(e4m3x2_f16(w0[j]), e4m3x2_f16(w1[j]), e4m3x2_f16(w0[j] >> 16), e4m3x2_f16(w1[j] >> 16), 8 * q + 2 * j);
          }
        }
      }
      // (the scales one after the other: their product may be below fp32's range where the sums are not)
      acc[m][0] = fmaf(p[0] * s0, inv[0], acc[m][0]), acc[m][1] = fmaf(p[1] * s0, inv[1], acc[m][1]);
      acc[m][2] = fmaf(p[2] * s1, inv[0], acc[m][2]), acc[m][3] = fmaf(p[3] * s1, inv[1], acc[m][3]);
    }
  }
}

static_assert(kFewSlots == 256, "eight bytes of Tables::slots");

// The entries, from every token's experts, in shared memory (slots: zeros).
__device__ __forceinline__ void make_entries(const FewArgs& f, Tables& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, R = f.T * f.k, i = threadIdx.x;
  const int e = i < R ? f.idx[i] : -1;
  if (i < R) s.wt[i] = f.wt[i];
  if (i < f.T) s.xinv[i] = f.xinv[i];
  // Slot i's rank among its expert's: those before it in its own 32 and in the earlier ones.  The first slot of an expert
  // lays down its entries, in the order of those slots.
  const uint32_t same = __match_any_sync(0xffffffffu, e);
  int rank = __popc(same & ((1u << lane) - 1)), total = 0;
  if (e >= 0 && rank == 0) s.slots[e][warp] = (uint8_t)__popc(same);
  __syncthreads();
  if (e >= 0) {
    const uint2 n = *(const uint2*)s.slots[e];
#pragma unroll
    for (int w = 0; w < kFewSlots / 32; ++w) {
      const int c = (w < 4 ? n.x >> (8 * w) : n.y >> (8 * w - 32)) & 0xFF;
      rank += w < warp ? c : 0;
      total += c;
    }
  }
  const int own = i < R && rank == 0 ? (total + kEntryRows - 1) / kEntryRows : 0;
  int upto = own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += o;
  }
  if (lane == 31) s.sums[warp] = upto;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kFewSlots / 32; ++w) {
    before += w < warp ? s.sums[w] : 0;
    all += s.sums[w];
  }
  if (i == 0) s.entries = all;
  if (own) {
    const int at = before + upto - own;
    s.first[e] = (uint16_t)at;
    for (int j = 0; j < own; ++j) {
      s.expert[at + j] = (uint8_t)e;
      s.count[at + j] = (uint8_t)min(kEntryRows, total - kEntryRows * j);
    }
  }
  __syncthreads();
  if (i < R) s.rows[s.first[e] + rank / kEntryRows][rank % kEntryRows] = (uint8_t)i;
  __syncthreads();
}

// Finishes 32 rows of an entry (one warp): lane 16 m + 2 g + t (t < 2) holds tile m's sums of its rows g and g + 8 for the
// entry's rows 2 t and 2 t + 1.  n0: the first feature or output; factor: what the two rows' sums are multiplied with.
template <int FMT>
__device__ __forceinline__ void finish_rows(const FewArgs& f, int kind, int rows, int n0, int lane, float (&c)[4], const bool (&live)[2],
                                            const int (&slot)[2], const float (&factor)[2]) {
  const int m = lane >> 4, g = lane >> 1 & 7;
  int feature = n0 + 8 * m + g, output = n0 + 16 * m + g, next = 8;
  if (Format<FMT>::kInt4) {
    const int q = four_rows(2 * (lane & 15));
    feature = n0 + 4 * (q & 3) + 2 * m + (g & 1), output = n0 + 4 * q + 2 * m, next = 1;
    if (kind == 0) {  // even g hold two features' gates, odd ones their ups: the first feature to the even ones
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float theirs = __shfl_xor_sync(0xffffffffu, g & 1 ? c[i] : c[2 + i], 2);
        if (g & 1) c[i] = theirs;
        else c[2 + i] = theirs;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (kind == 0) {
      const float gate = c[i] * factor[i], up = c[2 + i] * factor[i];
      if (live[i]) store_now(f.h + (size_t)slot[i] * rows + feature, gate / (1.f + expf(-gate)) * up);
    } else if (live[i]) {
      float* y = f.y + (size_t)slot[i] * rows + output;
      store_now(y, c[i] * factor[i]);
      store_now(y + next, c[2 + i] * factor[i]);
    }
  }
}

// out for 32 columns of four tokens, a lane for four columns of one (one warp): the token's rows of y, once they are there,
// in their order.  False if they never came.
__device__ __noinline__ bool combine(const float* y, __nv_bfloat16* out, int64_t ldo, int T, int k, int H, int lane, volatile int* abort) {
  const int token = lane >> 3, n = 4 * (lane & 7);
  const bool live = token < T;
  const float* at = y + (size_t)(live ? token : 0) * k * H + n;
  uint4 v[kMaxTopK];
  for (Patience p;;) {
    bool set = true;
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j)
      if (j < k) v[j] = load_now(at + (size_t)j * H);
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j)
      if (j < k) set = set && all_set(v[j]);
    if (__all_sync(0xffffffffu, set)) break;
    if (__any_sync(0xffffffffu, p.over(abort))) return false;
  }
  float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j)
    if (j < k)
      o[0] += __uint_as_float(v[j].x), o[1] += __uint_as_float(v[j].y), o[2] += __uint_as_float(v[j].z), o[3] += __uint_as_float(v[j].w);
  const __nv_bfloat162 w[2] = {__floats2bfloat162_rn(o[0], o[1]), __floats2bfloat162_rn(o[2], o[3])};
  if (live) *(uint2*)(out + token * ldo + n) = *(const uint2*)w;
  return true;
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) few_experts_kernel(const __grid_constant__ Args a) {
  using F = Format<FMT>;
  constexpr int kStageBytes = (F::kStage + 1023) / 1024 * 1024;
  extern __shared__ __align__(1024) char smem_raw[];
  __shared__ Tables s;
  __shared__ uint64_t full[kTeams][kMaxStages], empty[kTeams][kMaxStages], bfull[kTeams][kParts], bempty[kTeams][kParts];
  __shared__ int4 s_stage[kTeams][kMaxStages], s_block[kTeams][kParts];  // matrix (-1: no more), entry, first feature or output, step (kLast: the last)
  __shared__ int s_abort;
  char* ring = (char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  float4* parts = (float4*)(ring + kTeams * F::kStages * kStageBytes + kMulWarps * 4096);  // [team][block % 3][warp][tile][16]
  const FewArgs& f = a.f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int j = 0; j < kTeams * kMaxStages; ++j) {
      mbar_init(&full[0][j], F::kNvfp4 ? 33 : 1);
      mbar_init(&empty[0][j], kTeam);
    }
    for (int j = 0; j < kTeams * kParts; ++j) {
      mbar_init(&bfull[0][j], kTeam);
      mbar_init(&bempty[0][j], 1);
    }
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp >= kCopyWarp && lane < 2) prefetch_tmap(&a.map[lane]);
  for (int i = threadIdx.x; i < kMaxE; i += kThreads) *(uint2*)s.slots[i] = make_uint2(0, 0);
  __syncthreads();
  pdl_wait();  // the choice of experts and the scaled rows
  pdl_trigger();
  int ticket = 0;  // the team's next one
  if (warp >= kCopyWarp && lane == 0) ticket = atomicAdd(f.status + 1, 1);
  make_entries(f, s);
  const int ngu = s.entries * a.cut[0].units, nunits = ngu + s.entries * a.cut[1].units;

  if (warp >= kCopyWarp) {
    // ---------------- copies ----------------
    // A matrix's units are divided evenly into as many tickets as there are teams: a run stays with an entry, whose operands
    // the warps then keep (with eight times as many tickets 16 tokens of FP8 took 103 us for 94).
    const int team = warp - kCopyWarp, n0 = kTeams * gridDim.x, n1 = n0;
    int slot = 0, phase = 1, armed = 0;  // stage next, parity of its being free
    bool ok = true;
    for (;;) {
      const int t = __shfl_sync(0xffffffffu, ticket, 0);
      if (t >= n0 + n1) break;
      const int kind = t >= n0;
      const int64_t u = kind ? nunits - ngu : ngu, n = kind ? n1 : n0, nth = kind ? t - n0 : t;
      int unit = (int)(nth * u / n);
      const int end = (int)((nth + 1) * u / n);
      if (lane == 0) ticket = atomicAdd(f.status + 1, 1);
      const Cut cut = cut_of(a, kind);
      const int units = cut.units, blocks = cut.blocks, steps = cut.steps, add = cut.step, rows = kind ? 32 : 16;
      const bool lone = F::kNvfp4 && !cut.pairs;  // NVFP4's scales by every lane, eight bytes at a time
      const uint32_t bytes = min(cut.pieces, kStagePieces) * (F::kCodes + (F::kInt4 ? F::kScales : 0)) + (F::kNvfp4 && !lone ? 32 * 64 : 0);
      const CUtensorMap *map = kind ? &a.map[1] : &a.map[0], *smap = kind ? &a.smap[1] : &a.smap[0];
      int entry = unit / units, tile = unit - entry * units;
      // a stage's TMA copies (one thread)
      auto copy = [&](char* to, uint64_t* bar, int r, int piece, int e) {
        mbar_arrive_expect_tx(bar, bytes);
        char* sc = to + kStagePieces * F::kCodes;
        if constexpr (F::kInt4) {
          if (kind == 0) {
            tma_load_4d(to, map, bar, r, 0, 16 * piece, e);
            tma_load_4d(sc, smap, bar, r, 0, piece, e);
          } else {
            tma_load_3d(to, map, bar, r, 16 * piece, e);
            tma_load_3d(sc, smap, bar, r, piece, e);
          }
        } else {
          const int nth = F::kNvfp4 && !lone ? piece / 2 : piece;
          if (kind == 0) tma_load_5d(to, map, bar, 0, r, 0, nth, e);
          else tma_load_4d(to, map, bar, 0, r, nth, e);
          if (F::kNvfp4 && !lone) {
            if (kind == 0) tma_load_4d(sc, smap, bar, 8 * piece, r, 0, e);
            else tma_load_3d(sc, smap, bar, 8 * piece, r, e);
          }
        }
      };
      for (; ok && unit < end; ++unit) {
        const int e = s.expert[entry], row = tile * add;
        if (lane == 0 || lone)
          for (int block = 0; ok && block < blocks; ++block)
            for (int step = 0; ok && step < steps; ++step) {
              ok = wait(&empty[team][slot], phase, &s_abort);
              if (lone) ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              char* to = ring + (team * F::kStages + slot) * kStageBytes;
              uint64_t* bar = &full[team][slot];
              const int r = row + block * rows, piece = step * kStagePieces;
              if (lone) {
                const int i = kind ? 0 : lane >> 4, n = kind ? r + lane : r + (lane & 15);
                const char* sc = cut.scales + ((size_t)e * cut.N + i * cut.rows + n) * (cut.K / 16) + 8 * piece;
                for (int j = 0; j < kStagePieces && piece + j < cut.pieces; ++j) cp_async_8(smem_u32(to + kStagePieces * F::kCodes + j * F::kScales + 8 * lane), sc + 8 * j);
                cp_async_mbar_arrive_noinc(bar);
              } else if (F::kNvfp4) {  // (the barrier counts every lane's)
                mbar_arrive_many(bar, 32);
              }
              if (lane == 0) {
                s_stage[team][slot] = make_int4(kind, entry, r, step + 1 == steps ? step | kLast : step);
                copy(to, bar, r, piece, e);
              }
              armed |= 1 << slot;
              if (++slot == F::kStages) {
                slot = 0;
                phase ^= 1;
              }
            }
        if (++tile == units) {
          tile = 0;
          ++entry;
        }
      }
      __syncwarp();
      ok = __shfl_sync(0xffffffffu, ok, 0);
      slot = __shfl_sync(0xffffffffu, slot, 0);  // (lane 0's, where it worked alone)
      phase = __shfl_sync(0xffffffffu, phase, 0);
      if (!ok) break;
    }
    if (ok && lane == 0) {
      ok = wait(&empty[team][slot], phase, &s_abort);
      if (ok) {
        s_stage[team][slot] = make_int4(-1, 0, 0, 0);
        mbar_arrive_many(&full[team][slot], F::kNvfp4 ? 33 : 1);
        armed |= 1 << slot;
        if (++slot == F::kStages) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    // the combine, in tickets of its own behind all others
    const int sets = (f.T + kTokens - 1) / kTokens, pieces = f.d.H / 32 * sets;
    for (int t = __shfl_sync(0xffffffffu, ticket, 0) - n0 - n1; ok && t < pieces;) {
      if (lane == 0) ticket = atomicAdd(f.status + 1, 1);
      const int n = 32 * (t / sets), token = kTokens * (t % sets);
      ok = combine(f.y + (size_t)token * f.k * f.d.H + n, f.out + token * f.ldo + n, f.ldo, f.T - token, f.k, f.d.H, lane, &s_abort);
      t = __shfl_sync(0xffffffffu, ticket, 0) - n0 - n1;
    }
    if (F::kNvfp4) cp_async_wait<0>();
    if (lane == 0 && s_abort) {  // let every issued copy land before shared memory goes away
      volatile int no_abort = 0;
      for (int i = 0; i < F::kStages; ++i)
        if (armed >> i & 1) mbar_wait(&full[team][i], (i < slot ? phase : phase ^ 1) ^ 1, &no_abort);
    }
    __syncwarp();
  } else if (warp < kMulWarps) {
    // ---------------- pieces: decode and multiply ----------------
    const int team = warp / kTeam, w = warp % kTeam;
    uint4* kept = (uint4*)(ring + kTeams * F::kStages * kStageBytes + warp * 4096) + lane;  // [piece][4 registers][lane]
    float4* my_parts = parts + (team * kParts * kTeam + w) * 32 + (lane & 2) * 8 + (lane >> 2) * 2 + (lane & 1);
    int slot = 0, phase = 0, part = 0, part_phase = 1;
    int kind = -1, pieces = 0, rows = 0, steps = 0, pairs = 0;  // of the matrix
    const float* scales = nullptr;
    int entry = -1, have = 0;            // the steps of which entry's activations are kept,
    int line = -1, have_scales = 0;      // and of which 128 rows' scales (FP8)
    float inv[F::kKept][2], s0[F::kKept], s1[F::kKept];
#pragma unroll
    for (int i = 0; i < F::kKept; ++i) inv[i][0] = inv[i][1] = 1.f, s0[i] = s1[i] = 1.f;
    float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    bool ok = true;
#pragma unroll 1
    while (__all_sync(0xffffffffu, wait(&full[team][slot], phase, &s_abort))) {
      const int4 d = s_stage[team][slot];
      if (d.x < 0) break;
      if (d.x != kind) {
        kind = d.x;
        const Cut cut = cut_of(a, kind);
        pieces = cut.pieces;
        rows = cut.rows;
        steps = cut.steps;
        pairs = cut.pairs;
        scales = (const float*)cut.scales;
        entry = -1;
      }
      if (d.y != entry) {
        entry = d.y;
        have = have_scales = 0;
      }
      const int step = d.w & (kLast - 1), piece = step * kStagePieces + w;
      if (piece < pieces) {
        const int k = min(step, F::kKept - 1), keep = steps <= F::kKept || step < F::kKept - 1 ? 1 << k : 0;  // (past what is kept: loaded each time)
        uint4* mine = kept + k * (F::kRegs / 4 * 32);
        float f2[2] = {1.f, 1.f}, s2[2] = {1.f, 1.f};
        if (FMT == MOE_FMT_FP8_B128_W8A16) {
          if (d.z / 128 != line) {
            line = d.z / 128;
            have_scales = 0;
          }
          if (!(have_scales >> k & 1)) {
            const int e = s.expert[entry];
            s2[0] = __ldg(scales + (size_t)((kind ? e * rows : 2 * e * rows) / 128 + line) * pieces + piece);
            s2[1] = kind ? s2[0] : __ldg(scales + (size_t)((2 * e + 1) * rows / 128 + line) * pieces + piece);
#pragma unroll
            for (int i = 0; i < F::kKept; ++i)
              if (k == i) s0[i] = s2[0], s1[i] = s2[1];
            have_scales |= keep;
          }
        }
        if (!(have >> k & 1)) {
          uint32_t b[F::kRegs];
          if (kind == 0) load_x<FMT>(f, s, entry, piece * F::kPiece, lane, b);
          else ok = load_h<FMT>(f, s, entry, piece * F::kPiece, lane, b, f2, &s_abort);
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < F::kRegs / 4; ++i) mine[32 * i] = make_uint4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
#pragma unroll
          for (int i = 0; i < F::kKept; ++i)
            if (k == i) inv[i][0] = f2[0], inv[i][1] = f2[1];
          have |= keep;
        }
#pragma unroll
        for (int i = 0; i < F::kKept; ++i)
          if (k == i) f2[0] = inv[i][0], f2[1] = inv[i][1], s2[0] = s0[i], s2[1] = s1[i];
        const int pair = F::kNvfp4 && pairs ? w & 1 : -1;
        const char* stage = ring + (team * F::kStages + slot) * kStageBytes;
        const char* sm = stage + (pair < 0 ? w : w & ~1) * F::kCodes;
        const char* sc = stage + kStagePieces * F::kCodes + w * (pair < 0 ? F::kScales : 8);
        multiply<FMT>(sm, sc, pair, kind, s2[0], s2[1], f2, lane, mine, acc);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[team][slot]);
      if (++slot == F::kStages) {
        slot = 0;
        phase ^= 1;
      }
      if (!(d.w & kLast)) continue;
      // hand the block over to the ninth warp: lanes t < 2 tile 0, the others tile 1, both terms of h added up
      float4 sum;
      float* c = &sum.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float own = lane & 2 ? acc[1][i] : acc[0][i], other = __shfl_xor_sync(0xffffffffu, lane & 2 ? acc[0][i] : acc[1][i], 2);
        c[i] = kind ? own + other : lane & 2 ? other : own;
        acc[0][i] = acc[1][i] = 0.f;
      }
      ok = __all_sync(0xffffffffu, wait(&bempty[team][part], part_phase, &s_abort));
      if (!ok) break;
      my_parts[part * (kTeam * 32)] = sum;
      if (w == 0 && lane == 0) s_block[team][part] = d;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bfull[team][part]);
      if (++part == kParts) {
        part = 0;
        part_phase ^= 1;
      }
    }
    if (__all_sync(0xffffffffu, wait(&bempty[team][part], part_phase, &s_abort))) {  // no more
      if (w == 0 && lane == 0) s_block[team][part] = make_int4(-1, 0, 0, 0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bfull[team][part]);
    }
  } else {
    // ---------------- sums over the pieces, h and y ----------------
    const int team = warp - kMulWarps, t = lane & 1;
    int last_kind = 0, last_entry = -1, part = 0, phase = 0;
    bool live[2] = {false, false};
    int slot[2] = {0, 0};
    float factor[2] = {0.f, 0.f}, gs = 1.f;
    for (;;) {
      if (!__all_sync(0xffffffffu, wait(&bfull[team][part], phase, &s_abort))) break;
      const int4 u = s_block[team][part];
      const int kind = u.x, entry = u.y;
      if (kind < 0) break;
      const int columns = min(kTeam, kind ? a.cut[1].pieces : a.cut[0].pieces);
      if (kind != last_kind || entry != last_entry) {
        last_kind = kind;
        last_entry = entry;
        const int count = s.count[entry];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          live[i] = 2 * t + i < count;
          slot[i] = s.rows[entry][live[i] ? 2 * t + i : 0];
          factor[i] = kind ? s.wt[slot[i]] : F::kBf16 ? 1.f : s.xinv[slot[i] / f.k];
        }
        if (F::kNvfp4) gs = __ldg((kind ? a.cut[1].gs : a.cut[0].gs) + s.expert[entry]);
      }
      const float4* v = parts + (team * kParts + part) * (kTeam * 32) + lane;
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kTeam; ++i)
        if (i < columns) {
          const float4 x = v[32 * i];
          c[0] += x.x, c[1] += x.y, c[2] += x.z, c[3] += x.w;
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bempty[team][part]);  // the team may overwrite
      if (++part == kParts) {
        part = 0;
        phase ^= 1;
      }
      if (F::kNvfp4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = c[i] / gs;
      }
      finish_rows<FMT>(f, kind, kind ? a.cut[1].rows : a.cut[0].rows, u.z, lane, c, live, slot, factor);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && s_abort) set_dev_error(f.status, kDevTimeout);
}

template <int FMT>
bool make_cut(Args& a, int kind) {
  using F = Format<FMT>;
  const moe_packed_desc_t& d = a.f.d;
  Cut& c = a.cut[kind];
  const MatView v = mat_view(d, a.f.packed, kind);
  c.codes = (const char*)v.a;
  c.scales = (const char*)v.b;
  c.gs = v.gs;
  c.N = v.N;
  c.K = v.K;
  c.rows = kind ? d.H : d.I;
  c.pieces = c.K / F::kPiece;
  c.steps = (c.pieces + kStagePieces - 1) / kStagePieces;
  c.pairs = F::kNvfp4 && c.K % 256 == 0;
  // two blocks of rows per unit where K is a single stage, unless there are then fewer than four units for every SM
  const int R = a.f.T * a.f.k, active = R < d.E ? R : d.E;
  auto size = [&](int blocks) {
    c.blocks = blocks;
    c.step = blocks * (kind ? 32 : 16);
    c.units = c.rows / c.step;
  };
  size(c.steps == 1 ? 2 : 1);
  if ((long)active * c.units < 4l * tc_num_sms()) size(1);

  const uint64_t E = d.E, N = v.N, K = c.K, rows = c.rows;
  const uint32_t cols = c.pieces < kStagePieces ? c.pieces : kStagePieces;
  const auto U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, U16 = CU_TENSOR_MAP_DATA_TYPE_UINT16, U32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
  if (F::kInt4) {
    if (kind == 0) {
      const uint64_t dims[4] = {rows, 2, K / 8, E}, strides[3] = {4 * rows, 4 * N, N * K / 2};
      const uint64_t sdims[4] = {rows, 2, K / 128, E}, sstrides[3] = {2 * rows, 2 * N, N * K / 64};
      const uint32_t box[4] = {16, 2, 16 * cols, 1}, sbox[4] = {16, 2, cols, 1};
      return tc_make_map_nd(&a.map[0], U32, v.a, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B) &&
             tc_make_map_nd(&a.smap[0], U16, v.b, 4, sdims, sstrides, sbox, CU_TENSOR_MAP_SWIZZLE_NONE);
    }
    const uint64_t dims[3] = {N, K / 8, E}, strides[2] = {4 * N, N * K / 2};
    const uint64_t sdims[3] = {N, K / 128, E}, sstrides[2] = {2 * N, N * K / 64};
    const uint32_t box[3] = {32, 16 * cols, 1}, sbox[3] = {32, cols, 1};
    return tc_make_map_nd(&a.map[1], U32, v.a, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) &&
           tc_make_map_nd(&a.smap[1], U16, v.b, 3, sdims, sstrides, sbox, CU_TENSOR_MAP_SWIZZLE_NONE);
  }
  const uint64_t row = (uint64_t)c.pieces * F::kRowBytes;  // bytes of a matrix row
  const uint64_t rb = c.pairs ? 128 : F::kRowBytes, parts = row / rb;  // bytes of it that a piece, or two, take
  const uint32_t box_parts = c.pairs ? cols / 2 : cols;
  if (c.pairs) {
    const uint64_t sdims[4] = {K / 16, rows, kind ? E : 2, E}, sstrides[3] = {K / 16, kind ? N * (K / 16) : rows * (K / 16), N * (K / 16)};
    const uint32_t sbox[4] = {64, kind ? 32u : 16u, kind ? 1u : 2u, 1};
    if (!tc_make_map_nd(&a.smap[kind], U8, v.b, kind ? 3 : 4, sdims, sstrides, sbox, CU_TENSOR_MAP_SWIZZLE_NONE)) return false;
  }
  const CUtensorMapSwizzle sw = rb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE;
  if (kind == 0) {
    const uint64_t dims[5] = {rb, rows, 2, parts, E}, strides[4] = {row, row * rows, rb, row * N};
    const uint32_t box[5] = {(uint32_t)rb, 16, 2, box_parts, 1};
    return tc_make_map_nd(&a.map[0], U8, v.a, 5, dims, strides, box, sw);
  }
  const uint64_t dims[4] = {rb, N, parts, E}, strides[3] = {row, rb, row * N};
  const uint32_t box[4] = {(uint32_t)rb, 32, box_parts, 1};
  return tc_make_map_nd(&a.map[1], U8, v.a, 4, dims, strides, box, sw);
}

template <int FMT>
cudaError_t launch(const FewArgs& f, bool lose_h, cudaStream_t s) {
  static SmemOptIn opt_in;
  if (const cudaError_t e = opt_in(few_experts_kernel<FMT>, Format<FMT>::kSmem); e != cudaSuccess) return e;
  Args a;
  a.f = f;
  if (!make_cut<FMT>(a, 0) || !make_cut<FMT>(a, 1)) return cudaErrorInvalidValue;
  const long R = (long)f.T * f.k, active = R < f.d.E ? R : f.d.E, sms = tc_num_sms();
  const long most = active * (a.cut[0].units > a.cut[1].units ? a.cut[0].units : a.cut[1].units);  // (a team may go without)
  const unsigned blocks = (unsigned)(most < sms ? most : sms);
  if (lose_h) {  // the gate/up tickets as given out already
    const int tickets = kTeams * (int)blocks;
    if (const cudaError_t e = cudaMemcpyAsync(f.status + 1, &tickets, sizeof(tickets), cudaMemcpyHostToDevice, s); e != cudaSuccess) return e;
  }
  note_launches(1);
  return launch_pdl(few_experts_kernel<FMT>, dim3(blocks), dim3(kThreads), Format<FMT>::kSmem, s, a);
}

}  // namespace

cudaError_t launch_few_experts(const FewArgs& a, bool lose_h, cudaStream_t s) {
  switch (a.d.fmt) {
    case MOE_FMT_FP8_B128_W8A16:
    case MOE_FMT_FP8_B128_W8A8:
      return launch<MOE_FMT_FP8_B128_W8A16>(a, lose_h, s);
    case MOE_FMT_INT4_G128_W4A16:
      return launch<MOE_FMT_INT4_G128_W4A16>(a, lose_h, s);
    case MOE_FMT_BF16:
      return launch<MOE_FMT_BF16>(a, lose_h, s);
    default:
      return launch<MOE_FMT_NVFP4_W4A16>(a, lose_h, s);
  }
}

}  // namespace moe
