// The adapter kernels' search for a block's tile (csrc/moe_adapter_find.cuh) run on the CPU: one fibre per
// thread of a block, which switch where the warp's or the block's threads meet.  Shared memory is static, so
// that a block finds in it what the block before has left, as on the device.
#include <ucontext.h>

#include <algorithm>
#include <cstdint>
#include <vector>

#define __device__
#define __forceinline__ inline
#define __shared__ static

namespace host {

constexpr int kWarps = 2, kThreads = 32 * kWarps, kStack = 64 * 1024;

struct Meeting {  // of `size` threads: the last one to come opens it
  int size, here = 0;
  unsigned opened = 0;
};

ucontext_t g_main, g_fibre[kThreads];
char g_stack[kThreads][kStack];
int g_now;
Meeting g_warp[kWarps], g_block;
Meeting* g_waits[kThreads];
unsigned g_seen[kThreads];
bool g_done[kThreads];
long long g_said[kThreads];  // what each lane of a warp brings to an exchange

void meet(Meeting& m) {
  if (++m.here == m.size) {
    m.here = 0;
    ++m.opened;
    return;
  }
  g_waits[g_now] = &m;
  g_seen[g_now] = m.opened;
  swapcontext(&g_fibre[g_now], &g_main);
}

template <class F>
auto exchange(long long mine, F f) {  // f reads the warp's values
  g_said[g_now] = mine;
  meet(g_warp[g_now / 32]);
  const auto r = f(g_said + g_now / 32 * 32, g_now % 32);
  meet(g_warp[g_now / 32]);
  return r;
}

struct Index {
  operator int() const { return g_now; }
};
struct {
  Index x;
} threadIdx;

void (*g_body)();
void enter() {
  g_body();
  g_done[g_now] = true;
  swapcontext(&g_fibre[g_now], &g_main);
}

// One block; false: threads wait for one another without end.
bool run(void (*body)()) {
  g_body = body;
  for (Meeting& m : g_warp) m = Meeting{32};
  g_block = Meeting{kThreads};
  for (int i = 0; i < kThreads; ++i) {
    g_done[i] = false;
    g_waits[i] = nullptr;
    getcontext(&g_fibre[i]);
    g_fibre[i].uc_stack.ss_sp = g_stack[i];
    g_fibre[i].uc_stack.ss_size = kStack;
    g_fibre[i].uc_link = &g_main;
    makecontext(&g_fibre[i], enter, 0);
  }
  for (;;) {
    bool any = false, moved = false;
    for (g_now = 0; g_now < kThreads; ++g_now) {
      if (g_done[g_now]) continue;
      any = true;
      if (g_waits[g_now] && g_waits[g_now]->opened == g_seen[g_now]) continue;
      g_waits[g_now] = nullptr;
      moved = true;
      swapcontext(&g_main, &g_fibre[g_now]);
    }
    if (!any) return true;
    if (!moved) return false;
  }
}

}  // namespace host

using host::threadIdx;
using std::max;
using std::min;

inline void __syncthreads() { host::meet(host::g_block); }
inline void __syncwarp() { host::meet(host::g_warp[host::g_now / 32]); }
inline int __ffs(uint32_t v) { return __builtin_ffs((int)v); }
inline int __popc(uint32_t v) { return __builtin_popcount(v); }
inline int __shfl_sync(uint32_t, int v, int from) {
  return host::exchange(v, [=](const long long* said, int) { return (int)said[from]; });
}
inline int __shfl_up_sync(uint32_t, int v, int by) {
  return host::exchange(v, [=](const long long* said, int lane) { return (int)said[lane < by ? lane : lane - by]; });
}
inline uint32_t __match_any_sync(uint32_t, int v) {
  return host::exchange(v, [](const long long* said, int lane) {
    uint32_t m = 0;
    for (int i = 0; i < 32; ++i) m |= said[i] == said[lane] ? 1u << i : 0u;
    return m;
  });
}
inline uint32_t __ballot_sync(uint32_t, int v) {
  return host::exchange(v != 0, [](const long long* said, int) {
    uint32_t m = 0;
    for (int i = 0; i < 32; ++i) m |= said[i] ? 1u << i : 0u;
    return m;
  });
}
inline int __all_sync(uint32_t m, int v) { return __ballot_sync(m, v) == 0xffffffffu; }

namespace moe {
struct AdapterArgs {  // the fields of the kernels' own that the search reads
  const float* scale;
  const int32_t *rank, *starts, *slot;
  int T, R, n, r;
};
}  // namespace moe
#include "../nvfp4_expert_gemms_gb300/csrc/moe_adapter_find.cuh"

namespace {
moe::AdapterArgs g_args;
int g_want, g_bm;
moe::Tile g_tile[host::kThreads];
int g_from[16];
}  // namespace

// Every block's tile: found[block] = {slot, t0, rows, rank}, its scale, and (bm = 0, gathered) its tokens in
// from[block][16], -7 where none was written.  Returns the number of blocks (of `most`), or less than 0 where threads do not meet or
// disagree.
extern "C" int tiles(int T, int R, int n, int r, const int32_t* starts, const int32_t* slot, const int32_t* rank, const float* scale,
                     int bm, int most, int32_t (*found)[4], float* scales, int32_t (*from)[16]) {
  g_args = {scale, rank, starts, slot, T, R, n, r};
  g_bm = bm;
  const int64_t blocks = bm ? moe::tile_bound(g_args, bm) : moe::gather_bound(g_args);
  if (blocks > most) return -1;
  for (g_want = 0; g_want < blocks; ++g_want) {
    std::fill(g_from, g_from + 16, -7);
    const bool met = host::run([] {
      g_tile[host::g_now] = g_bm ? moe::find_tile<host::kWarps>(g_args, g_want, g_bm)
                                 : moe::gather_tile<host::kWarps>(g_args, g_want, g_from);
    });
    if (!met) return -2;
    const moe::Tile t = g_tile[0];
    for (const moe::Tile& o : g_tile)
      if (o.slot != t.slot || o.t0 != t.t0 || o.rows != t.rows || o.rk != t.rk || o.scale != t.scale) return -3;
    const int32_t all[4] = {t.slot, t.t0, t.rows, t.rk};
    std::copy(all, all + 4, found[g_want]);
    scales[g_want] = t.scale;
    if (!bm) std::copy(g_from, g_from + 16, from[g_want]);
  }
  return (int)blocks;
}
