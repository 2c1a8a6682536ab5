// Entry points of the norms before and after a block: argument checks and the choice of kernel by types
// and alignment.  The kernels are in moe_block_rows.cuh.
#include "moe_block.cuh"

namespace moe {
namespace {

// Rows of eight columns a piece: 16 bytes of a 16-bit type, 32 of fp32, on boundaries of their size.
bool aligned8(const void* p, int64_t ld, size_t size) { return (uintptr_t)p % (8 * size) == 0 && ld % 8 == 0; }

}  // namespace

// moe_block_*.cu: stream and block types
cudaError_t launch_block_bf16(const BlockArgs& a, int param_dtype, bool wide, cudaStream_t s);
cudaError_t launch_block_f16(const BlockArgs& a, int param_dtype, bool wide, cudaStream_t s);
cudaError_t launch_block_f32(const BlockArgs& a, int param_dtype, bool wide, cudaStream_t s);
cudaError_t launch_block_f32_bf16(const BlockArgs& a, int param_dtype, bool wide, cudaStream_t s);
cudaError_t launch_block_f32_f16(const BlockArgs& a, int param_dtype, bool wide, cudaStream_t s);

cudaError_t launch_block(const BlockArgs& a, int x_dtype, int act_dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const size_t sx = dtype_size(x_dtype), sa = dtype_size(act_dtype);
  const bool leave = a.block != nullptr;
  // eight columns an access where every tensor's rows allow it
  bool wide = a.H % 8 == 0 && aligned8(a.x, a.ldx, sx);
  if (leave) wide = wide && aligned8(a.block, a.ldb, sa) && aligned8(a.out, a.ldo, sx);
  if (a.next.kind) wide = wide && aligned8(a.y, a.ldy, sa);
  if (leave && a.gate && a.gate_step) wide = wide && aligned8(a.gate, a.gate_ld, dtype_size(a.gate_dtype));
  for (const moe_norm_t* n : {&a.post, &a.next})
    if (n->kind) wide = wide && aligned8(n->weight, 0, dtype_size(n->dtype)) && aligned8(n->bias, 0, dtype_size(n->dtype));
  // the one type of the parameters and the gate, or 0 where they differ
  int pt = -1;
  auto meet = [&](bool used, int dt) { pt = !used ? pt : pt < 0 || pt == dt ? dt : 0; };
  meet(a.post.kind && (a.post.weight || a.post.bias), a.post.dtype);
  meet(a.next.kind && (a.next.weight || a.next.bias), a.next.dtype);
  meet(leave && a.gate, a.gate_dtype);
  if (pt < 0) pt = act_dtype;
  note_launches(1);
  if (x_dtype == MOE_DT_BF16 && act_dtype == MOE_DT_BF16) return launch_block_bf16(a, pt, wide, s);
  if (x_dtype == MOE_DT_F16 && act_dtype == MOE_DT_F16) return launch_block_f16(a, pt, wide, s);
  if (x_dtype == MOE_DT_F32 && act_dtype == MOE_DT_F32) return launch_block_f32(a, pt, wide, s);
  if (x_dtype == MOE_DT_F32 && act_dtype == MOE_DT_BF16) return launch_block_f32_bf16(a, pt, wide, s);
  if (x_dtype == MOE_DT_F32 && act_dtype == MOE_DT_F16) return launch_block_f32_f16(a, pt, wide, s);
  return cudaErrorInvalidValue;  // refused by the entry points before
}

namespace {

bool norm_ok(const moe_norm_t* n) {
  if (n->kind != MOE_NORM_RMS && n->kind != MOE_NORM_LAYER) return false;
  if (!(n->eps > 0.f)) return false;  // NaN too
  if (!n->weight && !n->bias) return true;
  return dtype_ok(n->dtype) && (uintptr_t)n->weight % dtype_size(n->dtype) == 0 &&
         (uintptr_t)n->bias % dtype_size(n->dtype) == 0;
}

bool matrix_ok(const void* p, int64_t ld, int dt, int H) { return p && ld >= H && (uintptr_t)p % dtype_size(dt) == 0; }

// The stream's type and the block's: the same, or an fp32 stream.
bool types_ok(int x, int act) { return x == act || x == MOE_DT_F32; }

}  // namespace
}  // namespace moe

extern "C" {

using namespace moe;

moe_status_t moe_block_enter(const void* x, int64_t ldx, int x_dtype, const moe_norm_t* norm, void* y, int64_t ldy,
                             int y_dtype, int T, int H, moe_stream_t stream) {
  if (T < 0 || H < 1 || !norm || !norm_ok(norm) || !dtype_ok(x_dtype) || !dtype_ok(y_dtype)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!matrix_ok(x, ldx, x_dtype, H) || !matrix_ok(y, ldy, y_dtype, H))) return MOE_ERR_INVALID_ARG;
  if (!types_ok(x_dtype, y_dtype)) return MOE_ERR_UNSUPPORTED;
  const moe_status_t dv = device_ok();
  if (dv != MOE_OK) return dv;
  BlockArgs a = {};
  a.x = x;
  a.y = y;
  a.ldx = ldx;
  a.ldy = ldy;
  a.next = *norm;
  a.T = T;
  a.H = H;
  return launch_block(a, x_dtype, y_dtype, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t moe_block_leave(const void* x, int64_t ldx, int x_dtype, const void* block, int64_t ldb, int act_dtype,
                             const moe_norm_t* post, const void* gate, int64_t gate_ld, int gate_step, int gate_dtype,
                             int gate_act, float alpha, float beta, const moe_norm_t* next, void* out, int64_t ldo,
                             void* y, int64_t ldy, int T, int H, moe_stream_t stream) {
  if (T < 0 || H < 1 || !dtype_ok(x_dtype) || !dtype_ok(act_dtype)) return MOE_ERR_INVALID_ARG;
  if ((post && !norm_ok(post)) || (next && !norm_ok(next))) return MOE_ERR_INVALID_ARG;
  if (gate) {
    if (!dtype_ok(gate_dtype) || gate_act < MOE_GATE_LINEAR || gate_act > MOE_GATE_TANH) return MOE_ERR_INVALID_ARG;
    if ((gate_step != 0 && gate_step != 1) || gate_ld < 0 || (uintptr_t)gate % dtype_size(gate_dtype) != 0)
      return MOE_ERR_INVALID_ARG;
  }
  if (T > 0 && (!matrix_ok(x, ldx, x_dtype, H) || !matrix_ok(block, ldb, act_dtype, H) ||
                !matrix_ok(out, ldo, x_dtype, H) || (next && !matrix_ok(y, ldy, act_dtype, H))))
    return MOE_ERR_INVALID_ARG;
  if (!types_ok(x_dtype, act_dtype)) return MOE_ERR_UNSUPPORTED;
  const moe_status_t dv = device_ok();
  if (dv != MOE_OK) return dv;
  BlockArgs a = {};
  a.x = x;
  a.block = block;
  a.gate = gate;
  a.out = out;
  a.y = next ? y : nullptr;
  a.ldx = ldx;
  a.ldb = ldb;
  a.ldo = ldo;
  a.ldy = ldy;
  a.gate_ld = gate_ld;
  if (post) a.post = *post;
  if (next) a.next = *next;
  a.gate_step = gate_step;
  a.gate_dtype = gate_dtype;
  a.gate_act = gate_act;
  a.alpha = alpha;
  a.beta = beta;
  a.T = T;
  a.H = H;
  return launch_block(a, x_dtype, act_dtype, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
