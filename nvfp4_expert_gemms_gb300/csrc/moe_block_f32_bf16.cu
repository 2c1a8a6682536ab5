// Norm and residual kernels for a residual stream in fp32 around a block in bf16.
#include "moe_block_rows.cuh"

namespace moe {
MOE_BLOCK_TYPES(launch_block_f32_bf16, float, __nv_bfloat16, MOE_DT_BF16)
}  // namespace moe
