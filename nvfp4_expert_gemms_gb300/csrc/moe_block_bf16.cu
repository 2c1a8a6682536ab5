// Norm and residual kernels for a residual stream in bf16 around a block in bf16.
#include "moe_block_rows.cuh"

namespace moe {
MOE_BLOCK_TYPES(launch_block_bf16, __nv_bfloat16, __nv_bfloat16, MOE_DT_BF16)
}  // namespace moe
