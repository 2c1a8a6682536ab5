// Norm and residual kernels for a residual stream in fp32 around a block in fp16.
#include "moe_block_rows.cuh"

namespace moe {
MOE_BLOCK_TYPES(launch_block_f32_f16, float, __half, MOE_DT_F16)
}  // namespace moe
