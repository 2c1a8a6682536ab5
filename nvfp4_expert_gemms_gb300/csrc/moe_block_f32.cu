// Norm and residual kernels for a residual stream in fp32 around a block in fp32.
#include "moe_block_rows.cuh"

namespace moe {
MOE_BLOCK_TYPES(launch_block_f32, float, float, MOE_DT_F32)
}  // namespace moe
