// Fused steps of stacked layers (experts), bfloat16.
#include "forge_gemm_kernel.h"
namespace forge {
FORGE_INST_EXPERT(FORGE_SGD_MOMENTUM)
FORGE_INST_EXPERT(FORGE_LION)
}  // namespace forge
