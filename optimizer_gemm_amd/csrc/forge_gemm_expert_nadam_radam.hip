// Fused steps of stacked layers (experts), bfloat16.
#include "forge_gemm_kernel.h"
namespace forge {
FORGE_INST_EXPERT(FORGE_NADAM)
FORGE_INST_EXPERT(FORGE_RADAM)
}  // namespace forge
