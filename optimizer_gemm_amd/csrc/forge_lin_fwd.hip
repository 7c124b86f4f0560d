// bfloat16 products with the forward epilogues (linear, gated).
#include "forge_lin_kernel.h"
namespace forge {
template hipError_t lin_bf16<L_LINEAR, false, false>(const LinArgs&, hipStream_t);
template hipError_t lin_bf16<L_GATED, false, false>(const LinArgs&, hipStream_t);
}  // namespace forge
