// bfloat16 products grouped by expert, ragged sizes.
#include "forge_lin_kernel.h"
namespace forge {
template hipError_t lin_expert<L_LINEAR, false, LM_EXPERT>(const LinArgs&, hipStream_t);
template hipError_t lin_expert<L_ACC, false, LM_EXPERT>(const LinArgs&, hipStream_t);
template hipError_t lin_expert<L_GATED, false, LM_EXPERT>(const LinArgs&, hipStream_t);
template hipError_t lin_expert<L_DGATE, true, LM_EXPERT>(const LinArgs&, hipStream_t);
template hipError_t lin_expert<L_ACC, true, LM_EXPERT>(const LinArgs&, hipStream_t);
}  // namespace forge
