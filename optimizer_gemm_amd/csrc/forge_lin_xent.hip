// bfloat16 products of the cross entropy: partial maxima and sums, logit gradients.
#include "forge_lin_kernel.h"
namespace forge {
template hipError_t lin_bf16<L_LSE, false, false>(const LinArgs&, hipStream_t);
template hipError_t lin_bf16<L_DLOGIT, false, false>(const LinArgs&, hipStream_t);
}  // namespace forge
