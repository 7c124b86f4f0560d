// bfloat16 products of the backward passes: the gated block's, sums of products.
#include "forge_lin_kernel.h"
namespace forge {
template hipError_t lin_bf16<L_DGATE, true, false>(const LinArgs&, hipStream_t);
template hipError_t lin_bf16<L_ACC, true, false>(const LinArgs&, hipStream_t);
template hipError_t lin_bf16<L_ACC, true, true>(const LinArgs&, hipStream_t);
}  // namespace forge
