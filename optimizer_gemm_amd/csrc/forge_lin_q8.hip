// Forward products of 8-bit integers with a factor for each token and each output column, plain and
// grouped by expert.
#include "forge_lin_kernel.h"

namespace forge {
namespace {

template <int EPI>
hipError_t lin_q8(const LinArgs& g, hipStream_t st) {
  switch (lin_tile<EPI>(g.M, g.N)) {
    case LT_BIG: return lin_run<LinBig, EPI, false, false, LM_Q8>(g, st);
    case LT_SMALL: return lin_run<LinSmall, EPI, false, false, LM_Q8>(g, st);
    case LT_SPLIT: return lin_run<LinSplit, EPI, false, false, LM_Q8>(g, st);
    default: return lin_run<LinTiny, EPI, false, false, LM_Q8>(g, st);
  }
}

}  // namespace

hipError_t launch_lin_q8(int epi, const LinArgs& g, hipStream_t st) {
  if (g.experts > 0) {
    if (few_rows(g)) return launch_lin_skinny(LM_EXPERT | LM_Q8, epi, g, st);
    return epi == L_GATED ? lin_expert<L_GATED, false, LM_EXPERT | LM_Q8>(g, st)
                          : lin_expert<L_LINEAR, false, LM_EXPERT | LM_Q8>(g, st);
  }
  if (few_tokens(epi, g)) return launch_lin_skinny(LM_Q8, epi, g, st);
  return epi == L_GATED ? lin_q8<L_GATED>(g, st) : lin_q8<L_LINEAR>(g, st);
}

}  // namespace forge
