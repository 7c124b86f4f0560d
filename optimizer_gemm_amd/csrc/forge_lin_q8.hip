// Forward products of 8-bit integers with a factor for each token and each output column, plain and
// grouped by expert: the bfloat16 kernels with v_mfma_i32_16x16x64_i8 in the place of their matrix instruction. A
// fragment's 16 bytes hold 16 k instead of 8, so stages, LDS layout, swizzles and waits are the same with k counted in
// pairs, and a product takes half the stages of a bfloat16 one. The sums are integers until the epilogue, which
// converts them and applies the two factors, so no tile or split changes a result's bits.
// Measured: 8192 x 14336 -> 4096 with residual 333 us, 2890 TOP/s (bfloat16: 667 us, 1434); 777 x 4096 -> 2 x 14336
// gated 104; 1 x 4096 -> 4096 6.3, 10.4 with the quantisation. The choice of tiles is the bfloat16 products':
// within 5% of the best of them for 25 shapes from 1 x 4096 -> 4096 to 8192 x 14336 -> 4096, but for the one below.
#include "forge_lin_kernel.h"

namespace forge {
namespace {

template <int EPI>
hipError_t lin_q8(const LinArgs& g, hipStream_t st) {
  switch (lin_tile<EPI>(g.M, g.N)) {
    case LT_BIG: return lin_large<EPI, false, false, LM_Q8>(g, st);
    case LT_SMALL: return lin_run<LinSmall, EPI, false, false, LM_Q8>(g, st);
    case LT_SPLIT: return lin_run<LinSplit, EPI, false, false, LM_Q8>(g, st);
    default: return lin_run<LinTiny, EPI, false, false, LM_Q8>(g, st);
  }
}

// The gated product of a few tokens over much memory: the kernel for a few tokens gives each wave one batch of loads
// of each matrix there (1 x 4096 -> 2 x 14336, 117 MB: 31 us against 24 with tiles; 4 of 8 experts, 470 MB: 119
// against 96; but 5 of 16 experts, 4096 -> 2 x 1792, 73 MB: 20.6 against 22.2).
bool q8_much_memory(const LinArgs& g, int64_t used) { return used * g.M * g.K[0] * 4 >= 96 * 1000 * 1000; }
bool q8_few_rows(int epi, const LinArgs& g) {
  return few_rows(g) && !(epi == L_GATED && q8_much_memory(g, g.experts < g.N ? g.experts : g.N));
}

}  // namespace

int lin_q8_expert_edge(int epi, int64_t M, int64_t N, int64_t K, int experts) {
  LinArgs g{};
  set_pair(g, 0, nullptr, 0, nullptr, 0, K / 2);
  g.M = (int32_t)M;
  g.N = (int32_t)N;
  g.experts = experts;
  if (q8_few_rows(epi, g)) return 0;
  const double stages = (g.K[0] + 63) / 64;
  switch (epi) {
    case L_LINEAR: return lin_tile_edge(lin_expert_tile<L_LINEAR, false, LM_EXPERT | LM_Q8>(M, N, experts, stages));
    case L_ACC: return lin_tile_edge(lin_expert_tile<L_ACC, false, LM_EXPERT | LM_Q8>(M, N, experts, stages));
    case L_GATED: return lin_tile_edge(lin_expert_tile<L_GATED, false, LM_EXPERT | LM_Q8>(M, N, experts, stages));
    default: return FORGE_ERR_UNSUPPORTED;
  }
}

hipError_t launch_lin_q8(int epi, const LinArgs& g, hipStream_t st) {
  if (g.experts > 0) {
    if (q8_few_rows(epi, g)) return launch_lin_skinny(LM_EXPERT | LM_Q8, epi, g, st);
    return epi == L_GATED ? lin_expert<L_GATED, false, LM_EXPERT | LM_Q8>(g, st)
           : epi == L_ACC ? lin_expert<L_ACC, false, LM_EXPERT | LM_Q8>(g, st)
                          : lin_expert<L_LINEAR, false, LM_EXPERT | LM_Q8>(g, st);
  }
  if (few_tokens(epi, g) && !(epi == L_GATED && q8_much_memory(g, 1))) return launch_lin_skinny(LM_Q8, epi, g, st);
  return epi == L_GATED ? lin_q8<L_GATED>(g, st) : lin_q8<L_LINEAR>(g, st);
}

}  // namespace forge
