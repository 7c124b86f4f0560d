// Forward products of a few tokens (serving's single token, a short batch) on bfloat16
// operands: bound by reading the weights once.
//
// A workgroup of 8 waves owns 16 rows of W and all tokens; the waves take an eighth of k each
// (contiguous, so a row's bytes are read in long runs) straight from global memory into the
// operand layout of v_mfma_f32_16x16x32_bf16 - lane l holds row l mod 16, k = 8 (l / 16) .. + 7,
// 16 bytes - with UN loads of each operand in flight per wave. No LDS on the way: nothing is
// read twice by a workgroup but the tokens, which the second-level cache holds. 16 rows a
// workgroup make 256 of them from a 4096-row layer, one per compute unit; the eight partial sums
// are added in order through LDS.
// Measured: 1 x 4096 -> 2 x 14336 gated 47.3 us for 235 MB, 5.0 TB/s, what a copy reaches (the
// tiled kernel: 53); 1 x 4096 -> 4096 10.4 us, of which the kernel takes 8.4 and the rest is the
// call (17). Up to 32 tokens, two fragments of 16.
// What it leaves to the tiles is measured at the choice between them.
#include "forge_lin_kernel.h"

namespace forge {
namespace {

constexpr int K_NW = 8, K_UN = 8;

template <int EPI, int NF>
__global__ __launch_bounds__(64 * K_NW) void lin_skinny_kernel(LinArgs g) {
  constexpr bool TWO = EPI == L_GATED;
  constexpr int NA = TWO ? 2 : 1;
  __shared__ __attribute__((aligned(16))) float part[K_NW][NA][NF][16][16];  // [token][row]
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  const int m0 = blockIdx.x * 16, K = g.K[0];
  // this wave's k: whole steps of 32
  const int steps = (K + 31) / 32, per = (steps + K_NW - 1) / K_NW;
  const int s0 = wave * per, s1 = min(steps, s0 + per);
  const bool row_ok = m0 + l16 < g.M;
  const char* a[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i)
    a[i] = static_cast<const char*>(g.A[i]) + (int64_t)(row_ok ? m0 + l16 : 0) * g.lda[i] * 2 + 16 * q;
  const char* b[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int n = 16 * f + l16;
    b[f] = static_cast<const char*>(g.B[0]) + (int64_t)(n < g.N ? n : 0) * g.ldb[0] * 2 + 16 * q;
  }
  f32x4 acc[NA][NF];
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  // rows and tokens past the edge read row 0 (their sums are dropped); k past the end reads 0
  auto ld = [&](const char* p, int s) -> u32x4 {
    return s < s1 && 32 * s + 8 * q < K ? *reinterpret_cast<const u32x4*>(p + (int64_t)s * 64) : u32x4{0u, 0u, 0u, 0u};
  };
  for (int s = s0; s < s1; s += K_UN) {
    u32x4 x[NA][K_UN], y[NF][K_UN];
#pragma unroll
    for (int u = 0; u < K_UN; ++u) {
#pragma unroll
      for (int i = 0; i < NA; ++i) x[i][u] = ld(a[i], s + u);
#pragma unroll
      for (int f = 0; f < NF; ++f) y[f][u] = ld(b[f], s + u);
    }
#pragma unroll
    for (int u = 0; u < K_UN; ++u)
#pragma unroll
      for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int f = 0; f < NF; ++f)
          acc[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[i][u]),
                                                              __builtin_bit_cast(bf16x8, y[f][u]), acc[i][f], 0, 0, 0);
  }
  // lane holds C[row 4 q + j][token l16]
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int f = 0; f < NF; ++f) *reinterpret_cast<f32x4*>(&part[wave][i][f][l16][4 * q]) = acc[i][f];
  __syncthreads();
  const int t = threadIdx.x, f = t >> 6, n = 16 * f + ((t >> 2) & 15), c = (t & 3) * 4;
  if (f >= NF || n >= g.N || m0 + c >= g.M) return;
  f32x4 sum[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    sum[i] = *reinterpret_cast<const f32x4*>(&part[0][i][f][(t >> 2) & 15][c]);
#pragma unroll
    for (int w = 1; w < K_NW; ++w) sum[i] = sum[i] + *reinterpret_cast<const f32x4*>(&part[w][i][f][(t >> 2) & 15][c]);
  }
  act_dispatch<EPI>(g.e.act, [&](auto act_c) {
    epi_vec<uint16_t, EPI, decltype(act_c)::value>(g.e, n, m0 + c, g.M, sum[0], sum[NA - 1], 1.f);
  });
}

template <int EPI>
hipError_t run(const LinArgs& g, hipStream_t st) {
  const dim3 grid((uint32_t)((g.M + 15) / 16)), block(64 * K_NW);
  if (g.N <= 16)
    hipLaunchKernelGGL((lin_skinny_kernel<EPI, 1>), grid, block, 0, st, g);
  else
    hipLaunchKernelGGL((lin_skinny_kernel<EPI, 2>), grid, block, 0, st, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lin_skinny(int epi, const LinArgs& g, hipStream_t st) {
  return epi == L_GATED ? run<L_GATED>(g, st) : run<L_LINEAR>(g, st);
}

}  // namespace forge
