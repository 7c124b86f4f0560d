// Products with an epilogue on float32 operands, either index of either operand fast, one kernel for
// every operator of forge_ops.h; and the choice between the bfloat16 kernels.
//
// A workgroup of 4 waves stages BK k of both operands in LDS as rows of k (operands whose k is
// slow are transposed on the way in), and multiplies them with v_mfma_f32_32x32x2_f32. The next stage's global loads are in flight
// (in registers) during the current stage's products. The finished tile goes through LDS as
// float rows of the output, so that the epilogue reads and writes whole row segments.
// Two tiles. 64x64, a 32x32 block per wave; and 32x32, a quarter of the stage's k per wave, where
// the 64x64 tiles are fewer than the compute units: four times the workgroups, each with a
// quarter of the products per k and twice the k per stage (float32, 700 x 768 -> 432: 14.1 us
// against 26.0; 512 x 1024 -> 1024: 18.3 against 34.3).
// Bound: a small product by its chain of stages, about 1 us each, and the launch (512 x 256 ->
// 256: 10.0 us, 6.0 of them the kernel); a large one by the FP32 matrix rate and LDS staging
// (4096 x 1024 -> 4096: 107 TFLOP/s of the part's 154).
#include "forge_lin_kernel.h"

namespace forge {
namespace {

// B x B output elements, stages of BK k, LD: k per row of the staged operands. B = 64: the waves
// are 2 x 2 of 32x32; B = 32: each wave takes a quarter of the stage's k for the whole tile.
template <int B_>
struct STile {
  static constexpr int B = B_, BK = B_ == 64 ? 32 : 64, VE = 4, LD = BK + VE;
  static constexpr int KW = B_ == 64 ? BK : BK / 4;  // k of a wave's products per stage
  static constexpr int LDE = B + 4;
};
constexpr int S_B = 64, S_NT = 256;
// workgroups of a launch at most (each walks several tiles beyond that): a grid holds fewer
// than 2^32 threads
constexpr int64_t kSimpleGrid = 1 << 20;

// 16 bytes of an operand: KS: its rows are k (row k0 + r, columns c..), else its rows are
// the output index (row r, k = k0 + c ..). Zero outside.
__device__ __forceinline__ u32x4 load16(const float* base, int64_t ld, int row, int rows, int col, int cols) {
  u32x4 z{0u, 0u, 0u, 0u};
  if (row < rows && col < cols) z = *reinterpret_cast<const u32x4*>(base + (int64_t)row * ld + col);
  return z;
}

// One operand's stage: B output indexes x BK k, as rows of k of pitch LD.
template <class C, bool TR>
struct Stage {
  static constexpr int VE = C::VE, LD = C::LD, S_B = C::B, S_BK = C::BK;
  static constexpr int CH = S_B * S_BK / VE / S_NT;  // 16-byte chunks per thread
  u32x4 r[CH];
  // r0: first output index of the tile, R: how many there are
  __device__ __forceinline__ void load(const float* p, int64_t ld, int r0, int R, int k0, int K, int tid) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = tid + j * S_NT;
      if constexpr (TR) {
        const int kr = c / (S_B / VE), col = (c % (S_B / VE)) * VE;
        // a chunk may reach past R inside its row's pitch (R need not be a multiple of VE
        // where the row is padded); those elements feed outputs that are never stored
        r[j] = load16(p, ld, k0 + kr, K, r0 + col, R);
      } else {
        const int row = c / (S_BK / VE), kc = (c % (S_BK / VE)) * VE;
        r[j] = load16(p, ld, r0 + row, R, k0 + kc, K);
      }
    }
  }
  __device__ __forceinline__ void store(float* s, int tid) const {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = tid + j * S_NT;
      if constexpr (TR) {
        const int kr = c / (S_B / VE), col = (c % (S_B / VE)) * VE;
#pragma unroll
        for (int i = 0; i < VE; ++i) s[(col + i) * LD + kr] = bits_f32(r[j][i]);
      } else {
        const int row = c / (S_BK / VE), kc = (c % (S_BK / VE)) * VE;
        *reinterpret_cast<u32x4*>(s + row * LD + kc) = r[j];
      }
    }
  }
};

// 32 x 32 products over the wave's k of a stage, from 16-byte LDS reads: lane half hi holds
// elements 8 j + 4 hi .. of both operands' rows, so a product of two k takes one from each half
template <class C>
__device__ __forceinline__ void mma32(f32x16& acc, const float* as, const float* bs, int row_a, int row_b, int k0, int hi) {
#pragma unroll
  for (int k = 0; k < C::KW; k += 2 * C::VE) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(as + row_a * C::LD + k0 + k + C::VE * hi);
    const u32x4 b = *reinterpret_cast<const u32x4*>(bs + row_b * C::LD + k0 + k + C::VE * hi);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(bits_f32(a[i]), bits_f32(b[i]), acc, 0, 0, 0);
  }
}

template <class C, int EPI, bool TA, bool TB>
__global__ __launch_bounds__(S_NT) void lin_simple_kernel(LinArgs g) {
  constexpr bool TWO = EPI == L_GATED;
  constexpr int S_B = C::B, S_BK = C::BK, LDE = C::LDE;
  constexpr int PARTS = S_B == 64 ? 1 : 4, ET = S_B * LDE;  // partial tiles of a product, floats of one
  static_assert(EPI != L_LSE || S_B == 64, "the cross entropy's blocks are of 64 entries");
  constexpr int OP = S_B * C::LD * 4;
  constexpr int EB = (TWO ? 2 : 1) * PARTS * ET * 4, OB = (TWO ? 3 : 2) * OP;
  __shared__ __attribute__((aligned(16))) uint8_t smem[EB > OB ? EB : OB];
  float* as = reinterpret_cast<float*>(smem);
  float* bs = reinterpret_cast<float*>(smem + OP);
  float* as2 = reinterpret_cast<float*>(smem + (TWO ? 2 * OP : 0));
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l32 = lane & 31, hi = lane >> 5;
  const int wm = PARTS > 1 ? 0 : (wave & 1) * 32, wn = PARTS > 1 ? 0 : (wave >> 1) * 32;
  const int wk = PARTS > 1 ? wave * C::KW : 0;
  const float sc = (EPI == L_ACC || EPI == L_DLOGIT) ? epi_scale(g.e) : 1.f;

  const int tiles_m = (epi_width<EPI>(g.M) - g.m_off + S_B - 1) / S_B, tiles_n = (g.N - g.n_off + S_B - 1) / S_B;
  for (int64_t tile = blockIdx.x; tile < (int64_t)tiles_m * tiles_n; tile += gridDim.x) {
  const int m0 = g.m_off + (int)(tile % tiles_m) * S_B, n0 = g.n_off + (int)(tile / tiles_m) * S_B;
  f32x16 acc, acc2;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc2[i] = 0.f;
  Stage<C, TA> sa, sa2;
  Stage<C, TB> sb;
  for (int s = 0; s < g.nsrc; ++s) {
    const float* A = static_cast<const float*>(g.A[s]);
    const float* A2 = static_cast<const float*>(g.A[TWO ? 1 : 0]);
    const float* B = static_cast<const float*>(g.B[s]);
    const int K = g.K[s];
    auto fetch = [&](int k0) {
      sa.load(A, g.lda[s], m0, g.M, k0, K, tid);
      if constexpr (TWO) sa2.load(A2, g.lda[1], m0, g.M, k0, K, tid);
      sb.load(B, g.ldb[s], n0, g.N, k0, K, tid);
    };
    if (K > 0) fetch(0);
    for (int k0 = 0; k0 < K; k0 += S_BK) {
      __syncthreads();  // the previous stage is consumed
      sa.store(as, tid);
      if constexpr (TWO) sa2.store(as2, tid);
      sb.store(bs, tid);
      __syncthreads();
      if (k0 + S_BK < K) fetch(k0 + S_BK);
      mma32<C>(acc, as, bs, wm + l32, wn + l32, wk, hi);
      if constexpr (TWO) mma32<C>(acc2, as2, bs, wm + l32, wn + l32, wk, hi);
    }
  }
  __syncthreads();
  // lane holds C[m = 8q + 4 hi + j][n = l32] of its 32x32 block: rows of the output in LDS
  float* E = reinterpret_cast<float*>(smem);
  float* E2 = E + (TWO ? PARTS * ET : 0);
  const int ew = PARTS > 1 ? wave * ET : 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int at = ew + (wn + l32) * LDE + wm + 8 * q + 4 * hi;
    *reinterpret_cast<f32x4*>(E + at) = f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
    if constexpr (TWO)
      *reinterpret_cast<f32x4*>(E2 + at) = f32x4{acc2[4 * q], acc2[4 * q + 1], acc2[4 * q + 2], acc2[4 * q + 3]};
  }
  __syncthreads();
  if constexpr (EPI == L_LSE) {
    // four threads per output row, 16 of the tile's 64 entries each
    const int n = n0 + (tid >> 2), c0 = (tid & 3) * 16;
    const float* row = E + (tid >> 2) * LDE + c0;
    const int left = g.M - m0 - c0;  // entries inside the vocabulary
    float mx = -__builtin_huge_valf();
    for (int j = 0; j < 16; ++j)
      if (j < left) mx = fmaxf(mx, row[j]);
    mx = fmaxf(mx, __shfl_xor(mx, 1));
    mx = fmaxf(mx, __shfl_xor(mx, 2));
    float sum = 0.f;
    const float ref = mx > -__builtin_huge_valf() ? mx : 0.f;  // an empty or all -inf block sums to 0
    for (int j = 0; j < 16; ++j)
      if (j < left) sum += __expf(row[j] - ref);
    sum += __shfl_xor(sum, 1);
    sum += __shfl_xor(sum, 2);
    if (n < g.N) {
      const int64_t y = g.e.target[n], hit = y - (m0 + c0);
      if (y >= 0 && hit >= 0 && hit < 16 && hit < left) g.e.tlogit[n] = row[hit];
      if ((tid & 3) == 0) {
        float* o = g.e.part + ((int64_t)(m0 / S_B) * g.e.part_ld + n) * 2;
        o[0] = mx;
        o[1] = sum;
      }
    }
  } else {
    const int Mw = epi_width<EPI>(g.M);
    act_dispatch<EPI>(g.e.act, [&](auto act_c) {
      for (int j = 0; j < S_B * S_B / 4 / S_NT; ++j) {
        const int v = tid + j * S_NT, r = v / (S_B / 4), c = (v % (S_B / 4)) * 4;
        const int n = n0 + r, m = m0 + c;
        if (n >= g.N || m >= Mw) continue;
        f32x4 x = *reinterpret_cast<const f32x4*>(E + r * LDE + c), x2 = x;
        if constexpr (TWO) x2 = *reinterpret_cast<const f32x4*>(E2 + r * LDE + c);
#pragma unroll
        for (int p = 1; p < PARTS; ++p) {  // the waves' sums, in order
          x = x + *reinterpret_cast<const f32x4*>(E + p * ET + r * LDE + c);
          if constexpr (TWO) x2 = x2 + *reinterpret_cast<const f32x4*>(E2 + p * ET + r * LDE + c);
        }
        epi_vec<float, EPI, decltype(act_c)::value>(g.e, n, m, g.M, x, x2, sc);
      }
    });
  }
  }
}

template <class C, int EPI, bool TA, bool TB>
hipError_t run(const LinArgs& g, hipStream_t st) {
  const int64_t gx = (epi_width<EPI>(g.M) - g.m_off + C::B - 1) / C::B, gy = (g.N - g.n_off + C::B - 1) / C::B;
  if (gx <= 0 || gy <= 0) return hipSuccess;
  const int64_t tiles = gx * gy;
  hipLaunchKernelGGL((lin_simple_kernel<C, EPI, TA, TB>), dim3((uint32_t)(tiles < kSimpleGrid ? tiles : kSimpleGrid)),
                     dim3(S_NT), 0, st, g);
  return hipGetLastError();
}

// 32x32 tiles where the 64x64 ones are fewer than the compute units
template <int EPI, bool TA, bool TB>
hipError_t lin_f32(const LinArgs& g, hipStream_t st) {
  if constexpr (EPI != L_LSE) {
    if (((int64_t)g.M + 63) / 64 * (((int64_t)g.N + 63) / 64) < g_num_cus()) return run<STile<32>, EPI, TA, TB>(g, st);
  }
  return run<STile<64>, EPI, TA, TB>(g, st);
}

// Whether the kernel for a few tokens takes a forward product. It reads the tokens once per 16
// rows of W, past the first-level cache's rate as they grow in number, where the tiles read
// them once per 64: above 16 tokens it keeps the layers with tiles for a quarter of the chip at
// most (32 x 14336 -> 4096: 40 us against 47; 32 x 8192 -> 8192: 45 against 30), above 4 also those
// that fill more than two rounds or less than half of one (16 x 4096 -> 14336: 32 against 22; 16 x
// 4096 -> 4096: 11 against 17; 4 x 4096 -> 40000: 63 against 87).
bool few_tokens(int epi, const LinArgs& g) {
  // (a grid of fewer than 2^32 threads)
  if (g.N > kSkinny || g.M >= (1 << 26)) return false;
  const int64_t tiles = ((epi == L_GATED ? 2 : 1) * (int64_t)g.M + 63) / 64, cus = g_num_cus();
  if (g.N > 16) return 4 * tiles <= cus;
  return g.N <= 4 || 2 * tiles <= cus || tiles > 2 * cus;
}

}  // namespace

#define FORGE_EXTERN_LIN(E, A, B) extern template hipError_t lin_bf16<E, A, B>(const LinArgs&, hipStream_t);
FORGE_LIN_FORMS(FORGE_EXTERN_LIN)
#undef FORGE_EXTERN_LIN

hipError_t launch_lin(int bf16, int epi, bool ta, bool tb, const LinArgs& g, hipStream_t st) {
  if (bf16 && (epi == L_LINEAR || epi == L_GATED) && few_tokens(epi, g)) return launch_lin_skinny(epi, g, st);
#define FORGE_PICK(E, A, B) \
  if (epi == E && ta == A && tb == B) return bf16 ? lin_bf16<E, A, B>(g, st) : lin_f32<E, A, B>(g, st);
  FORGE_LIN_FORMS(FORGE_PICK)
#undef FORGE_PICK
  return hipErrorInvalidValue;
}

int lin_splits(int bf16, int64_t M, int64_t N, int64_t K) {
  if (!bf16) return 1;
  const LinTileKind kind = lin_tile<L_ACC>(M, N);
  const int64_t stages = (K + 63) / 64;
  if (kind == LT_BIG || kind == LT_SMALL || stages < kSplitStages) return 1;
  const int64_t b = lin_split_big(M, N, K) ? 256 : 128, slots = (int64_t)g_num_cus() * (b == 256 ? 1 : 2);
  int64_t s = slots / (((M + b - 1) / b) * ((N + b - 1) / b));
  if (s > stages / 12) s = stages / 12;
  if (s > 32) s = 32;
  return s < 2 ? 1 : (int)s;
}

int lin_lse_block(int bf16, int M, int N) {
  if (!bf16) return S_B;
  switch (lin_tile<L_LSE>(M, N)) {
    case LT_BIG: return LinBig::TM;  // a wave's entries
    case LT_SMALL: return LinSmall::TM;
    case LT_SPLIT: return LinSplit::BM;  // a tile's
    default: return LinTiny::BM;
  }
}

}  // namespace forge
