// Internal: the operators around the fused weight-gradient step: products with an
// epilogue (linear forward, gated block, their gradients, softmax cross entropy of a
// linear head). This file holds their arguments, the activations and the epilogues;
// the kernels are in forge_lin_kernel.h (bfloat16 products), forge_lin_skinny.hip (a few tokens),
// forge_lin_simple.hip (float32, and the choice between the bfloat16 ones) and forge_ops_rows.hip (passes
// without a product).
//
// Every product here is C[m][n] = sum_k A[m][k] B[n][k] with m the output's columns
// (features, contiguous in memory) and n its rows (tokens), so a lane's four consecutive
// accumulator rows are four neighbouring elements of one output row:
//   forward      m = out, n = tokens, k = in:   A = W (k fast), B = X (k fast)
//   input grad.  m = in, n = tokens, k = out:   A = W (k slow: its rows are k), B = dY (k fast)
//   weight grad. m = in, n = out, k = tokens:   A = X (k slow), B = dY (k slow)
#pragma once

#include <type_traits>

#include "forge_internal.h"

namespace forge {

// ---------------------------------------------------------------------------
// activations (FP32): value and derivative
// ---------------------------------------------------------------------------
// 1 / (1 + e^-z) on the hardware exponential and reciprocal (each within about an ulp);
// z -> -inf gives 1 / inf = 0.
__device__ __forceinline__ float sigmoid_f(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// Phi(z), the normal distribution function, and e^(-z^2/2), which its derivative needs as
// well. T: the type of the results.
// bfloat16: erfc(x) = t (a1 + t (a2 + ... )) e^(-x^2), t = 1 / (1 + 0.3275911 x) (Abramowitz and
// Stegun, Handbook of Mathematical Functions, 7.1.26), one exponential for both results. Its
// absolute error stays below 1.5e-7; the relative one of the left tail is 5e-4 at z = -4 and
// 1.7e-3 at -5, below half a bfloat16 step (3.9e-3) down to -6, where Phi is 1e-9.
// float32: the library's erfc and exponential; relative to Phi (z^2 + 1) 2^-23 from the rounding
// of z / sqrt 2, and erfc's own ulps, all the way down the tail (the short form: 5e-5 at z = -3).
// It costs the float32 epilogue backward pass of 8192 x 4096 93 us against 86, a product 1%.
template <class T>
__device__ __forceinline__ float normal_cdf_f(float z, float& gauss) {
  const float x = fabsf(z) * 0.70710678118654752f;
  float half_erfc;
  if constexpr (std::is_same<T, float>::value) {
    gauss = expf(-0.5f * z * z);
    half_erfc = 0.5f * erfcf(x);
  } else {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, x, 1.f));
    gauss = __expf(-0.5f * z * z);
    float p = fmaf(t, 1.061405429f, -1.453152027f);
    p = fmaf(t, p, 1.421413741f);
    p = fmaf(t, p, -0.284496736f);
    p = fmaf(t, p, 0.254829592f);
    half_erfc = 0.5f * t * p * gauss;
  }
  return z < 0.f ? half_erfc : 1.f - half_erfc;
}

constexpr float kGeluC = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluK = 0.044715f;

template <class T>
__device__ __forceinline__ float act_f(float z, int act) {
  switch (act) {
    case FORGE_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);  // NaN stays NaN
    case FORGE_ACT_SILU: return z * sigmoid_f(z);
    case FORGE_ACT_GELU: {
      float e;
      return z * normal_cdf_f<T>(z, e);
    }
    case FORGE_ACT_GELU_TANH:  // z (1 + tanh u) / 2 = z sigmoid(2u)
      return z * sigmoid_f(2.f * kGeluC * z * fmaf(kGeluK * z, z, 1.f));
    default: return z;
  }
}
// value a and derivative d
template <class T>
__device__ __forceinline__ void act_vd(float z, int act, float& a, float& d) {
  switch (act) {
    case FORGE_ACT_RELU:
      a = z > 0.f ? z : (z != z ? z : 0.f);
      d = z > 0.f ? 1.f : (z != z ? z : 0.f);
      return;
    case FORGE_ACT_SILU: {
      const float s = sigmoid_f(z);
      a = z * s;
      d = fmaf(a, 1.f - s, s);
      return;
    }
    case FORGE_ACT_GELU: {
      float e;
      const float c = normal_cdf_f<T>(z, e);
      a = z * c;
      d = fmaf(z * 0.39894228040143268f, e, c);
      return;
    }
    case FORGE_ACT_GELU_TANH: {
      const float s = sigmoid_f(2.f * kGeluC * z * fmaf(kGeluK * z, z, 1.f));
      a = z * s;
      // (a (1 - s) first and the slope of u bounded: z^2 and 2 z overflow where that product is 0
      // already, and 0 inf is NaN)
      d = fmaf(a * (1.f - s), 2.f * kGeluC * fminf(fmaf(3.f * kGeluK * z, z, 1.f), 1e30f), s);
      return;
    }
    default:
      a = z;
      d = 1.f;
      return;
  }
}

// ---------------------------------------------------------------------------
// element access: T = uint16_t holds bfloat16 bits, T = float holds float32
// ---------------------------------------------------------------------------
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
  const u32x2 r = *reinterpret_cast<const u32x2*>(p);
  return f32x4{bits_f32(r.x << 16), bits_f32(r.x & 0xFFFF0000u), bits_f32(r.y << 16), bits_f32(r.y & 0xFFFF0000u)};
}
__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ void store4(uint16_t* p, f32x4 x) {
  // the compiler's conversion: v_cvt_pk_bf16_f32, nearest-even, two elements per instruction
  *reinterpret_cast<u32x2*>(p) = __builtin_bit_cast(u32x2, __builtin_convertvector(x, bf16x4));
}
__device__ __forceinline__ void store4(float* p, f32x4 x) { *reinterpret_cast<f32x4*>(p) = x; }

// ---------------------------------------------------------------------------
// arguments
// ---------------------------------------------------------------------------
// Epilogues of the products. Outputs are rounded to the operands' type once. dG and dU (L_DGATE) and dz
// (L_DLOGIT) are rounded before the products that follow them: those run on the matrix cores in the
// operands' type, and the fused steps take dG, dU and dz as they are. For bf16 that is half a step
// (2^-9 to 2^-8) of each element, independent over the sum: the relative error of dX and dW is 0.0023
// and 0.0019 where float32 intermediates would leave the outputs' own 0.0017.
enum LinEpi {
  L_LINEAR = 0,  // out = act(x + bias) + in1; out2 = x + bias (the pre-activation), if asked for
  L_GATED = 1,   // two products g, u: out = act(g) u; out2 = g, out3 = u, if asked for
  L_DGATE = 2,   // x = dH: out = dG, out2 = dU, out3 = H (if asked for) from in1 = G, in2 = U
  L_ACC = 3,     // out = (x + acc) * scale, or acc = x (+ acc): products summed over pieces
  L_LSE = 4,     // per output row: the tile's maximum and sum of exponentials, the target's logit
  L_DLOGIT = 5,  // out = (exp(x - lse) - [m is the target]) * the token's weight
};

struct LinEpiArgs {
  int32_t act;
  void* out;
  void* out2;
  void* out3;
  int64_t ldo, ldo2, ldo3;
  const void* in1;
  const void* in2;
  int64_t ld1, ld2;
  const void* bias;  // one element per output column, float32 (bias_f32) or the operands' type
  int32_t bias_f32;
  // L_ACC: float32 sums over pieces; read and / or written instead of out
  float* acc;
  int64_t ldacc;
  int32_t acc_read, acc_write;
  // a factor held in device memory: scale[0] (1 where there is none), divided by count[0]
  // where count is given (0 where that count is 0)
  const float* scale;
  const float* count;
  // cross entropy (L_DLOGIT: m counts the entries of a piece whose first one is entry v0)
  const int64_t* target;
  int64_t ignore, v0, vocab;
  const float* lse;
  const float* weight;  // L_DLOGIT: one factor per token, or NULL
  float* part;          // L_LSE: [blocks of the vocabulary][tokens][2]: maximum, sum of exponentials
  int64_t part_ld;      // tokens
  float* tlogit;        // L_LSE: logit of each token's target
  // 8-bit operands: factors of the integer sums, one per token, one per output column (sw2: those
  // of L_GATED's second product)
  const float* sx;
  const float* sw;
  const float* sw2;
};

constexpr int kMaxSrc = FORGE_MAX_GROUP;
struct LinArgs {
  // operand pairs whose products are summed (L_GATED: A[0] and A[1] are gate and up, one B)
  const void* A[kMaxSrc];
  const void* B[kMaxSrc];
  int64_t lda[kMaxSrc], ldb[kMaxSrc];
  int32_t K[kMaxSrc];
  int32_t nsrc;
  int32_t M, N;
  int32_t m_off, n_off;  // origin of this launch's tiles
  // L_ACC with k-slow A, bf16: parts that share a tile's k range, each with float32 sums of its
  // own, N x ldacc apart from e.acc on (acc_write; added by launch_acc_join)
  int32_t splits;
  // Products grouped by expert: expert x owns rows offsets[x] .. offsets[x + 1] - 1 of the N rows of
  // B and of the output, and the x-th of the stacked matrices A
  int32_t experts;
  // workgroups of a whole round of the large tiles, where a last round that is at most half full is left
  // to the smaller ones of a second launch (LM_TAIL); 0: it is not
  int32_t round;
  const int64_t* offsets;
  LinEpiArgs e;
};

// One pair of operands of a product.
inline void set_pair(LinArgs& g, int s, const void* A, int64_t lda, const void* B, int64_t ldb, int64_t K) {
  g.A[s] = A;
  g.lda[s] = lda;
  g.B[s] = B;
  g.ldb[s] = ldb;
  g.K[s] = (int32_t)K;
}

// Forms of a product's kernel.
enum LinMode {
  LM_EXPERT = 1,  // grouped by expert
  LM_TAIL = 4,    // grouped by expert: quarters of the last round's large tiles
  LM_Q8 = 2,      // operands of 8-bit integers (LinArgs' K and pitches count pairs of them), bfloat16 output
};

// The rows of a product's experts, spread over the lanes of a wave (64 experts at a time): lane i
// holds those of expert base + i. The offsets come from device memory, so they are held to 0 .. N and to
// ascending order here: no value of theirs leads outside the operands.
template <int BN>
struct ExpertRows {
  const int64_t* off;
  int experts, rows;  // how many, all rows of the operand
  int base, r0, r1, upto;  // upto: tiles of BN rows of the experts base .. base + lane
  __device__ __forceinline__ void load(int first) {
    const int lane = static_cast<int>(threadIdx.x) & 63, x = first + lane;
    base = first;
    const bool in = x < experts;
    const int64_t a = in ? off[x] : 0, b = in ? off[x + 1] : 0;
    r0 = (int)(a < 0 ? 0 : a > rows ? rows : a);
    r1 = (int)(b < r0 ? r0 : b > rows ? rows : b);
    upto = (r1 - r0 + BN - 1) / BN;
#pragma unroll
    for (int h = 1; h < 64; h <<= 1) {
      const int other = __shfl_up(upto, h);
      if (lane >= h) upto += other;
    }
  }
  // tiles of rows of all experts (offsets that are none may claim rows twice: no more than there can be);
  // afterwards the first 64 are loaded
  __device__ __forceinline__ int total() {
    int64_t n = 0;
    for (int first = (experts - 1) / 64 * 64; first >= 0; first -= 64) {
      load(first);
      n += __builtin_amdgcn_readlane(upto, 63);
    }
    const int64_t most = (rows + BN - 1) / BN + min(experts, rows);
    return (int)(n < most ? n : most);
  }
  // the expert of row tile q, its first row and its end, its first row tile
  __device__ __forceinline__ void find(int q, int& x, int& first_row, int& end_row, int& first_tile) {
    int before = 0;
    if (base != 0) load(0);
    while (true) {
      const int here = __builtin_amdgcn_readlane(upto, 63);
      if (q < before + here || base + 64 >= experts) break;
      before += here;
      load(base + 64);
    }
    const uint64_t hit = __ballot(q - before < upto);
    const int lane = hit ? __builtin_ctzll(hit) : 0;
    x = base + lane;
    first_row = __builtin_amdgcn_readlane(r0, lane);
    end_row = __builtin_amdgcn_readlane(r1, lane);
    first_tile = before + __builtin_amdgcn_readlane(upto, lane) - (end_row - first_row + BN - 1) / BN;
  }
  // the q-th expert that has rows; false: there is none
  __device__ __forceinline__ bool find_used(int q, int& x, int& first_row, int& end_row) {
    for (int first = 0; first < experts; first += 64) {
      load(first);
      uint64_t used = __ballot(r1 > r0);
      const int n = __popcll(used);
      if (q < n) {
        for (; q > 0; --q) used &= used - 1;
        const int lane = __builtin_ctzll(used);
        x = first + lane;
        first_row = __builtin_amdgcn_readlane(r0, lane);
        end_row = __builtin_amdgcn_readlane(r1, lane);
        return true;
      }
      q -= n;
    }
    return false;
  }
};

// the integer sums of 8-bit operands as floats: exact below 2^24, else rounded once (2^-24, where the
// bfloat16 result is rounded to 2^-8)
typedef int i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ f32x4 int_sums(f32x4 bits) {
  return __builtin_convertvector(__builtin_bit_cast(i32x4, bits), f32x4);
}

// the factor of L_ACC / L_DLOGIT
__device__ __forceinline__ float epi_scale(const LinEpiArgs& e) {
  float s = e.scale ? e.scale[0] : 1.f;
  if (e.count) s = e.count[0] > 0.f ? s / e.count[0] : 0.f;
  return s;
}

// The arithmetic of an epilogue on 4 neighbouring columns: x the product (x2 the second one of
// L_GATED), a and b what it reads from in1 and in2 (zero where there is none), y0 .. y2 what it
// writes to out .. out3; T the type of the results.
template <class T, int EPI>
__device__ __forceinline__ void epi_math(int act, f32x4 x, f32x4 x2, f32x4 a, f32x4 b, f32x4& y0, f32x4& y1, f32x4& y2) {
  if constexpr (EPI == L_LINEAR) {  // x: bias added
    y1 = x;
    y0 = f32x4{act_f<T>(x.x, act), act_f<T>(x.y, act), act_f<T>(x.z, act), act_f<T>(x.w, act)} + a;
  } else if constexpr (EPI == L_GATED) {
    y0 = f32x4{act_f<T>(x.x, act), act_f<T>(x.y, act), act_f<T>(x.z, act), act_f<T>(x.w, act)} * x2;
    y1 = x;
    y2 = x2;
  } else if constexpr (EPI == L_DGATE) {  // x = dH, a = G, b = U
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v, d;
      act_vd<T>(a[j], act, v, d);
      y0[j] = x[j] * (b[j] * d);
      y1[j] = x[j] * v;
      y2[j] = v * b[j];
    }
  }
}

// dz of 4 logits x of one token: m the first one's place, M the piece's entries (past them the
// row is padded with zeros), hit the target's place (-1: not here), l = lse, w the factor (0
// with ignored = true, NaN for a target outside the vocabulary)
__device__ __forceinline__ f32x4 dlogit(f32x4 x, int m, int M, int hit, float l, float w, bool ignored) {
  f32x4 d;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float p = __expf(x[j] - l);
    d[j] = m + j < M && !ignored ? (p - (hit == m + j ? 1.f : 0.f)) * w : 0.f;
  }
  return d;
}
// a token's target as dlogit takes it
__device__ __forceinline__ void dlogit_row(const LinEpiArgs& e, int64_t y, float weight, float sc, int& hit, float& w,
                                           bool& ignored) {
  ignored = y == e.ignore;
  const bool bad = y < 0 || y >= e.vocab;
  const int64_t d = bad ? -1 : y - e.v0;
  hit = d >= 0 && d < ((int64_t)1 << 30) ? (int)d : -1;
  w = bad ? __builtin_nanf("") : weight * sc;
}

// f(integral_constant<act>): one branch on the activation around a whole loop, where the epilogue
// has one
template <int EPI, class F>
__device__ __forceinline__ void act_dispatch(int act, F&& f) {
  if constexpr (EPI != L_LINEAR && EPI != L_GATED && EPI != L_DGATE) {
    f(std::integral_constant<int, FORGE_ACT_NONE>{});
  } else {
    switch (act) {
      case FORGE_ACT_RELU: f(std::integral_constant<int, FORGE_ACT_RELU>{}); break;
      case FORGE_ACT_SILU: f(std::integral_constant<int, FORGE_ACT_SILU>{}); break;
      case FORGE_ACT_GELU: f(std::integral_constant<int, FORGE_ACT_GELU>{}); break;
      case FORGE_ACT_GELU_TANH: f(std::integral_constant<int, FORGE_ACT_GELU_TANH>{}); break;
      default: f(std::integral_constant<int, FORGE_ACT_NONE>{}); break;
    }
  }
}

// One 4-vector of the output: row n, columns m..m+3 (all inside the output's padded
// width); x the product, x2 the second product of L_GATED; sc = epi_scale; ACT = e.act; acc0: offset of
// the float32 sums.
template <class T, int EPI, int ACT>
__device__ __forceinline__ void epi_vec(const LinEpiArgs& e, int n, int m, int M, f32x4 x, f32x4 x2, float sc,
                                        int64_t acc0 = 0) {
  if constexpr (EPI == L_ACC) {
    if (e.acc_read) x = x + load4(e.acc + acc0 + (int64_t)n * e.ldacc + m);
    if (e.acc_write)
      store4(e.acc + acc0 + (int64_t)n * e.ldacc + m, x);
    else
      store4(static_cast<T*>(e.out) + (int64_t)n * e.ldo + m, x * sc);
  } else if constexpr (EPI == L_DLOGIT) {
    int hit;
    float w;
    bool ignored;
    dlogit_row(e, e.target[n], e.weight ? e.weight[n] : 1.f, sc, hit, w, ignored);
    store4(static_cast<T*>(e.out) + (int64_t)n * e.ldo + m, dlogit(x, m, M, hit, e.lse[n], w, ignored));
  } else {
    f32x4 a{0.f, 0.f, 0.f, 0.f}, b = a, y0, y1, y2;
    if constexpr (EPI == L_LINEAR) {
      if (e.bias)
        x = x + (e.bias_f32 ? load4(static_cast<const float*>(e.bias) + m) : load4(static_cast<const T*>(e.bias) + m));
    }
    if (e.in1) a = load4(static_cast<const T*>(e.in1) + (int64_t)n * e.ld1 + m);
    if (e.in2) b = load4(static_cast<const T*>(e.in2) + (int64_t)n * e.ld2 + m);
    epi_math<T, EPI>(ACT, x, x2, a, b, y0, y1, y2);
    store4(static_cast<T*>(e.out) + (int64_t)n * e.ldo + m, y0);
    if (e.out2) store4(static_cast<T*>(e.out2) + (int64_t)n * e.ldo2 + m, y1);
    if (e.out3) store4(static_cast<T*>(e.out3) + (int64_t)n * e.ldo3 + m, y2);
  }
}

// width of an output row that the epilogue writes: L_DLOGIT pads its rows with zeros to a
// multiple of 8 entries, which the products that read them take as whole 16-byte chunks
template <int EPI>
__host__ __device__ constexpr int epi_width(int M) {
  return EPI == L_DLOGIT ? (M + 7) / 8 * 8 : M;
}

// Host-side launchers. bf16: operands in bfloat16, else float32. ta / tb: the operand's
// slow index is k (its rows are k), else k is the fast index.
hipError_t launch_lin(int bf16, int epi, bool ta, bool tb, const LinArgs& g, hipStream_t st);
// products grouped by expert (g.offsets, g.experts); forward products of 8-bit operands, grouped where
// g.experts > 0
hipError_t launch_lin_expert(int bf16, int epi, bool ta, const LinArgs& g, hipStream_t st);
hipError_t launch_lin_q8(int epi, const LinArgs& g, hipStream_t st);
// forward products (L_LINEAR, L_GATED) of at most kSkinny tokens, bf16 (launch_lin chooses); mode: LinMode,
// grouped by expert any number
constexpr int kSkinny = 32;
hipError_t launch_lin_skinny(int mode, int epi, const LinArgs& g, hipStream_t st);
// whether a forward product of so few tokens is one for launch_lin_skinny
bool few_tokens(int epi, const LinArgs& g);
// the same of one that is grouped by expert
bool few_rows(const LinArgs& g);
// vocabulary entries per partial result that launch_lin(L_LSE) writes for this product
int lin_lse_block(int bf16, int M, int N);

// edge of the tiles that a bfloat16 or an 8-bit product by expert is cut into (0: the kernel for a few rows)
int lin_expert_edge(int epi, bool ta, int64_t M, int64_t N, int64_t K, int experts);
int lin_q8_expert_edge(int epi, int64_t M, int64_t N, int64_t K, int experts);
// parts a product of k-slow A should be cut into (1: none): too few tiles to fill the chip with,
// a k range long enough to share
int lin_splits(int bf16, int64_t M, int64_t N, int64_t K);
// the same of an input gradient that is grouped by expert (by rows and experts alone: the sizes are on the device)
int lin_expert_splits(int bf16, int64_t M, int64_t N, int experts, int64_t K);
// out = (sum of the parts' sums, in order) * scale
hipError_t launch_acc_join(const LinArgs& g, hipStream_t st);

// dZ = dY act'(Z) and db = its column sums in float32 (partial sums of blocks of rows go to
// ws, act_backward_blocks(T, out) x out floats, when there is more than one block)
int act_backward_blocks(int64_t T, int64_t out);
hipError_t launch_act_backward(int bf16, int act, const void* dY, int64_t lddy, const void* Z, int64_t ldz, void* dZ,
                               int64_t lddz, float* db, float* ws, int T, int out, hipStream_t st);
// dG, dU and (if H) H from dH, G, U
hipError_t launch_gated_backward(int bf16, const void* dH, int64_t lddh, const LinEpiArgs& e, int T, int hid,
                                 hipStream_t st);
// ---- experts (forge_expert.hip) ----
// blocks of routes that a plan of n routes takes (one: no workspace), routes of each
int64_t expert_plan_blocks(int64_t n, int64_t* per);
// counts: blocks x experts integers of workspace
hipError_t launch_expert_plan(const int64_t* idx, int64_t n, int experts, int64_t* offsets, int* pos, int* counts,
                              hipStream_t st);
// rows of `chunks` 16-byte pieces; places: rows of Y; sx, sy: factors that go along, or NULL
hipError_t launch_expert_dispatch(const void* X, int64_t ldx_bytes, const int* pos, int k, int64_t T, int64_t places,
                                  void* Y, int64_t ldy_bytes, int chunks, const float* sx, float* sy, hipStream_t st);
struct CombineArgs {
  const void* Yp;  // [places, cols]; may be NULL in the backward pass without dw
  int64_t ldp, places;
  const int* pos;  // [tokens, k]
  const float* w;  // [tokens, k], or NULL for ones
  int k;
  const void* R;   // residual or NULL
  int64_t ldr;
  void* Y;         // result; in the backward pass its gradient
  int64_t ldy, tokens;
  int cols;
  void* dYp;       // backward: either may be NULL
  int64_t lddp;
  float* dw;
};
// bf16: of the tokens' side (Y, R, dYp); wide: Yp in float32 beside it
hipError_t launch_expert_combine(int bf16, int wide, const CombineArgs& a, hipStream_t st);
hipError_t launch_expert_combine_backward(int bf16, int wide, const CombineArgs& a, hipStream_t st);
hipError_t launch_quantize_rows(int bf16, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* scale, int64_t rows,
                                int cols, hipStream_t st);

// joins the partial maxima and sums of nblk vocabulary blocks: lse, the per-token loss, and
// total = {sum of the losses, tokens counted, mean}; tsum: 2 * lse_join_groups(T) doubles
int lse_join_groups(int64_t T);
hipError_t launch_lse_join(const float* part, int64_t nblk, const float* tlogit, const int64_t* target, int64_t ignore,
                           int64_t vocab, float* loss, float* lse, float* total, double* tsum, int T, hipStream_t st);

}  // namespace forge
