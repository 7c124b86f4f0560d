// The operators' passes over rows that hold no product: the backward pass of the linear
// epilogue (gradient through the activation, bias gradient), the gated product's backward
// pass, and the join of the cross entropy's partial sums. All are bound by memory.
#include "forge_ops.h"

namespace forge {
namespace {

typedef uint16_t bf16_t;

// ---- dZ = dY act'(Z), db = column sums ------------------------------------
// A lane holds 16 bytes of a row (8 columns in bf16, 4 in fp32), a wave 64 such vectors; the 4
// waves of a workgroup take every fourth row of the workgroup's block of rows, AB_ROWS of their
// rows at a time: all loads of these rows are issued before the first of their stores, which
// the compiler could not move them across. A lane's column sums stay in float32 registers and
// are joined over the waves through LDS, then over the blocks of rows by act_bias_join, both
// in a fixed order. Memory bound: 8191 x 14336 bf16 GELU moves 705 MB in 153 us (4.6 TB/s, a
// copy reaches 4.9), 142 us among other calls; with 8 bytes per lane and one row at a time it
// took 178 us.
constexpr int AB_NT = 256, AB_ROWS = 4;
template <class T>
constexpr int kAbVec = 16 / (int)sizeof(T);  // columns per lane
template <class T>
constexpr int kAbCols = 64 * kAbVec<T>;

template <class T>
__global__ __launch_bounds__(AB_NT) void act_backward_kernel(int act, const T* dY, int64_t lddy, const T* Z, int64_t ldz,
                                                             T* dZ, int64_t lddz, float* part, int R, int out,
                                                             int rows_per) {
  constexpr int Q = kAbVec<T> / 4;  // 4-vectors per lane
  __shared__ __attribute__((aligned(16))) float red[3][Q][64 * 4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * kAbCols<T> + lane * kAbVec<T>;
  const int r0 = blockIdx.y * rows_per, r1 = min(R, r0 + rows_per);
  f32x4 sum[Q] = {};
  if (c < out) {
    act_dispatch<L_DGATE>(act, [&](auto act_c) {
      constexpr int ACT = decltype(act_c)::value;
      for (int r = r0 + wave; r < r1; r += 4 * AB_ROWS) {
        u32x4 d[AB_ROWS], z[AB_ROWS];
#pragma unroll
        for (int i = 0; i < AB_ROWS; ++i) {
          const int64_t ri = min(r + 4 * i, r1 - 1);  // past the block: its last row, not used
          d[i] = *reinterpret_cast<const u32x4*>(dY + ri * lddy + c);
          if constexpr (ACT != FORGE_ACT_NONE) z[i] = *reinterpret_cast<const u32x4*>(Z + ri * ldz + c);
        }
#pragma unroll
        for (int i = 0; i < AB_ROWS; ++i) {
          if (r + 4 * i >= r1) break;
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            f32x4 x = load4(reinterpret_cast<const T*>(&d[i]) + 4 * q);
            if constexpr (ACT != FORGE_ACT_NONE) {
              const f32x4 y = load4(reinterpret_cast<const T*>(&z[i]) + 4 * q);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float a, g;
                act_vd<T>(y[j], ACT, a, g);
                x[j] *= g;
              }
            }
            sum[q] = sum[q] + x;
            if (dZ) store4(reinterpret_cast<T*>(&d[i]) + 4 * q, x);
          }
          if (dZ) *reinterpret_cast<u32x4*>(dZ + (int64_t)(r + 4 * i) * lddz + c) = d[i];
        }
      }
    });
  }
  if (!part) return;
  if (wave) {
#pragma unroll
    for (int q = 0; q < Q; ++q) *reinterpret_cast<f32x4*>(&red[wave - 1][q][lane * 4]) = sum[q];
  }
  __syncthreads();
  if (wave == 0 && c < out) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
#pragma unroll
      for (int w = 0; w < 3; ++w) sum[q] = sum[q] + *reinterpret_cast<const f32x4*>(&red[w][q][lane * 4]);
      *reinterpret_cast<f32x4*>(part + (int64_t)blockIdx.y * out + c + 4 * q) = sum[q];
    }
  }
}

// 16 columns per workgroup, 16 threads to each: a thread adds every sixteenth block's sums, then
// the 16 partial sums are added in order. (One thread per column took 20 us of the 28 that 7839
// x 144 took; now 17 in all.)
constexpr int BJ_C = 16, BJ_G = 16;
__global__ __launch_bounds__(BJ_C* BJ_G) void act_bias_join(const float* part, int blocks, float* db, int out) {
  __shared__ float red[BJ_G][BJ_C];
  const int t = threadIdx.x % BJ_C, grp = threadIdx.x / BJ_C, c = blockIdx.x * BJ_C + t;
  float s = 0.f;
  if (c < out) {
#pragma unroll 8
    for (int b = grp; b < blocks; b += BJ_G) s += part[(int64_t)b * out + c];
  }
  red[grp][t] = s;
  __syncthreads();
  if (grp || c >= out) return;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < BJ_G; ++k) s += red[k][t];
  db[c] = s;
}

// ---- gated product's backward ---------------------------------------------
// Elementwise over 4-vectors; bound by memory (three tensors read, two or three written).
template <class T>
__global__ __launch_bounds__(256) void gated_backward_kernel(const T* dH, int64_t lddh, LinEpiArgs e, int R, int hid) {
  const int per = hid / 4;  // 4-vectors per row
  const int64_t total = (int64_t)R * per;
  act_dispatch<L_DGATE>(e.act, [&](auto act_c) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
      const int n = (int)(i / per), m = (int)(i - (int64_t)n * per) * 4;
      const f32x4 x = load4(dH + (int64_t)n * lddh + m);
      epi_vec<T, L_DGATE, decltype(act_c)::value>(e, n, m, hid, x, x, 1.f);
    }
  });
}

// ---- join of a split product's parts --------------------------------------
// In order, so the same bits every time; the parts come from the second-level cache mostly (1999
// x 1024 in 8 parts, 66 MB: 13 us). Grouped by expert: of the rows that belong to one.
__global__ __launch_bounds__(256) void acc_join_kernel(LinArgs g) {
  const int per = g.M / 4;
  const int64_t total = (int64_t)g.N * per, part = (int64_t)g.N * g.e.ldacc;
  const float sc = epi_scale(g.e);
  const int64_t n0 = g.offsets ? g.offsets[0] : 0, n1 = g.offsets ? g.offsets[g.experts] : g.N;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int n = (int)(i / per), m = (int)(i - (int64_t)n * per) * 4;
    if (n < n0 || n >= n1) continue;
    const float* p = g.e.acc + (int64_t)n * g.e.ldacc + m;
    f32x4 x = load4(p);
#pragma unroll 4
    for (int s = 1; s < g.splits; ++s) x = x + load4(p + s * part);
    store4(static_cast<bf16_t*>(g.e.out) + (int64_t)n * g.e.ldo + m, x * sc);
  }
}

// ---- join of the cross entropy's partial results --------------------------
// lse = M + log sum_b s_b e^(m_b - M) over the vocabulary blocks' (maximum, sum) pairs. 16
// tokens per workgroup, 16 threads of it (stride 16) share a token's blocks; the pairs of
// neighbouring tokens are neighbours in memory. The losses' sum is taken in double, in order.
// 1999 tokens x 393 blocks: 13 us, and 5 for the total.
constexpr int LJ_T = 16, LJ_G = 16;

__device__ __forceinline__ void lse_add(float& m, float& s, float m2, float s2) {
  const float M = fmaxf(m, m2);
  if (M == -__builtin_huge_valf()) {  // nothing yet (a NaN sum stays one)
    s += s2;
    return;
  }
  s = s * __expf(m - M) + s2 * __expf(m2 - M);
  m = M;
}

__global__ __launch_bounds__(256) void lse_join_kernel(const float* part, int64_t nblk, const float* tlogit,
                                                       const int64_t* target, int64_t ignore, int64_t vocab, float* loss,
                                                       float* lse, double* tsum, float* total, int R) {
  __shared__ float sm[LJ_G][LJ_T], ss[LJ_G][LJ_T];
  __shared__ float ls[LJ_T], cnt[LJ_T];
  const int t = threadIdx.x % LJ_T, grp = threadIdx.x / LJ_T, n = blockIdx.x * LJ_T + t;
  float m = -__builtin_huge_valf(), s = 0.f;
  if (n < R) {
#pragma unroll 4
    for (int64_t b = grp; b < nblk; b += LJ_G) {
      const float2 p = *reinterpret_cast<const float2*>(part + (b * R + n) * 2);
      lse_add(m, s, p.x, p.y);
    }
  }
  sm[grp][t] = m;
  ss[grp][t] = s;
  __syncthreads();
  if (grp == 0) {
    for (int k = 1; k < LJ_G; ++k) lse_add(m, s, sm[k][t], ss[k][t]);
    float l = 0.f, c = 0.f;
    if (n < R) {
      // no finite logit: m = -inf, s = 0: log 0 = -inf, as the sum says
      const float v = (m == -__builtin_huge_valf() ? 0.f : m) + logf(s);
      lse[n] = v;
      const int64_t y = target[n];
      if (y != ignore) {
        c = 1.f;
        l = (y >= 0 && y < vocab) ? v - tlogit[n] : __builtin_nanf("");
      }
      if (loss) loss[n] = l;
    }
    ls[t] = l;
    cnt[t] = c;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double a = 0.0, c = 0.0;
    for (int k = 0; k < LJ_T; ++k) {
      a += ls[k];
      c += cnt[k];
    }
    if (gridDim.x == 1) {
      total[0] = (float)a;
      total[1] = (float)c;
      total[2] = (float)(a / c);
    } else {
      tsum[2 * blockIdx.x] = a;
      tsum[2 * blockIdx.x + 1] = c;
    }
  }
}

__global__ __launch_bounds__(256) void lse_total_kernel(const double* tsum, int groups, float* total) {
  __shared__ double sa[256], sc[256];
  double a = 0.0, c = 0.0;
  for (int k = threadIdx.x; k < groups; k += 256) {
    a += tsum[2 * k];
    c += tsum[2 * k + 1];
  }
  sa[threadIdx.x] = a;
  sc[threadIdx.x] = c;
  __syncthreads();
  for (int h = 128; h > 0; h >>= 1) {
    if ((int)threadIdx.x < h) {
      sa[threadIdx.x] += sa[threadIdx.x + h];
      sc[threadIdx.x] += sc[threadIdx.x + h];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    total[0] = (float)sa[0];
    total[1] = (float)sc[0];
    total[2] = (float)(sa[0] / sc[0]);  // no token counted: NaN, as the mean of nothing
  }
}

template <class T>
hipError_t act_backward(int act, const void* dY, int64_t lddy, const void* Z, int64_t ldz, void* dZ, int64_t lddz,
                        float* db, float* ws, int R, int out, hipStream_t st) {
  const int blocks = act_backward_blocks(R, out);
  const int rows_per = (R + blocks - 1) / blocks;
  float* part = !db ? nullptr : (blocks == 1 ? db : ws);
  hipLaunchKernelGGL((act_backward_kernel<T>), dim3((out + kAbCols<T> - 1) / kAbCols<T>, blocks), dim3(AB_NT), 0, st, act,
                     static_cast<const T*>(dY), lddy, static_cast<const T*>(Z), ldz, static_cast<T*>(dZ), lddz, part, R,
                     out, rows_per);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !db || blocks == 1) return e;
  hipLaunchKernelGGL(act_bias_join, dim3((out + BJ_C - 1) / BJ_C), dim3(BJ_C * BJ_G), 0, st, ws, blocks, db, out);
  return hipGetLastError();
}

}  // namespace

// Blocks of rows: one for few rows, else enough workgroups to fill the chip several times, at
// least 16 rows each.
int act_backward_blocks(int64_t T, int64_t out) {
  if (T <= 64) return 1;  // no join: 34 x 6416 11.8 us against 16.4; at 128 rows 18 against 16
  const int64_t cols = (out + kAbCols<bf16_t> - 1) / kAbCols<bf16_t>;
  int64_t b = cols > 0 ? (2048 + cols - 1) / cols : 1;
  const int64_t most = (T + 15) / 16;
  if (b > most) b = most;
  if (b > 1024) b = 1024;
  if (b < 1) b = 1;
  // no empty block at the end: the last of ceil(T / rows_per) blocks holds a row
  const int64_t rows_per = T > 0 ? (T + b - 1) / b : 1;
  return (int)(T > 0 ? (T + rows_per - 1) / rows_per : 1);
}

hipError_t launch_act_backward(int bf16, int act, const void* dY, int64_t lddy, const void* Z, int64_t ldz, void* dZ,
                               int64_t lddz, float* db, float* ws, int T, int out, hipStream_t st) {
  return bf16 ? act_backward<bf16_t>(act, dY, lddy, Z, ldz, dZ, lddz, db, ws, T, out, st)
              : act_backward<float>(act, dY, lddy, Z, ldz, dZ, lddz, db, ws, T, out, st);
}

hipError_t launch_gated_backward(int bf16, const void* dH, int64_t lddh, const LinEpiArgs& e, int T, int hid,
                                 hipStream_t st) {
  const int64_t vecs = (int64_t)T * (hid / 4);
  if (vecs == 0) return hipSuccess;
  const int64_t want = (vecs + 255) / 256;
  const int grid = (int)(want < 4096 ? want : 4096);
  if (bf16)
    hipLaunchKernelGGL((gated_backward_kernel<bf16_t>), dim3(grid), dim3(256), 0, st, static_cast<const bf16_t*>(dH), lddh,
                       e, T, hid);
  else
    hipLaunchKernelGGL((gated_backward_kernel<float>), dim3(grid), dim3(256), 0, st, static_cast<const float*>(dH), lddh, e,
                       T, hid);
  return hipGetLastError();
}

hipError_t launch_acc_join(const LinArgs& g, hipStream_t st) {
  const int64_t want = ((int64_t)g.N * (g.M / 4) + 255) / 256;
  hipLaunchKernelGGL(acc_join_kernel, dim3((uint32_t)(want < 4096 ? want : 4096)), dim3(256), 0, st, g);
  return hipGetLastError();
}

int lse_join_groups(int64_t T) { return (int)((T + LJ_T - 1) / LJ_T); }

hipError_t launch_lse_join(const float* part, int64_t nblk, const float* tlogit, const int64_t* target, int64_t ignore,
                           int64_t vocab, float* loss, float* lse, float* total, double* tsum, int T, hipStream_t st) {
  const int groups = T > 0 ? lse_join_groups(T) : 1;  // no tokens: one group writes the empty total
  hipLaunchKernelGGL(lse_join_kernel, dim3(groups), dim3(256), 0, st, part, nblk, tlogit, target, ignore, vocab, loss, lse,
                     tsum, total, T);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || groups == 1) return e;
  hipLaunchKernelGGL(lse_total_kernel, dim3(1), dim3(256), 0, st, tsum, groups, total);
  return hipGetLastError();
}

}  // namespace forge
