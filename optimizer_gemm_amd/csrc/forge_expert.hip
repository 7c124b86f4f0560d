// The way of rows to their experts and back, and the quantisation of rows to 8 bits: passes without a
// product, all bound by memory or, for a few tokens, by the launch.
#include "forge_ops.h"

namespace forge {
namespace {

typedef uint16_t bf16_t;

// ---- plan: a stable counting sort of the routes by expert -------------------
// Routes are cut into blocks; a block counts its routes per expert (plan_count), and then, knowing the
// counts of all blocks, gives each of its routes its place: the experts' first rows, plus the routes of that expert in
// the blocks before, plus those before it in the block, which it takes NT at a time (a wave's equals by
// one ballot per bit of the expert's number). Counts are integers, so their order does not matter. One
// block needs no first launch, and takes 1024 routes at a time from 512 routes on. One block and blocks of 1024: 2048 routes to
// 8 experts 5.6 us and 7.1, to 1024 experts 7.3 and 11.1; 4000 to 8 8.1 and 7.3, to 300 10.3 and 9.3. One block of 1024
// lanes and of 256: 1000 routes to 64 experts 4.5 and 5.6; 300 to 64 4.4 and 4.0.
constexpr int PL_NT = 256, PL_BLOCK = 1024, PL_ONE_NT = 1024, PL_ONE = 2048;

// the route's expert, or `experts` for one that goes nowhere
__device__ __forceinline__ int route_key(const int64_t* idx, int64_t i, int64_t n, int experts) {
  if (i >= n) return experts;
  const int64_t x = idx[i];
  return x >= 0 && x < experts ? (int)x : experts;
}

template <int NT>
__device__ __forceinline__ void plan_histogram(int* hist, const int64_t* idx, int64_t i0, int64_t i1, int experts) {
  for (int e = threadIdx.x; e <= experts; e += NT) hist[e] = 0;
  __syncthreads();
  for (int64_t i = i0 + threadIdx.x; i < i1; i += NT) atomicAdd(&hist[route_key(idx, i, i1, experts)], 1);
  __syncthreads();
}

__global__ __launch_bounds__(PL_NT) void plan_count_kernel(const int64_t* idx, int64_t n, int64_t per, int experts,
                                                           int* counts) {
  __shared__ int hist[FORGE_MAX_EXPERTS + 1];
  const int64_t i0 = blockIdx.x * per, i1 = i0 + per < n ? i0 + per : n;
  plan_histogram<PL_NT>(hist, idx, i0, i1, experts);
  for (int e = threadIdx.x; e < experts; e += PL_NT) counts[(int64_t)blockIdx.x * experts + e] = hist[e];
}

template <int NT>
__global__ __launch_bounds__(NT) void plan_place_kernel(const int64_t* idx, int64_t n, int64_t per, int experts,
                                                        const int* counts, int64_t* offsets, int* pos) {
  constexpr int W = NT / 64;
  __shared__ int at[FORGE_MAX_EXPERTS + 1];       // next free row of each expert
  __shared__ int seen[W][FORGE_MAX_EXPERTS + 1];  // routes of a pass, per wave
  __shared__ int wave_sum[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t i0 = blockIdx.x * per, i1 = i0 + per < n ? i0 + per : n;
  if (gridDim.x == 1) plan_histogram<NT>(at, idx, i0, i1, experts);
  for (int e = tid; e < W * (FORGE_MAX_EXPERTS + 1); e += NT) (&seen[0][0])[e] = 0;
  // first rows: a running sum over the experts, NT at a time
  int before = 0;  // rows of the experts of earlier turns
  for (int e0 = 0; e0 < experts; e0 += NT) {
    const int e = e0 + tid;
    int all = 0, mine = 0;  // routes of the expert, and of those in blocks before this one
    if (e < experts) {
      if (gridDim.x == 1) {
        all = at[e];
      } else {
#pragma unroll 16
        for (int b = 0; b < (int)gridDim.x; ++b) {
          const int c = counts[(int64_t)b * experts + e];
          mine += b < (int)blockIdx.x ? c : 0;
          all += c;
        }
      }
    }
    int sum = all;
#pragma unroll
    for (int h = 1; h < 64; h <<= 1) {
      const int other = __shfl_up(sum, h);
      if (lane >= h) sum += other;
    }
    if (lane == 63) wave_sum[wave] = sum;
    __syncthreads();
    int first = before + sum - all;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < wave) first += wave_sum[w];
      before += wave_sum[w];
    }
    if (e < experts) {
      at[e] = first + mine;
      if (blockIdx.x == 0) {
        if (e == 0) offsets[0] = 0;
        offsets[e + 1] = first + all;
      }
    }
    __syncthreads();
  }
  const int bits = 32 - __builtin_clz(experts);
  for (int64_t p = i0; p < i1; p += NT) {
    const int64_t i = p + tid;
    const int key = route_key(idx, i, i1, experts);
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((key >> b) & 1);
      same &= (key >> b) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1ull));
    const bool leads = rank == 0;
    if (leads) seen[wave][key] = __popcll(same);
    __syncthreads();
    int row = at[key] + rank;
#pragma unroll
    for (int w = 0; w < W; ++w) row += w < wave ? seen[w][key] : 0;
    if (i < i1) pos[i] = key < experts ? row : -1;
    __syncthreads();
    if (leads) {
      atomicAdd(&at[key], seen[wave][key]);
      seen[wave][key] = 0;
    }
    __syncthreads();
  }
}

// ---- rows to their experts --------------------------------------------------
// LANES lanes hold a token's row, 16 bytes each, and write it to each of its places: a row is read once
// however many experts take it.
template <int LANES>
__global__ __launch_bounds__(256) void dispatch_kernel(const char* X, int64_t ldx, const int* pos, int k, int64_t T,
                                                       int64_t places, char* Y, int64_t ldy, int chunks,
                                                       const float* sx, float* sy) {
  const int64_t t = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  if (t >= T) return;
  const int l = threadIdx.x % LANES;
  const int* p = pos + t * k;
  for (int c0 = l; c0 < chunks; c0 += 4 * LANES) {
    u32x4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u * LANES;
      v[u] = *reinterpret_cast<const u32x4*>(X + t * ldx + (int64_t)(c < chunks ? c : c0) * 16);
    }
    for (int j = 0; j < k; ++j) {
      const int64_t row = p[j];
      if (row < 0 || row >= places) continue;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = c0 + u * LANES;
        if (c < chunks) *reinterpret_cast<u32x4*>(Y + row * ldy + (int64_t)c * 16) = v[u];
      }
    }
  }
  if (sx) {
    for (int j = l; j < k; j += LANES) {
      const int64_t row = p[j];
      if (row >= 0 && row < places) sy[row] = sx[t];
    }
  }
}

// ---- and back: Y[t] = sum_j w[t][j] Yp[pos[t][j]] + R[t] ----------------------
// P: the type of Yp, T: that of the tokens' side (float32 sums may go with bfloat16 tokens). A lane holds the 16 bytes
// of a P row at a time; the rows of up to eight routes are asked for before the first is used. Summed in float32 in
// the order of the routes. 8191 tokens of 8 routes, 2048 bfloat16 columns (302 MB), by itself on three sets of rows in
// turn: 58 us, 5.2 TB/s; right after its backward pass, whose results are still being written, 80 (both 178).
template <class T>
constexpr int kVec = 16 / (int)sizeof(T);

template <class T>
__device__ __forceinline__ void unpack(u32x4 r, float (&x)[kVec<T>]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = bits_f32(r[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bits_f32(r[i] << 16);
      x[2 * i + 1] = bits_f32(r[i] & 0xFFFF0000u);
    }
  }
}
// V neighbouring elements as floats
template <class T, int V>
__device__ __forceinline__ void get(const T* p, float (&x)[V]) {
  if constexpr (V * sizeof(T) == 16) {
    unpack<T>(*reinterpret_cast<const u32x4*>(p), x);
  } else {
    static_assert(V == 4, "8 bytes");
    const f32x4 y = load4(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = y[i];
  }
}
template <class T, int V>
__device__ __forceinline__ void put(T* p, const float (&x)[V]) {
  if constexpr (V * sizeof(T) == 16) {  // in one piece
    u32x4 r;
#pragma unroll
    for (int q = 0; q < V / 4; ++q)
      store4(reinterpret_cast<T*>(&r) + 4 * q, f32x4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]});
    *reinterpret_cast<u32x4*>(p) = r;
  } else {
    static_assert(V == 4, "8 bytes");
    store4(p, f32x4{x[0], x[1], x[2], x[3]});
  }
}

constexpr int CB_K = 8;  // routes at a time

template <class P, class T, int LANES>
__global__ __launch_bounds__(256) void combine_kernel(const P* Yp, int64_t ldp, int64_t places, const int* pos,
                                                      const float* w, int k, const T* R, int64_t ldr, T* Y, int64_t ldy,
                                                      int64_t tokens, int cols) {
  constexpr int V = kVec<P>;
  const int64_t t = (int64_t)blockIdx.x * (256 / LANES) + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / LANES);
  if (t >= tokens) return;
  const int l = threadIdx.x % LANES;
  // eight routes' rows (NULL: dropped or past the last one) and factors, the same for all lanes
  const P* row[CB_K];
  float f[CB_K];
  auto routes = [&](int j0) {
#pragma unroll
    for (int j = 0; j < CB_K; ++j) {
      const bool in = j0 + j < k;
      const int64_t r = in ? pos[t * k + j0 + j] : -1;
      row[j] = r >= 0 && r < places ? Yp + r * ldp : nullptr;
      f[j] = in && w ? w[t * k + j0 + j] : 1.f;
    }
  };
  routes(0);
  for (int c = l * V; c < cols; c += LANES * V) {
    float sum[V] = {};
    for (int j0 = 0; j0 < k; j0 += CB_K) {
      if (k > CB_K) routes(j0);
      u32x4 v[CB_K];
#pragma unroll
      for (int j = 0; j < CB_K; ++j)
        if (row[j]) v[j] = *reinterpret_cast<const u32x4*>(row[j] + c);
#pragma unroll
      for (int j = 0; j < CB_K; ++j) {
        if (row[j]) {
          float x[V];
          unpack<P>(v[j], x);
#pragma unroll
          for (int i = 0; i < V; ++i) sum[i] = fmaf(f[j], x[i], sum[i]);
        }
      }
    }
    if (R) {
      float x[V];
      get<T, V>(R + t * ldr + c, x);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += x[i];
    }
    put<T, V>(Y + t * ldy + c, sum);
  }
}

// ---- its backward pass: dYp[pos] = w dY[t], dw = <dY[t], Yp[pos]> -------------
// A token's lanes go over its row once for every eight routes; the products' sums are joined over the
// lanes, and over a workgroup's waves where it holds one token, in a fixed order.
template <class P, class T, int LANES>
__global__ __launch_bounds__(256) void combine_backward_kernel(const T* dY, int64_t lddy, const P* Yp, int64_t ldp,
                                                               int64_t places, const int* pos, const float* w, int k,
                                                               T* dYp, int64_t lddp, float* dw, int64_t tokens, int cols) {
  constexpr int V = kVec<P>;
  __shared__ float part[4][CB_K];
  const int64_t t = (int64_t)blockIdx.x * (256 / LANES) + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / LANES);
  if (t >= tokens) return;  // (a wave's or a workgroup's lanes hold one token: all of them leave)
  const int l = threadIdx.x % LANES;
  const int* p = pos + t * k;
  for (int j0 = 0; j0 < k; j0 += CB_K) {
    int64_t row[CB_K];
    float f[CB_K], dot[CB_K];
#pragma unroll
    for (int j = 0; j < CB_K; ++j) {
      row[j] = -1;
      f[j] = 1.f;
      dot[j] = 0.f;
      if (j0 + j < k) {
        const int64_t r = p[j0 + j];
        row[j] = r < places ? r : -1;
        if (w) f[j] = w[t * k + j0 + j];
      }
    }
    for (int c = l * V; c < cols; c += LANES * V) {
      float d[V];
      get<T, V>(dY + t * lddy + c, d);
      u32x4 v[CB_K];
      if (dw) {
#pragma unroll
        for (int j = 0; j < CB_K; ++j)
          if (row[j] >= 0) v[j] = *reinterpret_cast<const u32x4*>(Yp + row[j] * ldp + c);
      }
#pragma unroll
      for (int j = 0; j < CB_K; ++j) {
        if (row[j] < 0) continue;
        if (dw) {
          float x[V];
          unpack<P>(v[j], x);
#pragma unroll
          for (int i = 0; i < V; ++i) dot[j] = fmaf(d[i], x[i], dot[j]);
        }
        if (dYp) {
          float x[V];
#pragma unroll
          for (int i = 0; i < V; ++i) x[i] = f[j] * d[i];
          put<T, V>(dYp + row[j] * lddp + c, x);
        }
      }
    }
    if (!dw) continue;
#pragma unroll
    for (int j = 0; j < CB_K; ++j)
#pragma unroll
      for (int h = 32; h > 0; h >>= 1) dot[j] += __shfl_xor(dot[j], h);
    if constexpr (LANES == 64) {
#pragma unroll
      for (int j = 0; j < CB_K; ++j)
        if (l == j && j0 + j < k) dw[t * k + j0 + j] = row[j] >= 0 ? dot[j] : 0.f;
    } else {
      if ((l & 63) == 0) {
#pragma unroll
        for (int j = 0; j < CB_K; ++j) part[l >> 6][j] = dot[j];
      }
      __syncthreads();
      if (l < CB_K && j0 + l < k) {
        const int64_t r = p[j0 + l];
        dw[t * k + j0 + l] = r >= 0 && r < places ? (part[0][l] + part[1][l]) + (part[2][l] + part[3][l]) : 0.f;
      }
      __syncthreads();
    }
  }
}

// ---- rows to 8 bits -----------------------------------------------------------
// scale = max |x| / 127, code = x / scale to the nearest whole number (ties to even), both quotients as IEEE
// divides. A row of zeros has scale 0 and codes 0, one with an infinity or NaN scale NaN and codes 0, so that
// its products are NaN. LANES lanes hold a row, up to NV vectors each in registers: one pass over memory;
// a longer row's are read again.
template <class T, int LANES, int NV>
__global__ __launch_bounds__(256) void quantize_kernel(const T* X, int64_t ldx, int8_t* Q, int64_t ldq, float* scale,
                                                       int64_t rows, int cols) {
  constexpr int V = kVec<T>;
  __shared__ uint32_t top[4];
  const int64_t t = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  if (t >= rows) return;  // (a wave's or a workgroup's lanes hold one row: all of them leave)
  const int l = threadIdx.x % LANES;
  const T* x = X + t * ldx;
  u32x4 v[NV];
  // magnitudes compare as integers, infinities above all numbers and NaN above them
  uint32_t mx = 0;
  auto take = [&](u32x4 r) {
    float f[V];
    unpack<T>(r, f);
#pragma unroll
    for (int i = 0; i < V; ++i) mx = max(mx, f32_bits(f[i]) & 0x7FFFFFFFu);
  };
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int c = (u * LANES + l) * V;
    v[u] = c < cols ? *reinterpret_cast<const u32x4*>(x + c) : u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int u = 0; u < NV; ++u) take(v[u]);
  for (int c = (NV * LANES + l) * V; c < cols; c += LANES * V) take(*reinterpret_cast<const u32x4*>(x + c));
#pragma unroll
  for (int h = 32; h > 0; h >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, h));
  if constexpr (LANES == 256) {
    if ((l & 63) == 0) top[l >> 6] = mx;
    __syncthreads();
    mx = max(max(top[0], top[1]), max(top[2], top[3]));
  }
  const bool bad = mx >= 0x7F800000u;
  const float s = bits_f32(mx) / 127.f;
  const bool zero = bad || s == 0.f;
  if (l == 0) scale[t] = bad ? __builtin_nanf("") : s;
  auto codes = [&](u32x4 r, int c) {
    float f[V];
    unpack<T>(r, f);
    uint32_t q[V / 4];
#pragma unroll
    for (int w = 0; w < V / 4; ++w) {
      q[w] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = fminf(fmaxf(rintf(f[4 * w + i] / s), -127.f), 127.f);
        q[w] |= (zero ? 0u : (uint32_t)(int32_t)y & 0xFFu) << (8 * i);
      }
    }
    if constexpr (V == 8)
      *reinterpret_cast<u32x2*>(Q + t * ldq + c) = u32x2{q[0], q[1]};
    else
      *reinterpret_cast<uint32_t*>(Q + t * ldq + c) = q[0];
  };
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int c = (u * LANES + l) * V;
    if (c < cols) codes(v[u], c);
  }
  for (int c = (NV * LANES + l) * V; c < cols; c += LANES * V) codes(*reinterpret_cast<const u32x4*>(x + c), c);
}

// workgroups of 256 lanes for `rows` rows of `lanes` lanes each
uint32_t row_blocks(int64_t rows, int lanes) { return (uint32_t)((rows * lanes + 255) / 256); }
// Lanes of a row of so many 16-byte chunks: a wave's, or a workgroup's where a wave would go over it more than
// twice and either that often that its loads wait for one another (8191 tokens of 8 routes, 256 chunks:
// combination by itself 59 us against 74), or the rows alone do not fill the chip.
bool wide_rows(int64_t rows, int64_t chunks) { return chunks >= 256 || (chunks > 128 && rows < 4096); }
// Of a row to quantise, which a wave holds in registers up to 512 chunks of: a workgroup's from there on or for few rows
// (65528 rows of 256 chunks 78 us against 148).
bool wide_quant(int64_t rows, int64_t chunks) { return chunks > 512 || (chunks > 128 && rows < 4096); }

}  // namespace

int64_t expert_plan_blocks(int64_t n, int64_t* per) {
  // one block of up to PL_ONE routes; else blocks of PL_BLOCK, larger ones (whole turns of a workgroup) beyond 512 of them, since each block reads all
  // blocks' counts
  int64_t p = n <= PL_ONE ? PL_ONE : PL_BLOCK;
  if ((n + p - 1) / p > 512) p = ((n + 511) / 512 + PL_NT - 1) / PL_NT * PL_NT;
  *per = p;
  return n > 0 ? (n + p - 1) / p : 1;
}

hipError_t launch_expert_plan(const int64_t* idx, int64_t n, int experts, int64_t* offsets, int* pos, int* counts,
                              hipStream_t st) {
  int64_t per;
  const uint32_t blocks = (uint32_t)expert_plan_blocks(n, &per);
  if (blocks > 1) {
    hipLaunchKernelGGL(plan_count_kernel, dim3(blocks), dim3(PL_NT), 0, st, idx, n, per, experts, counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (blocks == 1 && n > 2 * PL_NT)
    hipLaunchKernelGGL((plan_place_kernel<PL_ONE_NT>), dim3(1), dim3(PL_ONE_NT), 0, st, idx, n, per, experts, counts, offsets, pos);
  else
    hipLaunchKernelGGL((plan_place_kernel<PL_NT>), dim3(blocks), dim3(PL_NT), 0, st, idx, n, per, experts, counts, offsets, pos);
  return hipGetLastError();
}

hipError_t launch_expert_dispatch(const void* X, int64_t ldx_bytes, const int* pos, int k, int64_t T, int64_t places,
                                  void* Y, int64_t ldy_bytes, int chunks, const float* sx, float* sy, hipStream_t st) {
  const char* x = static_cast<const char*>(X);
  char* y = static_cast<char*>(Y);
  if (wide_rows(T, chunks))
    hipLaunchKernelGGL((dispatch_kernel<256>), dim3(row_blocks(T, 256)), dim3(256), 0, st, x, ldx_bytes, pos, k, T, places, y,
                       ldy_bytes, chunks, sx, sy);
  else
    hipLaunchKernelGGL((dispatch_kernel<64>), dim3(row_blocks(T, 64)), dim3(256), 0, st, x, ldx_bytes, pos, k, T, places, y,
                       ldy_bytes, chunks, sx, sy);
  return hipGetLastError();
}

template <class P, class T>
static hipError_t combine(const CombineArgs& a, hipStream_t st) {
  auto go = [&](auto lanes_c) {
    constexpr int L = decltype(lanes_c)::value;
    hipLaunchKernelGGL((combine_kernel<P, T, L>), dim3(row_blocks(a.tokens, L)), dim3(256), 0, st,
                       static_cast<const P*>(a.Yp), a.ldp, a.places, a.pos, a.w, a.k, static_cast<const T*>(a.R), a.ldr,
                       static_cast<T*>(a.Y), a.ldy, a.tokens, a.cols);
  };
  if (wide_rows(a.tokens, a.cols / kVec<P>))
    go(std::integral_constant<int, 256>{});
  else
    go(std::integral_constant<int, 64>{});
  return hipGetLastError();
}
hipError_t launch_expert_combine(int bf16, int wide, const CombineArgs& a, hipStream_t st) {
  if (!bf16) return combine<float, float>(a, st);
  return wide ? combine<float, bf16_t>(a, st) : combine<bf16_t, bf16_t>(a, st);
}

template <class P, class T>
static hipError_t combine_backward(const CombineArgs& a, hipStream_t st) {
  auto go = [&](auto lanes_c) {
    constexpr int L = decltype(lanes_c)::value;
    hipLaunchKernelGGL((combine_backward_kernel<P, T, L>), dim3(row_blocks(a.tokens, L)), dim3(256), 0, st,
                       static_cast<const T*>(a.Y), a.ldy, static_cast<const P*>(a.Yp), a.ldp, a.places, a.pos, a.w, a.k,
                       static_cast<T*>(a.dYp), a.lddp, a.dw, a.tokens, a.cols);
  };
  if (wide_rows(a.tokens, a.cols / kVec<P>))
    go(std::integral_constant<int, 256>{});
  else
    go(std::integral_constant<int, 64>{});
  return hipGetLastError();
}
hipError_t launch_expert_combine_backward(int bf16, int wide, const CombineArgs& a, hipStream_t st) {
  if (!bf16) return combine_backward<float, float>(a, st);
  return wide ? combine_backward<float, bf16_t>(a, st) : combine_backward<bf16_t, bf16_t>(a, st);
}

template <class T>
static hipError_t quantize(const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* scale, int64_t rows, int cols,
                           hipStream_t st) {
  const int64_t chunks = cols / kVec<T>;
  const T* x = static_cast<const T*>(X);
  if (wide_quant(rows, chunks))
    hipLaunchKernelGGL((quantize_kernel<T, 256, 8>), dim3(row_blocks(rows, 256)), dim3(256), 0, st, x, ldx, Q, ldq, scale,
                       rows, cols);
  else
    hipLaunchKernelGGL((quantize_kernel<T, 64, 8>), dim3(row_blocks(rows, 64)), dim3(256), 0, st, x, ldx, Q, ldq, scale, rows,
                       cols);
  return hipGetLastError();
}
hipError_t launch_quantize_rows(int bf16, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* scale, int64_t rows,
                                int cols, hipStream_t st) {
  return bf16 ? quantize<bf16_t>(X, ldx, Q, ldq, scale, rows, cols, st) : quantize<float>(X, ldx, Q, ldq, scale, rows, cols, st);
}

}  // namespace forge
