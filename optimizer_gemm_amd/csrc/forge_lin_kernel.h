// Internal: products with an epilogue (forge_ops.h) on bfloat16 operands.
//
// C[m][n] = sum_k A[m][k] B[n][k], m along the output's columns. Either operand may have k
// as its fast index (rows of W in a forward product, rows of X or dY) or as its slow index
// (rows of W in an input gradient, rows of X and dY in a weight gradient).
//
// Mainloop. A group of 2 x 2 waves owns a B x B tile. Stages of 64 k go from global memory
// straight into LDS (buffer loads with the LDS bit, 1 KiB per wave instruction), one operand's
// stage to a slot, five slots in a ring: two and a half stages, all of the 160 KiB with 256x256
// tiles. 64 k make a k-fast row 128 bytes, one cache line: with 32 k per stage every line was
// requested twice (TCP_TCC_READ_REQ 117.8 M against 58.7 M on 8192 x 14336 -> 4096). k-fast rows
// are read with 16-byte LDS reads, k-slow rows with the LDS transpose read; XOR swizzles of the
// 16-byte chunks keep both free of bank conflicts. v_mfma_f32_16x16x32_bf16, FP32 sums: on
// normally distributed data the part holds a higher clock with it than with the 32x32x16 form
// (2071 against 1791 TFLOP/s from registers alone), which moves twice the accumulators per
// product; on constant data both reach 2430.
// A stage is two k-steps of 32 k. Each multiplies one fragment set while the next one is read
// between the first half of its products. One barrier per stage, between the two: by then every
// wave has read the whole stage and its own loads of the next one have landed but for one
// operand's, so the barrier publishes that stage and frees this one's slots. The loads of the
// stage after next are issued between the products of both k-steps.
// The 256x256 tile has one wave per SIMD of 128x128 (256 accumulators): each fragment byte read
// from LDS feeds twice the products of a 64-wide wave tile. The smaller tiles serve outputs of
// few tiles: 128x128 with two workgroups per compute unit; and with KS > 1 that many groups of
// waves, each with a ring of its own, share the tile's k range, whose chain of stages is what
// takes the time there (1 x 4096 -> 4096: 30 us -> 17 with four groups on 64x64 tiles).
// Several products may run into one accumulation (MULTI: their stages follow one another), and
// several workgroups may share one tile's k range (SPLIT, LinArgs::splits).
// Operands are addressed from the tile's own origin (64-bit base, 32-bit offsets), so a
// k-fast operand may be of any size; a k-slow one spans less than 2^31 bytes. A load whose
// row, column or k lies outside takes an offset past every extent and writes zeros.
//
// Epilogue. Vector epilogues hand each wave's accumulators through an LDS region of its own,
// 32 output rows x 64 columns at a time, so that whole row segments are read and written
// without a workgroup barrier; the cross entropy's maximum and sum are taken from the
// accumulators directly (a lane holds a quarter of a token's logits of the wave's tile). The
// 256x256 tile's regions are the fifth slot, so the next tile's first two stages are on their way
// during the epilogue. With KS > 1 the groups' sums are added in order in LDS.
//
// Measured (256x256 tiles): 8192 x 4096 -> 4096 204 us, 1350 TFLOP/s; 8192 x 14336 -> 4096 with
// residual 671 us, 1434; 8192 x 4096 -> 2 x 14336 gated, projections kept, 1.39 ms, 1384; a large
// library product of these shapes, without an epilogue, reaches 1295, 1598 and 1564. 1.33 to 1.4 us per stage and tile,
// of which the products with their LDS reads alone take 0.92; with loads that return zeros
// 1.06. The part's clock is what gives: 1.76 GHz at 72% busy matrix pipes.
#pragma once

#include "forge_gemm_kernel.h"
#include "forge_ops.h"

namespace forge {

// B x B tiles, OCC waves per SIMD, KS groups of 2 x 2 waves that share a tile's k range.
template <int B_, int OCC_, bool AHEAD_, int KS_ = 1>
struct LTile {
  static constexpr int BM = B_, BN = B_, BK = 64, WM = 2, WN = 2, OCC = OCC_, KS = KS_;
  // AHEAD: the epilogue's LDS is one slot, the next tile's first stages load beside it
  static constexpr bool AHEAD = AHEAD_;
  static constexpr int NW = WM * WN * KS, NT = 64 * NW, GT = 64 * WM * WN;  // GT: threads of a group
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  static constexpr int KST = BK / 32;  // k-steps per stage
  // LDS: five slots of one operand's stage per group. Stage s has A in slot 2s mod 5, B in slot
  // (2s + 1) mod 5: B of stage s + 2 takes the slot that A of stage s leaves, A of stage
  // s + 3 the one that B of stage s leaves.
  static constexpr int SLOT = B_ * BK * 2, PL = SLOT / 16 / GT;  // PL: loads per slot and wave
  // epilogue: KS = 1: 32 rows x 64 floats per wave; else the whole tile as rows of BM + 4 floats
  static constexpr int EPIW = 32 * 64 * 4, EPI0 = AHEAD ? 4 * SLOT : 0, LDE = BM + 4;
  static constexpr int SMEM = 5 * SLOT * KS;
  static_assert(SMEM * (OCC * 4 / NW) <= 160 * 1024, "LDS");
  static_assert(KS > 1 ? BN * LDE * 4 <= SMEM : (EPI0 + NW * EPIW <= SMEM && FM % 4 == 0 && FN % 2 == 0), "epilogue");
};

// Layout of one operand's stage in LDS: R output indexes x BK k.
template <class C, int R, bool TR>
struct LOper {
  static constexpr int ROWB = (TR ? R : C::BK) * 2;  // bytes per LDS row
  static constexpr int CPR = ROWB / 16;              // 16-byte chunks per row
  static constexpr int RSTEP = C::GT / CPR;          // rows between a thread's chunks
  // transpose reads: half a wave touches 32 bytes of 8 rows (r .. r + 3 and r + 8 .. r + 11), all
  // in different 32-byte bank groups; k-fast rows (two per 256-byte bank period): 16 consecutive
  // rows in all 16 chunk groups
  // (rows of 128 bytes, two per bank period, take the pairs of rows apart by the row's own bit)
  __host__ __device__ static constexpr int swz(int row) {
    return !TR ? (row >> 1) & 7 : (CPR >= 16 ? 4 * (row & 3) + 2 * ((row >> 3) & 1) : 4 * ((row >> 1) & 1) + 2 * ((row >> 3) & 1));
  }
  static_assert(C::GT % CPR == 0 && (TR ? RSTEP % 8 : RSTEP % 16) == 0, "rows of a thread's chunks");
  static_assert(TR ? CPR >= 8 : CPR == 8, "row length");
};

// 16 bytes per lane from buffer offset off + soff into LDS at dst + 16 * lane
__device__ __forceinline__ void dma16s(__amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t off, uint32_t soff) {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Wold-style-cast"
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, off, soff, 0, 0);
#pragma clang diagnostic pop
}

// c += a b in place, in accumulation registers. Written as assembly so that the sum keeps its
// registers: with all 256 of them in use the compiler gives the builtin's result others and
// moves the sums around. What the compiler's hazard checks would do is done at the uses: the
// operands come from LDS reads that have been waited for, a sum is used again 64 (16, 4) products
// later, and mfma_drain() stands between the last product and the first read of a sum.
__device__ __forceinline__ void mfma_acc(f32x4& c, bf16x8 a, bf16x8 b) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma_drain() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

// The kernel's argument where it lies (its only one, at the start of the argument segment): its
// arrays can be indexed there by a run-time number, which on the by-value copy would put that
// copy into scratch memory.
typedef const __attribute__((address_space(4))) LinArgs* LinArgsPtr;
__device__ __forceinline__ LinArgsPtr lin_args() { return (LinArgsPtr)__builtin_amdgcn_kernarg_segment_ptr(); }

// the kernel's lambdas hold references to register arrays: one that is called instead of
// inlined would put them into scratch memory
#define FORGE_INLINE __attribute__((always_inline))

template <class C, int EPI, bool TA, bool TB>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::OCC, C::OCC)))
void lin_kernel(LinArgs g) {
  using OA = LOper<C, C::BM, TA>;
  using OB = LOper<C, C::BN, TB>;
  constexpr bool TWO = EPI == L_GATED;              // A: BM / 2 rows of gate, then BM / 2 of up
  constexpr bool MULTI = EPI == L_ACC && TA && !TB;  // several operand pairs
  constexpr int OM = TWO ? C::BM / 2 : C::BM;        // output columns per tile
  constexpr int PA = C::PL, PB = C::PL;
  static_assert(!TWO || (!TA && PA % 2 == 0), "gate and up: k fast, half of the loads each");
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::SMEM];
  const int tid = C::KS > 1 ? static_cast<int>(threadIdx.x) % C::GT : static_cast<int>(threadIdx.x);
  // the wave in its group, the group (its share of the k range, its ring)
  const int wave_a = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int wave_u = C::KS > 1 ? wave_a % (C::WM * C::WN) : wave_a, grp = C::KS > 1 ? wave_a / (C::WM * C::WN) : 0;
  const int wm = wave_u % C::WM, wn = wave_u / C::WM;
  uint8_t* const ring = smem + grp * 5 * C::SLOT;
  const uint32_t lds0 = lds_addr(smem) + (uint32_t)(grp * 5 * C::SLOT);
  const int ntm = (epi_width<EPI>(g.M) - g.m_off + OM - 1) / OM, ntn = (g.N - g.n_off + C::BN - 1) / C::BN;
  const int ntiles = ntm * ntn * (EPI == L_ACC && TA && !TB ? g.splits : 1);
  const LinArgsPtr ga = lin_args();
  const int nsrc = MULTI ? ga->nsrc : 1;
  int nst = (g.K[0] + C::BK - 1) / C::BK;
  if constexpr (MULTI) {
    for (int s = 1; s < nsrc; ++s) nst += (ga->K[s] + C::BK - 1) / C::BK;
  }
  // SPLIT: g.splits workgroups share a tile's k range, each writing its part of the sums
  constexpr bool SPLIT = MULTI;
  const int splits = SPLIT ? g.splits : 1;
  const int mine = (nst + C::KS * splits - 1) / (C::KS * splits);  // stages of a group

  // ---- operand loads ----
  // The stage of each operand that is loaded next (the two are one stage apart): the pair it
  // belongs to, that pair's K, the stage's first k (past the end: k >= K, every load out of
  // range), bytes per k.
  int fa_K = 0, fa_k = 0, fa_src = 0, fb_K = 0, fb_k = 0, fb_src = 0;
  uint32_t fa_kb = 0, fb_kb = 0;
  __amdgpu_buffer_rsrc_t rA, rA2, rB;
  uint32_t av[PA], bv[PB];     // this thread's offsets in a stage
  int lm0 = 0, ln0 = 0, lsp = 0;  // the tile that is being loaded, its part of the k range
  // offsets of the loads from a panel whose first output index is the tile's (lim of them exist)
  auto ext = [&](bool tr, int64_t ld, int64_t lim, int64_t rows, int K) FORGE_INLINE -> uint32_t {
    if (K <= 0 || lim <= 0) return 0u;
    // a k-fast operand's rows of this tile, a k-slow one from this tile's columns on, in whole
    // 16-byte chunks (rows are padded to them)
    const int64_t n = tr ? (K - 1) * ld + (lim + 7) / 8 * 8 : ((lim < rows ? lim : rows) - 1) * ld + (K + 7) / 8 * 8;
    return (uint32_t)(n * 2);
  };
  auto source_a = [&](int s) FORGE_INLINE {
    const int64_t ld = (MULTI ? ga->lda[s] : g.lda[0]);
    const int lim = g.M - lm0;
    fa_src = s;
    fa_K = (MULTI ? ga->K[s] : g.K[0]);
    fa_k = 0;
    fa_kb = TA ? (uint32_t)(ld * 2) : 2u;
    rA = make_rsrc(static_cast<const char*>((MULTI ? ga->A[s] : g.A[0])) + (TA ? (int64_t)lm0 : (int64_t)lm0 * ld) * 2,
                   ext(TA, ld, lim, OM, fa_K));
    if constexpr (TWO)
      rA2 = make_rsrc(static_cast<const char*>(g.A[1]) + (int64_t)lm0 * g.lda[1] * 2,
                      ext(false, g.lda[1], lim, OM, fa_K));
    int t = tid;
    asm volatile("" : "+v"(t));
    const int row0 = t / OA::CPR;
#pragma unroll
    for (int j = 0; j < PA; ++j) {
      const bool second = TWO && j >= PA / 2;
      const int row = row0 + (second ? j - PA / 2 : j) * OA::RSTEP, ch = (t % OA::CPR) ^ OA::swz(row);
      const bool in = TA ? ch * 8 < lim : row < lim;
      av[j] = in ? (uint32_t)(row * (second ? g.lda[1] : ld) * 2 + ch * 16) : kOOB;
    }
  };
  auto source_b = [&](int s) FORGE_INLINE {
    const int64_t ld = (MULTI ? ga->ldb[s] : g.ldb[0]);
    const int lim = g.N - ln0;
    fb_src = s;
    fb_K = (MULTI ? ga->K[s] : g.K[0]);
    fb_k = 0;
    fb_kb = TB ? (uint32_t)(ld * 2) : 2u;
    rB = make_rsrc(static_cast<const char*>((MULTI ? ga->B[s] : g.B[0])) + (TB ? (int64_t)ln0 : (int64_t)ln0 * ld) * 2,
                   ext(TB, ld, lim, C::BN, fb_K));
    int t = tid;
    asm volatile("" : "+v"(t));
    const int row0 = t / OB::CPR;
#pragma unroll
    for (int j = 0; j < PB; ++j) {
      const int row = row0 + j * OB::RSTEP, ch = (t % OB::CPR) ^ OB::swz(row);
      const bool in = TB ? ch * 8 < lim : row < lim;
      bv[j] = in ? (uint32_t)(row * ld * 2 + ch * 16) : kOOB;
    }
  };
  // this thread's first k in a stage, per operand
  const int a_k = TA ? tid / OA::CPR : ((tid % OA::CPR) ^ OA::swz(tid / OA::CPR)) * 8;
  const int b_k = TB ? tid / OB::CPR : ((tid % OB::CPR) ^ OB::swz(tid / OB::CPR)) * 8;
  // the common part of a load's offset stays inside the extent, from which the range check
  // subtracts it; a stage past the end is marked by k >= K
  auto soff = [&](int k, int K, uint32_t kb) FORGE_INLINE -> uint32_t { return k < K ? (uint32_t)k * kb : 0u; };
  // the j-th load of an operand's next stage, into slot (0..4)
  auto dma_a = [&](int slot, auto j_c) FORGE_INLINE {
    constexpr int j = decltype(j_c)::value;
    uint8_t* dst = ring + slot * C::SLOT + j * C::GT * 16 + wave_u * 1024;
    const uint32_t off = fa_k + a_k + (TA ? j * OA::RSTEP : 0) < fa_K ? av[j] : kOOB;
    if constexpr (TWO && j >= PA / 2)
      dma16s(rA2, dst, off, soff(fa_k, fa_K, fa_kb));
    else
      dma16s(rA, dst, off, soff(fa_k, fa_K, fa_kb));
  };
  auto dma_b = [&](int slot, auto j_c) FORGE_INLINE {
    constexpr int j = decltype(j_c)::value;
    uint8_t* dst = ring + slot * C::SLOT + j * C::GT * 16 + wave_u * 1024;
    const uint32_t off = fb_k + b_k + (TB ? j * OB::RSTEP : 0) < fb_K ? bv[j] : kOOB;
    dma16s(rB, dst, off, soff(fb_k, fb_K, fb_kb));
  };
  auto next_a = [&]() FORGE_INLINE {
    fa_k += C::BK;
    if constexpr (MULTI) {
      if (fa_k >= fa_K && fa_src + 1 < nsrc) source_a(fa_src + 1);
    }
  };
  auto next_b = [&]() FORGE_INLINE {
    fb_k += C::BK;
    if constexpr (MULTI) {
      if (fb_k >= fb_K && fb_src + 1 < nsrc) source_b(fb_src + 1);
    }
  };
  using N0 = std::integral_constant<int, 0>;
  // stages 0 and 1 of a tile, into slots 0..3
  auto dma_begin = [&](int tile) FORGE_INLINE {
    int tm, tn, part = 0;
    if constexpr (SPLIT) {
      part = tile % splits;
      tile /= splits;
    }
    g_tile(tile, ntm, ntn, tm, tn);
    lsp = part;
    lm0 = g.m_off + tm * OM;
    ln0 = g.n_off + tn * C::BN;
    int src0 = 0, k0 = (part * C::KS + grp) * mine * C::BK;  // the group's first stage: its pair and k
    if constexpr (MULTI) {
      while (src0 + 1 < nsrc && k0 >= (ga->K[src0] + C::BK - 1) / C::BK * C::BK) {
        k0 -= (ga->K[src0] + C::BK - 1) / C::BK * C::BK;
        ++src0;
      }
    }
    source_a(src0);
    source_b(src0);
    fa_k = k0;
    fb_k = k0;
    static_for<0, 2>([&](auto s_c) FORGE_INLINE {
      constexpr int s = decltype(s_c)::value;
      static_for<0, PA>([&](auto j_c) FORGE_INLINE { dma_a(2 * s, j_c); });
      static_for<0, PB>([&](auto j_c) FORGE_INLINE { dma_b(2 * s + 1, j_c); });
      next_a();
      next_b();
    });
  };

  // ---- fragment addresses (in the slots that are being read; at first 0 and 1) ----
  // Operand lane of v_mfma_f32_16x16x32: output index l mod 16, k = 8 (l / 16) .. + 7.
  // k fast: one 16-byte read. k slow, transpose read: lane (q, r4, c4) = (l / 16, l mod 16 / 4,
  // l mod 4) reads row 8 q + r4, elements 4 c4 .. + 3 of the 16-wide fragment and receives 4 k of
  // output index l mod 16; a second read 4 rows on gives the other 4.
  const int lane = tid & 63, q16 = lane >> 4, l16 = lane & 15;
  auto tr_addr = [&](int base, int rowb, int swz, int col0) FORGE_INLINE -> uint32_t {
    const int row = 8 * q16 + (l16 >> 2), chunk = col0 / 8 + ((lane & 3) >> 1);
    return lds0 + (uint32_t)(base + row * rowb + 16 * (chunk ^ swz) + 8 * (lane & 1));
  };
  const int tr_row = 8 * q16 + (l16 >> 2);
  const int a_r0 = TWO ? wm * (C::TM / 2) : wm * C::TM, b_r0 = wn * C::TN;
  // k fast: one per k-step. k slow: one per fragment (the swizzle takes the column's bits); the
  // second read's row differs in bit 2, which the swizzle does not see.
  constexpr int NAA = TA ? C::FM : C::KST, NBA = TB ? C::FN : C::KST;
  uint32_t a_ad[NAA], b_ad[NBA];
  if constexpr (TA) {
#pragma unroll
    for (int f = 0; f < C::FM; ++f) a_ad[f] = tr_addr(0, OA::ROWB, OA::swz(tr_row), a_r0 + 16 * f);
  } else {
#pragma unroll
    for (int kk = 0; kk < C::KST; ++kk)
      a_ad[kk] = lds0 + (uint32_t)((a_r0 + l16) * OA::ROWB + 16 * ((4 * kk + q16) ^ OA::swz(l16)));
  }
  if constexpr (TB) {
#pragma unroll
    for (int f = 0; f < C::FN; ++f) b_ad[f] = tr_addr(C::SLOT, OB::ROWB, OB::swz(tr_row), b_r0 + 16 * f);
  } else {
#pragma unroll
    for (int kk = 0; kk < C::KST; ++kk)
      b_ad[kk] = lds0 + (uint32_t)(C::SLOT + (b_r0 + l16) * OB::ROWB + 16 * ((4 * kk + q16) ^ OB::swz(l16)));
  }
  // One k-step's fragments: per 16 output indexes one 16-byte read (k fast) or two 8-byte reads
  struct Frag {
    u32x4 ak[TA ? 1 : C::FM];
    u32x2 at[TA ? C::FM : 1][2];
    u32x4 bk[TB ? 1 : C::FN];
    u32x2 bt[TB ? C::FN : 1][2];
  };
  constexpr int NRA = TA ? 2 * C::FM : C::FM, NRB = TB ? 2 * C::FN : C::FN, NR = NRA + NRB;
  auto read_one = [&](Frag& F, auto kk_c, auto r_c) FORGE_INLINE {
    constexpr int kk = decltype(kk_c)::value, r = decltype(r_c)::value;
    if constexpr (r < NRA) {
      if constexpr (TA) {
        F.at[r / 2][r % 2] = ds_tr_asm<(kk * 32 + (r % 2) * 4) * OA::ROWB>(a_ad[r / 2]);
      } else {
        constexpr int half = C::FM / 2;
        constexpr int row = !TWO ? 16 * r : (r < half ? 16 * r : C::BM / 2 + 16 * (r - half));
        F.ak[r] = ds_b128_asm<row * OA::ROWB>(a_ad[kk]);
      }
    } else {
      constexpr int q = r - NRA;
      if constexpr (TB)
        F.bt[q / 2][q % 2] = ds_tr_asm<(kk * 32 + (q % 2) * 4) * OB::ROWB>(b_ad[q / 2]);
      else
        F.bk[q] = ds_b128_asm<16 * q * OB::ROWB>(b_ad[kk]);
    }
  };
  // orders every later use of F's registers after the wait that precedes this
  auto settle = [&](Frag& F) FORGE_INLINE {
    if constexpr (TA) {
#pragma unroll
      for (int f = 0; f < C::FM; ++f) {
        pin_reg(F.at[f][0]);
        pin_reg(F.at[f][1]);
      }
    } else {
#pragma unroll
      for (int f = 0; f < C::FM; ++f) pin_reg(F.ak[f]);
    }
    if constexpr (TB) {
#pragma unroll
      for (int f = 0; f < C::FN; ++f) {
        pin_reg(F.bt[f][0]);
        pin_reg(F.bt[f][1]);
      }
    } else {
#pragma unroll
      for (int f = 0; f < C::FN; ++f) pin_reg(F.bk[f]);
    }
  };

  // stores of an epilogue that follow the next tile's first loads, at least
  constexpr int WAIT0 = C::AHEAD && EPI != L_LSE ? C::FN / 2 * (C::FM / 4) * (32 * ((TWO ? 32 : 64) / 8) / 64) : 0;
  static_assert(WAIT0 <= 63, "vmcnt range");
  if (blockIdx.x < ntiles) dma_begin(blockIdx.x);
  for (int tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {
    const int m0 = lm0, n0 = ln0, part = lsp;
    f32x4 acc[C::FM][C::FN];
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[fm][fn][e] = 0.f;
    auto mfma_one = [&](const Frag& F, auto i_c) FORGE_INLINE {
      constexpr int fm = decltype(i_c)::value / C::FN, fn = decltype(i_c)::value % C::FN;
      bf16x8 a, b;
      if constexpr (TA)
        a = __builtin_bit_cast(bf16x8, u32x4{F.at[fm][0].x, F.at[fm][0].y, F.at[fm][1].x, F.at[fm][1].y});
      else
        a = __builtin_bit_cast(bf16x8, F.ak[fm]);
      if constexpr (TB)
        b = __builtin_bit_cast(bf16x8, u32x4{F.bt[fn][0].x, F.bt[fn][0].y, F.bt[fn][1].x, F.bt[fn][1].y});
      else
        b = __builtin_bit_cast(bf16x8, F.bk[fn]);
      mfma_acc(acc[fm][fn], a, b);
    };
    // the MFMAs of F; the reads of G (k-step kk of the slots the addresses point to) and the loads
    // of an operand's stage spread over the first half of them; sched_barrier keeps the order
    constexpr int NM = C::FM * C::FN, LW = 2;  // (the loads: over the first 1 / LW)
    auto step = [&](const Frag& F, Frag& G, auto kk_c, auto&& load) FORGE_INLINE {
      static_for<0, NM>([&](auto i_c) FORGE_INLINE {
        constexpr int i = decltype(i_c)::value;
        mfma_one(F, i_c);
        constexpr int R0 = 2 * i * NR / NM < NR ? 2 * i * NR / NM : NR;
        constexpr int R1 = 2 * (i + 1) * NR / NM < NR ? 2 * (i + 1) * NR / NM : NR;
        static_for<R0, R1>([&](auto r_c) FORGE_INLINE { read_one(G, kk_c, r_c); });
        constexpr int L0 = LW * i * PA / NM < PA ? LW * i * PA / NM : PA;
        constexpr int L1 = LW * (i + 1) * PA / NM < PA ? LW * (i + 1) * PA / NM : PA;
        static_for<L0, L1>([&](auto l_c) FORGE_INLINE { load(l_c); });
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    Frag F0, F1;
    // stages 0 and 1 have landed, for every wave, and the epilogue's slot is free; the last
    // WAIT0 operations, stores of the epilogue, may still be on their way
    if (tile == (int)blockIdx.x)
      vm_wait_barrier<0>();
    else
      vm_wait_barrier<WAIT0>();
    static_for<0, NR>([&](auto r_c) FORGE_INLINE { read_one(F0, N0{}, r_c); });
    int sa = 0, sb = 1, pb_slot = 4;  // slots of A and B of the stage being multiplied, of B of the one before
    auto hop = [&](auto to_first) FORGE_INLINE {   // the addresses to the next stage's slots, or back to 0 and 1
      const int na = decltype(to_first)::value ? 0 : (sa + 2 >= 5 ? sa - 3 : sa + 2);
      const int nb = decltype(to_first)::value ? 1 : (sb + 2 >= 5 ? sb - 3 : sb + 2);
      const uint32_t da = (uint32_t)((na - sa) * C::SLOT), db = (uint32_t)((nb - sb) * C::SLOT);
#pragma unroll
      for (int j = 0; j < NAA; ++j) a_ad[j] += da;
#pragma unroll
      for (int j = 0; j < NBA; ++j) b_ad[j] += db;
      sa = na;
      sb = nb;
    };
    // Stage s, two k-steps: A of stage s + 2 is loaded over the first (into the slot that B of
    // stage s - 1 left); after the barrier B of stage s + 2 over the second (into the slot of A of
    // stage s). One body for every stage: the accumulators fill half of the register file,
    // and a second copy of their MFMAs on another path makes the compiler move them through
    // memory; the stages past the last one are loaded too, as zeros.
#pragma unroll 1
    for (int s = 0; s < mine; ++s) {
      const int slot_a2 = pb_slot, slot_b2 = sa;
      pb_slot = sb;
      lgkm_wait<0>();
      settle(F0);
      step(F0, F1, std::integral_constant<int, 1>{}, [&](auto j_c) FORGE_INLINE { dma_a(slot_a2, j_c); });
      next_a();
      hop(std::false_type{});
      // this wave has read the whole stage; of its loads only A of stage s + 2 may still be on
      // its way
      vm_wait_barrier<PA>();
      settle(F1);
      step(F1, F0, N0{}, [&](auto j_c) FORGE_INLINE { dma_b(slot_b2, j_c); });
      next_b();
    }
    mfma_drain();
    __builtin_amdgcn_sched_barrier(0);  // (no read of a sum moves in front of it)
    hop(std::true_type{});
    // the last k-step read fragments that nothing consumes: their registers stay pinned until
    // those reads have landed; and the zeros of the stages past the end
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    settle(F0);
    // Every wave passed the last stage's barrier (or, with no stage, the first one), so no slot is
    // read any more, and of each slot the pieces that this wave's own loads write are free: those
    // loads have landed. The next tile's first stages go there before this tile's epilogue (whose
    // first inputs are asked for before them: loads return in order).
    auto next_tile = [&]() FORGE_INLINE {
      if constexpr (C::AHEAD) {
        if (tile + (int)gridDim.x < ntiles) dma_begin(tile + gridDim.x);
      }
    };

    // ---- epilogue ----
    int etid = static_cast<int>(threadIdx.x);
    asm volatile("" : "+v"(etid));
    const int e_lane = etid & 63, e_q = e_lane >> 4, e_l16 = e_lane & 15;
    if constexpr (C::KS > 1) {
      // the groups' partial tiles are summed in order in LDS, as rows of the output
      float* E = reinterpret_cast<float*>(smem);
      const int t = static_cast<int>(threadIdx.x);
      __syncthreads();
#pragma unroll 1
      for (int kg = 0; kg < C::KS; ++kg) {
        if (grp == kg) {
#pragma unroll
          for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
            for (int fm = 0; fm < C::FM; ++fm) {
              const int col = !TWO ? wm * C::TM + 16 * fm
                                   : (fm < C::FM / 2 ? 0 : C::BM / 2 - C::TM / 2) + wm * (C::TM / 2) + 16 * fm;
              f32x4* p = reinterpret_cast<f32x4*>(E + (wn * C::TN + 16 * fn + e_l16) * C::LDE + col + 4 * e_q);
              *p = kg == 0 ? acc[fm][fn] : *p + acc[fm][fn];
            }
        }
        __syncthreads();
      }
      if constexpr (EPI == L_LSE) {
        // NT / BN threads per token, each a stretch of its logits
        constexpr int TP = C::NT / C::BN, W = C::BM / TP;
        const int n = n0 + t / TP, c0 = (t % TP) * W;
        const float* row = E + (t / TP) * C::LDE + c0;
        const int left = g.M - m0 - c0;
        float mx = -__builtin_huge_valf(), sum = 0.f;
        for (int j = 0; j < W; ++j)
          if (j < left) mx = fmaxf(mx, row[j]);
#pragma unroll
        for (int h = 1; h < TP; h <<= 1) mx = fmaxf(mx, __shfl_xor(mx, h));
        const float ref = mx > -__builtin_huge_valf() ? mx : 0.f;
        for (int j = 0; j < W; ++j)
          if (j < left) sum += __expf(row[j] - ref);
#pragma unroll
        for (int h = 1; h < TP; h <<= 1) sum += __shfl_xor(sum, h);
        if (n < g.N) {
          const int64_t y = g.e.target[n], d = y - (m0 + c0);
          if (y >= 0 && d >= 0 && d < W && d < left) g.e.tlogit[n] = row[d];
          if (t % TP == 0)
            *reinterpret_cast<float2*>(g.e.part + ((int64_t)(m0 / C::BM) * g.e.part_ld + n) * 2) = float2{mx, sum};
        }
      } else {
        const float sc = (EPI == L_ACC || EPI == L_DLOGIT) ? epi_scale(g.e) : 1.f;
        const int Mw = epi_width<EPI>(g.M);
        act_dispatch<EPI>(g.e.act, [&](auto act_c) {
          for (int v = t; v < C::BN * OM / 4; v += C::NT) {
            const int row = v / (OM / 4), col = (v % (OM / 4)) * 4, n = n0 + row, m = m0 + col;
            if (n < g.N && m < Mw) {
              const f32x4 x = *reinterpret_cast<const f32x4*>(E + row * C::LDE + col);
              f32x4 x2 = x;
              if constexpr (TWO) x2 = *reinterpret_cast<const f32x4*>(E + row * C::LDE + C::BM / 2 + col);
              epi_vec<uint16_t, EPI, decltype(act_c)::value>(g.e, n, m, g.M, x, x2, sc,
                                                             SPLIT ? (int64_t)part * g.N * g.e.ldacc : 0);
            }
          }
        });
      }
    } else if constexpr (EPI == L_LSE) {
      next_tile();
      // lane (q, l16): logits m = 16 fm + 4 q + j of token n = l16
      const int mb = m0 + wm * C::TM;
      const int left = g.M - mb;  // entries inside the vocabulary
      // a lane's own maximum and sum per token first (no lane waits for another), then the four
      // lanes of a token joined, all the tokens' exchanges in flight together
      float mx[C::FN], sum[C::FN];
      auto own = [&](auto tail_c) FORGE_INLINE {
        static_for<0, C::FN>([&](auto f_c) FORGE_INLINE {
          constexpr int f = decltype(f_c)::value;
          float x[C::FM * 4], m = -__builtin_huge_valf(), t = 0.f;
          int room = left - 4 * e_q;
          if constexpr (decltype(tail_c)::value) asm volatile("" : "+v"(room));  // (compared anew for each f)
#pragma unroll
          for (int i = 0; i < C::FM * 4; ++i) {
            x[i] = acc[i / 4][f][i % 4];
            // the last block: entries past the vocabulary count nothing
            if constexpr (decltype(tail_c)::value) x[i] = 16 * (i / 4) + i % 4 < room ? x[i] : -__builtin_huge_valf();
            m = fmaxf(m, x[i]);
          }
          const float ref = m > -__builtin_huge_valf() ? m : 0.f;
#pragma unroll
          for (int i = 0; i < C::FM * 4; ++i) t += __expf(x[i] - ref);
          mx[f] = m;
          sum[f] = t;
          __builtin_amdgcn_sched_barrier(0);  // (bounds the registers in use at once)
        });
      };
      if (left < C::TM)
        own(std::true_type{});
      else
        own(std::false_type{});
      static_for<0, C::FN>([&](auto f_c) FORGE_INLINE {
        constexpr int f = decltype(f_c)::value;
        float m = fmaxf(mx[f], __shfl_xor(mx[f], 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const float ref = m > -__builtin_huge_valf() ? m : 0.f;
        // (a lane without a finite logit has sum 0, or NaN, which stays)
        float t = sum[f] * __expf((mx[f] > -__builtin_huge_valf() ? mx[f] : ref) - ref);
        t += __shfl_xor(t, 16);
        t += __shfl_xor(t, 32);
        mx[f] = m;
        sum[f] = t;
        if constexpr (f % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      });
#pragma unroll
      for (int fn = 0; fn < C::FN; ++fn) {
        const int n = n0 + wn * C::TN + 16 * fn + e_l16;
        if (n < g.N && e_q == 0 && left > 0)
          *reinterpret_cast<float2*>(g.e.part + ((int64_t)(mb / C::TM) * g.e.part_ld + n) * 2) = float2{mx[fn], sum[fn]};
      }
      // the targets' logits: few tokens have theirs in this block
      static_for<0, C::FN>([&](auto f_c) FORGE_INLINE {
        constexpr int f = decltype(f_c)::value;
        const int n = n0 + wn * C::TN + 16 * f + e_l16;
        const int64_t y = n < g.N ? g.e.target[n] : -1, d = y - mb;
        const int at = (y >= 0 && d >= 0 && d < C::TM && d < left && ((d >> 2) & 3) == e_q) ? (int)d - 4 * e_q : -1;
        if (__any(at >= 0)) {
          float tl = 0.f;
#pragma unroll
          for (int i = 0; i < C::FM * 4; ++i) tl = at == 16 * (i / 4) + i % 4 ? acc[i / 4][f][i % 4] : tl;
          if (at >= 0) g.e.tlogit[n] = tl;
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    } else {
      const float sc = (EPI == L_ACC || EPI == L_DLOGIT) ? epi_scale(g.e) : 1.f;
      const LinEpiArgs& e = g.e;
      float* const e_acc = e.acc + (SPLIT ? (int64_t)part * g.N * e.ldacc : 0);
      const int Mw = epi_width<EPI>(g.M);
      // blocks of 32 output rows x 64 floats of C (32 columns of gate and of up)
      constexpr int CH = C::FM / 4, OWB = TWO ? 32 : 64, NB = C::FN / 2 * CH;
      constexpr int VPR = OWB / 8, NV = 32 * VPR / 64;  // 8-vectors per row, per lane and block
      // This wave's region: four rows in each KiB that its own loads write in a slot. Another
      // wave's loads of the stages past the end may still be on their way into theirs.
      static_assert(C::EPIW == C::NW * 2048 && C::NW * 1024 == C::GT * 16, "the wave's pieces of a slot");
      float* Ew = reinterpret_cast<float*>(smem + C::EPI0) + wave_u * 256;
      auto e_at = [&](int row) FORGE_INLINE { return (row >> 2) * (C::GT * 4) + (row & 3) * 64; };
      const int mw = m0 + wm * (TWO ? C::TM / 2 : C::TM), nw = n0 + wn * C::TN;
      // vector k of this lane in a block: row e_row + k * (64 / VPR), columns 8 e_col ..
      const int e_row = e_lane / VPR, e_col = e_lane % VPR;
      constexpr int RS = 64 / VPR;
      // what the epilogue reads and writes, from this wave's first row on
      const int rows = g.N - nw < C::TN ? g.N - nw : C::TN;
      auto res = [&](const void* p, int64_t ld, int es) FORGE_INLINE -> __amdgpu_buffer_rsrc_t {
        return make_rsrc(static_cast<const char*>(p) + (int64_t)nw * ld * es,
                         rows > 0 ? (uint32_t)(((int64_t)(rows - 1) * ld + Mw) * es) : 0u);
      };
      // byte offsets of this lane's vectors of block blk in a matrix of pitch ld
      auto offs = [&](int blk, int64_t ld, int es, uint32_t (&o)[NV]) FORGE_INLINE {
        const int n = 32 * (blk / CH) + e_row, m = mw + OWB * (blk % CH) + 8 * e_col;
        const bool okm = blk < NB && m < Mw;
        const uint32_t base = (uint32_t)n * (uint32_t)(ld * es) + (uint32_t)(m * es), step = (uint32_t)(RS * ld * es);
#pragma unroll
        for (int k = 0; k < NV; ++k) o[k] = okm && n + k * RS < rows ? base + k * step : kOOB;
      };
      // The inputs of a block; with one wave per SIMD, which has no other to wait behind, they are
      // loaded two blocks ahead.
      struct Pre {
        u32x4 a[NV], b[NV];
      };
      auto get = [&](u32x4 (&x)[NV], const void* p, int64_t ld, int es, int at, int blk) FORGE_INLINE {
        uint32_t o[NV];
        offs(blk, ld, es, o);
        const __amdgpu_buffer_rsrc_t r = res(p, ld, es);
#pragma unroll
        for (int k = 0; k < NV; ++k) x[k] = __builtin_amdgcn_raw_buffer_load_b128(r, o[k], at, 0);
      };
      auto load = [&](Pre& P, int blk) FORGE_INLINE {
        if constexpr (EPI == L_LINEAR) {
          if (e.in1) get(P.a, e.in1, e.ld1, 2, 0, blk);
        } else if constexpr (EPI == L_DGATE) {
          get(P.a, e.in1, e.ld1, 2, 0, blk);
          get(P.b, e.in2, e.ld2, 2, 0, blk);
        } else if constexpr (EPI == L_ACC) {
          if (e.acc_read) {
            get(P.a, e_acc, e.ldacc, 4, 0, blk);
            get(P.b, e_acc, e.ldacc, 4, 16, blk);
          }
        } else if constexpr (EPI == L_DLOGIT) {
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            // the row's target and log sum (rows past the end: the last row's)
            const int n0k = nw + 32 * (blk / CH) + e_row + k * RS, n = n0k < g.N ? n0k : g.N - 1;
            const u32x2 y = __builtin_bit_cast(u32x2, e.target[n]);
            P.a[k] = u32x4{y.x, y.y, f32_bits(e.lse[n]), e.weight ? f32_bits(e.weight[n]) : f32_bits(1.f)};
          }
        }
      };
      auto lo4 = [](u32x4 r) -> f32x4 {
        return f32x4{bits_f32(r.x << 16), bits_f32(r.x & 0xFFFF0000u), bits_f32(r.y << 16), bits_f32(r.y & 0xFFFF0000u)};
      };
      auto hi4 = [](u32x4 r) -> f32x4 {
        return f32x4{bits_f32(r.z << 16), bits_f32(r.z & 0xFFFF0000u), bits_f32(r.w << 16), bits_f32(r.w & 0xFFFF0000u)};
      };
      // 8 elements, rounded to nearest-even (v_cvt_pk_bf16_f32)
      auto pack = [&](f32x4 y, f32x4 z) FORGE_INLINE -> u32x4 {
        const u32x2 p = __builtin_bit_cast(u32x2, __builtin_convertvector(y, bf16x4));
        const u32x2 q = __builtin_bit_cast(u32x2, __builtin_convertvector(z, bf16x4));
        return u32x4{p.x, p.y, q.x, q.y};
      };
      auto put = [&](const u32x4 (&x)[NV], void* p, int64_t ld, int es, int at, int blk) FORGE_INLINE {
        uint32_t o[NV];
        offs(blk, ld, es, o);
        const __amdgpu_buffer_rsrc_t r = res(p, ld, es);
#pragma unroll
        for (int k = 0; k < NV; ++k) __builtin_amdgcn_raw_buffer_store_b128(x[k], r, o[k], at, 0);
      };
      auto process = [&](const Pre& P, int blk) FORGE_INLINE {
        // 16-byte chunk c of row r sits at chunk c ^ (r mod 16)
        static_for<0, NB>([&](auto b_c) FORGE_INLINE {
          constexpr int f = decltype(b_c)::value / CH, c = decltype(b_c)::value % CH;
          if (decltype(b_c)::value == blk) {
            static_for<0, 8>([&](auto h_c) FORGE_INLINE {
              constexpr int h = decltype(h_c)::value, fn = 2 * f + h / 4, i = h % 4;
              constexpr int fm = !TWO ? 4 * c + i : (i < 2 ? 2 * c + i : C::FM / 2 + 2 * c + i - 2);
              *reinterpret_cast<f32x4*>(Ew + e_at(16 * (h / 4) + e_l16) + ((4 * i + e_q) ^ e_l16) * 4) = acc[fm][fn];
            });
            // keeps the branches apart: merged, they would index the accumulators at run time,
            // which puts them into scratch memory
            asm volatile("" ::"i"(decltype(b_c)::value));
          }
        });
        const int m = mw + OWB * (blk % CH) + 8 * e_col;
        f32x4 bias0{0.f, 0.f, 0.f, 0.f}, bias1 = bias0;
        if constexpr (EPI == L_LINEAR) {
          if (e.bias) {
            const int mc = m < g.M ? m : 0;
            if (e.bias_f32) {
              bias0 = load4(static_cast<const float*>(e.bias) + mc);
              bias1 = load4(static_cast<const float*>(e.bias) + mc + 4);
            } else {
              bias0 = load4(static_cast<const uint16_t*>(e.bias) + mc);
              bias1 = load4(static_cast<const uint16_t*>(e.bias) + mc + 4);
            }
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        u32x4 r0[NV], r1[NV], r2[NV];
        // vector k of the block, and of the second product
        auto chunk = [&](int k, int c) FORGE_INLINE -> f32x4 {
          const int row = e_row + k * RS;
          return *reinterpret_cast<const f32x4*>(Ew + e_at(row) + (c ^ (row & 15)) * 4);
        };
        if constexpr (EPI == L_ACC) {
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            f32x4 x0 = chunk(k, 2 * e_col), x1 = chunk(k, 2 * e_col + 1);
            if (e.acc_read) {
              x0 = x0 + __builtin_bit_cast(f32x4, P.a[k]);
              x1 = x1 + __builtin_bit_cast(f32x4, P.b[k]);
            }
            r0[k] = __builtin_bit_cast(u32x4, x0);
            r1[k] = __builtin_bit_cast(u32x4, x1);
            r2[k] = pack(x0 * sc, x1 * sc);
          }
          if (e.acc_write) {
            put(r0, e_acc, e.ldacc, 4, 0, blk);
            put(r1, e_acc, e.ldacc, 4, 16, blk);
          } else {
            put(r2, e.out, e.ldo, 2, 0, blk);
          }
        } else if constexpr (EPI == L_DLOGIT) {
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            int hit;
            float w;
            bool ignored;
            dlogit_row(e, __builtin_bit_cast(int64_t, u32x2{P.a[k].x, P.a[k].y}), bits_f32(P.a[k].w), sc, hit, w, ignored);
            const float l = bits_f32(P.a[k].z);
            r0[k] = pack(dlogit(chunk(k, 2 * e_col), m, g.M, hit, l, w, ignored),
                         dlogit(chunk(k, 2 * e_col + 1), m + 4, g.M, hit, l, w, ignored));
          }
          put(r0, e.out, e.ldo, 2, 0, blk);
        } else {
          // one branch per block on the activation: with one wave per SIMD a branch per element
          // costs more than the arithmetic
          auto math = [&](auto act_c) FORGE_INLINE {
            constexpr int act = decltype(act_c)::value;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
              const f32x4 zero{0.f, 0.f, 0.f, 0.f};
              f32x4 x0 = chunk(k, 2 * e_col), x1 = chunk(k, 2 * e_col + 1), z0 = zero, z1 = zero, a0 = zero, a1 = zero,
                    b0 = zero, b1 = zero, y0, y1, y2, v0, v1, v2;
              if constexpr (TWO) {
                z0 = chunk(k, 8 + 2 * e_col);
                z1 = chunk(k, 8 + 2 * e_col + 1);
              }
              if constexpr (EPI == L_LINEAR) {
                x0 = x0 + bias0;
                x1 = x1 + bias1;
                if (e.in1) {
                  a0 = lo4(P.a[k]);
                  a1 = hi4(P.a[k]);
                }
              } else if constexpr (EPI == L_DGATE) {
                a0 = lo4(P.a[k]);
                a1 = hi4(P.a[k]);
                b0 = lo4(P.b[k]);
                b1 = hi4(P.b[k]);
              }
              epi_math<uint16_t, EPI>(act, x0, z0, a0, b0, y0, y1, y2);
              epi_math<uint16_t, EPI>(act, x1, z1, a1, b1, v0, v1, v2);
              r0[k] = pack(y0, v0);
              r1[k] = pack(y1, v1);
              if constexpr (EPI != L_LINEAR) r2[k] = pack(y2, v2);
            }
          };
          act_dispatch<EPI>(e.act, math);
          put(r0, e.out, e.ldo, 2, 0, blk);
          if (e.out2) put(r1, e.out2, e.ldo2, 2, 0, blk);
          if constexpr (EPI != L_LINEAR) {
            if (e.out3) put(r2, e.out3, e.ldo3, 2, 0, blk);
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      };
      if constexpr (C::AHEAD) {
        Pre P0, P1;
        load(P0, 0);
        load(P1, 1);
        next_tile();
#pragma unroll 1
        for (int blk = 0; blk < NB; blk += 2) {
          process(P0, blk);
          load(P0, blk + 2);
          process(P1, blk + 1);
          load(P1, blk + 3);
        }
      } else {
        Pre P;
        __syncthreads();  // every wave is done reading the operand stages
#pragma unroll 1
        for (int blk = 0; blk < NB; ++blk) {
          load(P, blk);
          process(P, blk);
        }
      }
    }
    if constexpr (!C::AHEAD) {
      __syncthreads();  // the epilogue is done with LDS
      if (tile + (int)gridDim.x < ntiles) dma_begin(tile + gridDim.x);
    }
  }
}

using LinBig = LTile<256, 1, true>;
using LinSmall = LTile<128, 2, false>;
using LinSplit = LTile<128, 2, false, 2>;
using LinTiny = LTile<64, 4, false, 4>;

template <class C, int EPI, bool TA, bool TB>
hipError_t lin_run(const LinArgs& g, hipStream_t st) {
  constexpr int OM = EPI == L_GATED ? C::BM / 2 : C::BM;
  const int64_t ntm = (epi_width<EPI>(g.M) - g.m_off + OM - 1) / OM, ntn = (g.N - g.n_off + C::BN - 1) / C::BN;
  const int64_t tiles = ntm * ntn * (EPI == L_ACC && TA && !TB ? g.splits : 1);
  if (tiles <= 0) return hipSuccess;
  const int64_t resident = (int64_t)(C::OCC * 4 / C::NW) * g_num_cus();
  hipLaunchKernelGGL((lin_kernel<C, EPI, TA, TB>), dim3((uint32_t)(tiles < resident ? tiles : resident)), dim3(C::NT), 0,
                     st, g);
  return hipGetLastError();
}

// Which tiles: 256x256 for more than half a round of them (one partial round beats two of
// 128x128 tiles, whose operand bytes per product are twice as many); 128x128, two workgroups
// per compute unit, for more than one per unit; 128x128 with two groups of waves on a tile's k
// range for more than half a unit's worth; else 64x64 with four groups, where the chain of
// stages, each a trip to memory, is what takes the time.
enum LinTileKind { LT_BIG, LT_SMALL, LT_SPLIT, LT_TINY };
template <int EPI>
inline LinTileKind lin_tile(int64_t M, int64_t N) {
  const int64_t cus = g_num_cus(), w = EPI == L_GATED ? 2 * M : M;
  if (2 * ((w + 255) / 256) * ((N + 255) / 256) > cus) return LT_BIG;
  const int64_t t = ((w + 127) / 128) * ((N + 127) / 128);
  return t > cus ? LT_SMALL : (((w + 63) / 64) * ((N + 63) / 64) > cus ? LT_SPLIT : LT_TINY);
}

// A product of too few tiles for the chip may be shared along k (LinArgs::splits): from 96 stages
// on, where one workgroup's chain takes longer than the join (15 x 8192 -> 512: 18 us against 23;
// 100 x 4096 -> 1024, 64 stages: 18 against 16), at least 12 stages and at most 32 parts (their
// join reads them all). 256x256 tiles where they fill the chip with parts of 48 stages or more
// (1999 x 50264 -> 1024: 217 us against 277; 1000 x 16384 -> 1000, 16 stages: 60 against 50).
constexpr int64_t kSplitStages = 96;
inline bool lin_split_big(int64_t M, int64_t N, int64_t K) {
  const int64_t s = g_num_cus() / (((M + 255) / 256) * ((N + 255) / 256));
  return M >= 192 && N >= 192 && s > 0 && (K + 63) / 64 >= 48 * s;
}

template <int EPI, bool TA, bool TB>
hipError_t lin_bf16(const LinArgs& g, hipStream_t st) {
  if constexpr (EPI == L_ACC && TA && !TB) {
    if (g.splits > 1) {
      int64_t k = 0;
      for (int s = 0; s < g.nsrc; ++s) k += g.K[s];
      return lin_split_big(g.M, g.N, k) ? lin_run<LinBig, EPI, TA, TB>(g, st) : lin_run<LinSmall, EPI, TA, TB>(g, st);
    }
  }
  switch (lin_tile<EPI>(epi_width<EPI>(g.M), g.N)) {
    case LT_BIG: {
      // A last round of large tiles that would be at most half full: the whole rounds run as large
      // tiles over a band of tile columns (or rows, whichever band holds more of them), the rest as
      // 128x128 tiles in a second launch. (Not the cross entropy's maxima and sums: their blocks
      // follow the tile.) A tile owns its output elements either way.
      constexpr int OM = EPI == L_GATED ? 128 : 256;
      const int cus = g_num_cus(), Mw = epi_width<EPI>(g.M);
      const int ntm = (Mw + OM - 1) / OM, ntn = (g.N + 255) / 256;
      const int64_t tiles = (int64_t)ntm * ntn, full = tiles / cus * cus, rem = tiles - full;
      if (EPI != L_LSE && full > 0 && rem > 0 && 2 * rem <= cus && g.K[0] >= 512) {
        LinArgs g1 = g, g2 = g;
        const int mb = (int)(full / ntn), nb = (int)(full / ntm);  // whole bands the rounds hold
        if (mb * (int64_t)ntn >= nb * (int64_t)ntm) {
          g1.M = mb * OM;
          g2.m_off = g1.M;
        } else {
          g1.N = nb * 256;
          g2.n_off = g1.N;
        }
        if (g1.M > 0 && g1.N > 0) {
          hipError_t e = lin_run<LinBig, EPI, TA, TB>(g1, st);
          if (e != hipSuccess) return e;
          const int64_t t = (int64_t)((Mw - g2.m_off + OM / 2 - 1) / (OM / 2)) * ((g.N - g2.n_off + 127) / 128);
          return t > cus ? lin_run<LinSmall, EPI, TA, TB>(g2, st) : lin_run<LinSplit, EPI, TA, TB>(g2, st);
        }
      }
      return lin_run<LinBig, EPI, TA, TB>(g, st);
    }
    case LT_SMALL: return lin_run<LinSmall, EPI, TA, TB>(g, st);
    case LT_SPLIT: return lin_run<LinSplit, EPI, TA, TB>(g, st);
    default: return lin_run<LinTiny, EPI, TA, TB>(g, st);
  }
}

#define FORGE_LIN_FORMS(X)                                                                                  \
  X(L_LINEAR, false, false) X(L_GATED, false, false) X(L_LSE, false, false) X(L_DLOGIT, false, false)       \
  X(L_DGATE, true, false) X(L_ACC, true, false) X(L_ACC, true, true)

}  // namespace forge
