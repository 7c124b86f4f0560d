// Internal: products with an epilogue (forge_ops.h) on bfloat16 operands, large tiles.
//
// C[m][n] = sum_k A[m][k] B[n][k], m along the output's columns. Either operand may have k
// as its fast index (rows of W in a forward product, rows of X or dY) or as its slow index
// (rows of W in an input gradient, rows of X and dY in a weight gradient).
//
// Mainloop. Stages of BK k go from global memory straight into LDS (buffer loads with the
// LDS bit, 1 KiB per wave instruction; out-of-range offsets write zeros, so ragged k and
// rows past the edge need no other masking) into a ring of NSTAGE stages. k-fast rows are
// read with 16-byte LDS reads, k-slow rows with the LDS transpose read; XOR swizzles of the
// 16-byte chunks keep both free of bank conflicts. v_mfma_f32_32x32x16_bf16, FP32 sums.
// The 256x256 tile (8 waves of 128x64, two per SIMD) runs the ping-pong schedule of the
// weight-gradient kernel: two groups with one wave of each on every SIMD, one multiplying
// from registers while the other reads LDS and issues loads; the 128x128 tile (4 waves of
// 64x64, two workgroups per compute unit) uses one barrier per stage. Several products may
// run into one accumulation (MULTI: the stages of the pairs follow one another).
// Operands are addressed from the tile's own origin (64-bit base, 32-bit offsets), so a
// k-fast operand may be of any size; a k-slow one spans less than 2^31 bytes.
//
// Epilogue. Vector epilogues hand each wave's accumulators through a private LDS region, 32
// output rows at a time, so that whole row segments are read and written without a
// workgroup barrier; the cross entropy's maximum and sum are taken from the accumulators
// directly (a lane holds TM / 2 of a token's logits, its partner lane the other half).
#pragma once

#include "forge_gemm_kernel.h"
#include "forge_ops.h"

namespace forge {

template <int BM_, int BN_, int BK_, int WM_, int WN_, bool PP_, int NSTAGE_ = 4>
struct LTile {
  static constexpr int BM = BM_, BN = BN_, BK = BK_, WM = WM_, WN = WN_, NSTAGE = NSTAGE_;
  static constexpr bool PP = PP_;
  static constexpr int NW = WM * WN, NT = 64 * NW, OCC = 2;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  static constexpr int KST = BK / 16;  // k-steps per stage
  static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2;
  static constexpr int LDW = TM + 4;  // epilogue rows (floats)
  static constexpr int RING = NSTAGE * (A_BYTES + B_BYTES), EPIB = NW * 32 * LDW * 4;
  static constexpr int SMEM = RING > EPIB ? RING : EPIB;
  static constexpr int PA = A_BYTES / 16 / NT, PB = B_BYTES / 16 / NT;  // loads per stage and wave
  static constexpr int LPS = PA + PB;
  static_assert(KST == 2 && NSTAGE == 4, "two k-steps per stage, a ring of four");
  static_assert((NSTAGE - 1) * LPS <= 63, "vmcnt range");
  static_assert(!PP || NW == 8, "ping-pong: two waves per SIMD");
};

// Layout of one operand's stage in LDS: R output indexes x BK k.
template <class C, int R, bool TR>
struct LOper {
  static constexpr int ROWB = (TR ? R : C::BK) * 2;  // bytes per LDS row
  static constexpr int CPR = ROWB / 16;              // 16-byte chunks per row
  static constexpr int RSTEP = C::NT / CPR;          // rows between a thread's chunks
  static constexpr int KW = TR ? 1 : 16 / CPR;       // k-fast rows per 256 bytes
  static constexpr int STAGE = R * C::BK * 2;
  __host__ __device__ static constexpr int swz(int row) {
    return TR ? 4 * (row & 3) : (row / KW) % CPR;
  }
  static_assert(C::NT % CPR == 0 && RSTEP % (TR ? 4 : 16) == 0, "a thread's chunks share a swizzled column");
  static_assert(!TR || CPR >= 16, "transpose reads: rows of 256 bytes or more");
};

template <class C, int EPI, bool TA, bool TB>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::OCC, C::OCC)))
void lin_kernel(LinArgs g) {
  using OA = LOper<C, C::BM, TA>;
  using OB = LOper<C, C::BN, TB>;
  constexpr bool TWO = EPI == L_GATED;              // A: BM / 2 rows of gate, then BM / 2 of up
  constexpr bool MULTI = EPI == L_ACC && TA && !TB;  // several operand pairs
  constexpr int OM = TWO ? C::BM / 2 : C::BM;        // output columns per tile
  static_assert(!TWO || (!TA && C::PA % 2 == 0), "gate and up: k fast, half of the loads each");
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::SMEM];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave_u = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave_u % C::WM, wn = wave_u / C::WM;
  const uint32_t lds0 = lds_addr(smem);
  const int ntm = (epi_width<EPI>(g.M) - g.m_off + OM - 1) / OM, ntn = (g.N - g.n_off + C::BN - 1) / C::BN;
  const int ntiles = ntm * ntn;
  int nst = (g.K[0] + C::BK - 1) / C::BK;
  if constexpr (MULTI) {
    for (int s = 1; s < g.nsrc; ++s) nst += (g.K[s] + C::BK - 1) / C::BK;
  }
  const int nstr = (nst + C::NSTAGE - 1) / C::NSTAGE * C::NSTAGE;

  for (int tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {
    int tm, tn;
    g_tile(tile, ntm, ntn, tm, tn);
    const int m0 = g.m_off + tm * OM, n0 = g.n_off + tn * C::BN;
    // per-thread values from an opaque copy of the thread index: recomputed per tile, so
    // nothing is held through the epilogue
    int ttid = tid;
    asm volatile("" : "+v"(ttid));
    const int t_lane = ttid & 63, t_hi = t_lane >> 5, t_l32 = t_lane & 31;

    // ---- operand sources ----
    const int a_row = ttid / OA::CPR, b_row = ttid / OB::CPR;
    const int a_chunk = (ttid % OA::CPR) ^ OA::swz(a_row), b_chunk = (ttid % OB::CPR) ^ OB::swz(b_row);
    __amdgpu_buffer_rsrc_t rA, rA2, rB;
    int fK, fk = 0, fsrc = 0;       // current pair: its K, the next stage's first k
    uint32_t a_off, b_off;          // this thread's first chunk of stage 0
    uint32_t a_rowb, b_rowb;        // bytes between its chunks
    uint32_t a_kb, b_kb;            // bytes per k (k-slow: the pitch)
    auto source = [&](int s) {
      const int64_t lda = g.lda[s], ldb = g.ldb[s];
      fK = g.K[s];
      const int64_t K8 = (fK + 7) / 8 * 8;
      // extents: a k-fast operand's rows of this tile; a k-slow one from this tile's columns
      // on, whole 16-byte chunks (rows are padded to them)
      auto ext = [&](bool tr, int64_t ld, int64_t left, int64_t rows) -> uint32_t {
        if (fK <= 0 || left <= 0) return 0u;
        const int64_t n = tr ? (fK - 1) * ld + (left + 7) / 8 * 8 : ((left < rows ? left : rows) - 1) * ld + K8;
        return (uint32_t)(n * 2);
      };
      const char* pa = static_cast<const char*>(g.A[s]);
      const char* pb = static_cast<const char*>(g.B[s]);
      rA = make_rsrc(pa + (TA ? (int64_t)m0 : (int64_t)m0 * lda) * 2, ext(TA, lda, g.M - m0, OM));
      if constexpr (TWO) {
        const char* p2 = static_cast<const char*>(g.A[1]);
        rA2 = make_rsrc(p2 + (int64_t)m0 * g.lda[1] * 2, ext(false, g.lda[1], g.M - m0, OM));
      }
      rB = make_rsrc(pb + (TB ? (int64_t)n0 : (int64_t)n0 * ldb) * 2, ext(TB, ldb, g.N - n0, C::BN));
      a_off = (uint32_t)(a_row * lda * 2 + a_chunk * 16);
      b_off = (uint32_t)(b_row * ldb * 2 + b_chunk * 16);
      a_rowb = (uint32_t)(OA::RSTEP * lda * 2);
      b_rowb = (uint32_t)(OB::RSTEP * ldb * 2);
      a_kb = TA ? (uint32_t)(lda * 2) : 2u;
      b_kb = TB ? (uint32_t)(ldb * 2) : 2u;
    };
    source(0);
    uint32_t a2_off = 0;
    if constexpr (TWO) a2_off = (uint32_t)(a_row * g.lda[1] * 2 + a_chunk * 16);
    // Issues the next stage (in order: 0, 1, ...) into ring buffer buf. Stages past the end
    // load zeros.
    auto dma = [&](auto buf_c) {
      constexpr int buf = decltype(buf_c)::value;
      const uint32_t ak = (uint32_t)fk * a_kb, bk = (uint32_t)fk * b_kb;
#pragma unroll
      for (int j = 0; j < C::PA; ++j) {
        const bool second = TWO && j >= C::PA / 2;
        const int k = fk + (TA ? a_row + j * OA::RSTEP : a_chunk * 8);
        const uint32_t row = (uint32_t)(second ? j - C::PA / 2 : j) * a_rowb;
        const uint32_t off = k < fK ? (second ? a2_off : a_off) + ak + row : kOOB;
        dma16(second ? rA2 : rA, smem + buf * C::A_BYTES + (j * C::NT + wave_u * 64) * 16, off);
      }
#pragma unroll
      for (int j = 0; j < C::PB; ++j) {
        const int k = fk + (TB ? b_row + j * OB::RSTEP : b_chunk * 8);
        const uint32_t off = k < fK ? b_off + bk + (uint32_t)j * b_rowb : kOOB;
        dma16(rB, smem + C::NSTAGE * C::A_BYTES + buf * C::B_BYTES + (j * C::NT + wave_u * 64) * 16, off);
      }
      fk += C::BK;
      if constexpr (MULTI) {
        if (fk >= fK && fsrc + 1 < g.nsrc) {
          source(++fsrc);
          fk = 0;
        }
      }
    };

    // ---- fragment addresses (stage buffer 0, k-step 0) ----
    // k-slow rows, transpose read: lane (r4, c4, half, hi) reads row 8 hi + r4, elements
    // 16 half + 4 c4 .. +3 of the 32-wide fragment; it receives 4 k of column l32
    auto tr_addr = [&](int base, int rowb, auto swz, int col0) -> uint32_t {
      const int r4 = (t_lane & 15) >> 2, c4 = t_lane & 3;
      const int row = 8 * t_hi + r4, chunk = col0 / 8 + 2 * ((t_lane >> 4) & 1) + (c4 >> 1);
      return lds0 + (uint32_t)(base + row * rowb + 16 * (chunk ^ swz(row)) + 8 * (c4 & 1));
    };
    const int a_r0 = TWO ? wm * (C::TM / 2) : wm * C::TM, b_r0 = wn * C::TN;
    uint32_t a_ad[TA ? C::FM : C::KST], b_ad[TB ? C::FN : C::KST];
    if constexpr (TA) {
#pragma unroll
      for (int f = 0; f < C::FM; ++f) a_ad[f] = tr_addr(0, OA::ROWB, [](int r) { return OA::swz(r); }, a_r0 + 32 * f);
    } else {
#pragma unroll
      for (int kk = 0; kk < C::KST; ++kk)
        a_ad[kk] = lds0 + (uint32_t)((a_r0 + t_l32) * OA::ROWB + 16 * ((2 * kk + t_hi) ^ OA::swz(t_l32)));
    }
    if constexpr (TB) {
#pragma unroll
      for (int f = 0; f < C::FN; ++f)
        b_ad[f] = tr_addr(C::NSTAGE * C::A_BYTES, OB::ROWB, [](int r) { return OB::swz(r); }, b_r0 + 32 * f);
    } else {
#pragma unroll
      for (int kk = 0; kk < C::KST; ++kk)
        b_ad[kk] = lds0 + (uint32_t)(C::NSTAGE * C::A_BYTES + (b_r0 + t_l32) * OB::ROWB +
                                     16 * ((2 * kk + t_hi) ^ OB::swz(t_l32)));
    }
    // One k-step's fragments: per 32 rows one 16-byte read (k fast) or two 8-byte reads
    struct Frag {
      u32x4 ak[TA ? 1 : C::FM];
      u32x2 at[TA ? C::FM : 1][2];
      u32x4 bk[TB ? 1 : C::FN];
      u32x2 bt[TB ? C::FN : 1][2];
    };
    constexpr int NRA = TA ? 2 * C::FM : C::FM, NRB = TB ? 2 * C::FN : C::FN, NR = NRA + NRB;
    auto read_one = [&](Frag& F, auto buf_c, auto kk_c, auto r_c) {
      constexpr int buf = decltype(buf_c)::value, kk = decltype(kk_c)::value, r = decltype(r_c)::value;
      if constexpr (r < NRA) {
        if constexpr (TA) {
          F.at[r / 2][r % 2] = ds_tr_asm<buf * C::A_BYTES + (kk * 16 + (r % 2) * 4) * OA::ROWB>(a_ad[r / 2]);
        } else {
          constexpr int half = C::FM / 2;
          constexpr int row = !TWO ? 32 * r : (r < half ? 32 * r : C::BM / 2 + 32 * (r - half));
          F.ak[r] = ds_b128_asm<buf * C::A_BYTES + row * OA::ROWB>(a_ad[kk]);
        }
      } else {
        constexpr int q = r - NRA;
        if constexpr (TB)
          F.bt[q / 2][q % 2] = ds_tr_asm<buf * C::B_BYTES + (kk * 16 + (q % 2) * 4) * OB::ROWB>(b_ad[q / 2]);
        else
          F.bk[q] = ds_b128_asm<buf * C::B_BYTES + 32 * q * OB::ROWB>(b_ad[kk]);
      }
    };
    auto settle = [&](Frag& F) {
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

    f32x16 acc[C::FM][C::FN];
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < C::FN; ++fn)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[fm][fn][e] = 0.f;
    auto mfma_one = [&](const Frag& F, auto i_c) {
      constexpr int fm = decltype(i_c)::value / C::FN, fn = decltype(i_c)::value % C::FN;
      bf16x8 av, bv;
      if constexpr (TA)
        av = __builtin_bit_cast(bf16x8, u32x4{F.at[fm][0].x, F.at[fm][0].y, F.at[fm][1].x, F.at[fm][1].y});
      else
        av = __builtin_bit_cast(bf16x8, F.ak[fm]);
      if constexpr (TB)
        bv = __builtin_bit_cast(bf16x8, u32x4{F.bt[fn][0].x, F.bt[fn][0].y, F.bt[fn][1].x, F.bt[fn][1].y});
      else
        bv = __builtin_bit_cast(bf16x8, F.bk[fn]);
      acc[fm][fn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(av, bv, acc[fm][fn], 0, 0, 0);
    };
    // the MFMAs of F with the reads of G over the first half of them; sched_barrier keeps
    // the order
    constexpr int NM = C::FM * C::FN;
    constexpr int RPM = (NR + NM / 2 - 1) / (NM / 2);
    auto mma_reading = [&](const Frag& F, Frag& G, auto buf_c, auto kk_c, auto&& after_first) {
      static_for<0, NM>([&](auto i_c) {
        constexpr int i = decltype(i_c)::value;
        mfma_one(F, i_c);
        if constexpr (i == 0) after_first();
        constexpr int lo = i * RPM < NR ? i * RPM : NR, up = (i + 1) * RPM < NR ? (i + 1) * RPM : NR;
        static_for<lo, up>([&](auto r_c) { read_one(G, buf_c, kk_c, r_c); });
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;

    __syncthreads();  // the previous tile's epilogue is done with LDS
    static_for<0, C::NSTAGE>([&](auto b_c) { dma(b_c); });
    if constexpr (C::PP) {
      // Group A: waves 0..3, group B: waves 4..7, B one barrier behind. Memory phase M_i:
      // issue stage i + 3, read k-step 1 of stage i. Compute phase C_i: the stage's MFMAs,
      // reading k-step 0 of stage i + 1 over the first of them; then wait for the own loads
      // of stage i + 2, which the next barrier publishes. Stage i's buffer is refilled two
      // phases after its last read. Loads past the end are issued too: the vmcnt waits
      // count a fixed number per phase.
      const bool grp_b = wave_u >= C::NW / 2;
      Frag F0[2], F1;
      vm_wait_barrier<(C::NSTAGE - 2) * C::LPS>();  // stages 0 and 1 published
      static_for<0, NR>([&](auto r_c) { read_one(F0[0], I0{}, I0{}, r_c); });
      if (grp_b) wg_barrier();
      auto pp_stage = [&](auto R_c, int i) {
        constexpr int R = decltype(R_c)::value;  // i % NSTAGE
        constexpr int cur = R % 2, nxt = 1 - cur;
        if (i >= 1) dma(std::integral_constant<int, (R + C::NSTAGE - 1) % C::NSTAGE>{});
        static_for<0, NR>([&](auto r_c) { read_one(F1, R_c, I1{}, r_c); });
        vm_wait_barrier<(C::NSTAGE - 2) * C::LPS>();  // fragments landed
        settle(F0[cur]);
        settle(F1);
        __builtin_amdgcn_sched_barrier(0);
        issue_prio<1>();
        mma_reading(F0[cur], F0[nxt], std::integral_constant<int, (R + 1) % C::NSTAGE>{}, I0{}, [] {});
        static_for<0, NM>([&](auto i_c) { mfma_one(F1, i_c); });
        issue_prio<0>();
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0)" ::"i"((C::NSTAGE - 3) * C::LPS) : "memory");
        wg_barrier();
      };
      for (int i0 = 0; i0 < nst; i0 += C::NSTAGE)
        static_for<0, C::NSTAGE>([&](auto r_c) {
          const int i = i0 + decltype(r_c)::value;
          if (i < nst) pp_stage(r_c, i);
        });
      // k-step 0 of a stage past the end was read: its registers stay pinned until it landed
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      settle(F0[0]);
      settle(F0[1]);
      if (!grp_b) wg_barrier();  // both groups pass the same number of barriers
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    } else {
      // one barrier per stage, before its last k-step: own loads of the next stage and own
      // LDS reads done; it publishes that stage and frees this one's buffer
      Frag F0, F1;
      vm_wait_barrier<(C::NSTAGE - 1) * C::LPS>();
      static_for<0, NR>([&](auto r_c) { read_one(F0, I0{}, I0{}, r_c); });
      for (int st = 0; st < nstr; st += C::NSTAGE)
        static_for<0, C::NSTAGE>([&](auto r_c) {
          constexpr int R = decltype(r_c)::value;
          lgkm_wait<0>();
          settle(F0);
          mma_reading(F0, F1, r_c, I1{}, [] {});
          vm_wait_barrier<(C::NSTAGE - 2) * C::LPS>();
          settle(F1);
          mma_reading(F1, F0, std::integral_constant<int, (R + 1) % C::NSTAGE>{}, I0{}, [&] { dma(r_c); });
        });
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      settle(F0);
      settle(F1);
    }

    // ---- epilogue ----
    int etid = static_cast<int>(threadIdx.x);
    asm volatile("" : "+v"(etid));
    const int e_lane = etid & 63, e_hi = e_lane >> 5, e_l32 = e_lane & 31;
    if constexpr (EPI == L_LSE) {
      // lane (l32, hi): logits m = 32 fm + 8 q + 4 hi + j of token n = l32
      const int mb = m0 + wm * C::TM;
      const int left = g.M - mb;  // entries inside the vocabulary
#pragma unroll
      for (int fn = 0; fn < C::FN; ++fn) {
        const int n = n0 + wn * C::TN + 32 * fn + e_l32;
        const bool ok = n < g.N;
        if (left < C::TM) {  // the last block: entries past the vocabulary count nothing
#pragma unroll
          for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (32 * fm + 8 * (e / 4) + 4 * e_hi + e % 4 >= left) acc[fm][fn][e] = -__builtin_huge_valf();
        }
        float mx = -__builtin_huge_valf();
#pragma unroll
        for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
          for (int e = 0; e < 16; ++e) mx = fmaxf(mx, acc[fm][fn][e]);
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float ref = mx > -__builtin_huge_valf() ? mx : 0.f;
        const int64_t y = ok ? g.e.target[n] : -1;
        // this lane's place of the target in its block, if it holds it
        const int64_t d = y - mb;
        const int at = (y >= 0 && d >= 0 && d < C::TM && d < left && ((d >> 2) & 1) == e_hi) ? (int)d : -1;
        float sum = 0.f, tl = 0.f;
#pragma unroll
        for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float x = acc[fm][fn][e];
            sum += __expf(x - ref);
            tl = at == 32 * fm + 8 * (e / 4) + 4 * e_hi + e % 4 ? x : tl;
          }
        sum += __shfl_xor(sum, 32);
        if (at >= 0) g.e.tlogit[n] = tl;
        if (ok && e_hi == 0 && left > 0)
          *reinterpret_cast<float2*>(g.e.part + ((int64_t)(mb / C::TM) * g.e.part_ld + n) * 2) = float2{mx, sum};
      }
    } else {
      const float sc = (EPI == L_ACC || EPI == L_DLOGIT) ? epi_scale(g.e) : 1.f;
      const int Mw = epi_width<EPI>(g.M);
      constexpr int OW = TWO ? C::TM / 2 : C::TM;      // output columns per wave
      constexpr int VPR = OW / 4, NV = 32 * VPR / 64;  // 4-vectors per row, per lane and block
      float* Ew = reinterpret_cast<float*>(smem) + wave_u * (32 * C::LDW);
      const int mw = m0 + wm * OW, nw = n0 + wn * C::TN;
      __syncthreads();  // every wave is done reading the operand stages
#pragma unroll 1
      for (int fn = 0; fn < C::FN; ++fn) {
#pragma unroll
        for (int f = 0; f < C::FN; ++f) {
          if (f == fn) {
#pragma unroll
            for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4*>(Ew + e_l32 * C::LDW + 32 * fm + 8 * q + 4 * e_hi) =
                    f32x4{acc[fm][f][4 * q], acc[fm][f][4 * q + 1], acc[fm][f][4 * q + 2], acc[fm][f][4 * q + 3]};
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 2
        for (int k = 0; k < NV; ++k) {
          const int v = e_lane + k * 64, row = v / VPR, col = (v % VPR) * 4;
          const int n = nw + 32 * fn + row, m = mw + col;
          if (n < g.N && m < Mw) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(Ew + row * C::LDW + col);
            f32x4 x2 = x;
            if constexpr (TWO) x2 = *reinterpret_cast<const f32x4*>(Ew + row * C::LDW + C::TM / 2 + col);
            epi_vec<uint16_t, EPI>(g.e, n, m, g.M, x, x2, sc);
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
    }
  }
}

using LinBig = LTile<256, 256, 32, 2, 4, true>;
using LinSmall = LTile<128, 128, 32, 2, 2, false>;

template <class C, int EPI, bool TA, bool TB>
hipError_t lin_run(const LinArgs& g, hipStream_t st) {
  constexpr int OM = EPI == L_GATED ? C::BM / 2 : C::BM;
  const int64_t ntm = (epi_width<EPI>(g.M) - g.m_off + OM - 1) / OM, ntn = (g.N - g.n_off + C::BN - 1) / C::BN;
  const int64_t tiles = ntm * ntn;
  if (tiles <= 0) return hipSuccess;
  const int64_t resident = (int64_t)(C::OCC * 4 / C::NW) * g_num_cus();
  hipLaunchKernelGGL((lin_kernel<C, EPI, TA, TB>), dim3((uint32_t)(tiles < resident ? tiles : resident)), dim3(C::NT), 0,
                     st, g);
  return hipGetLastError();
}

// Large tiles for more than half a round of them (one partial round of 256x256 tiles beats
// two of 128x128 tiles, whose operand bytes per product are twice as many); else 128x128.
template <int EPI>
inline bool lin_big(int64_t M, int64_t N) {
  const int64_t OM = EPI == L_GATED ? 128 : 256;
  return 2 * ((M + OM - 1) / OM) * ((N + 255) / 256) > g_num_cus();
}

template <int EPI, bool TA, bool TB>
hipError_t lin_bf16(const LinArgs& g, hipStream_t st) {
  return lin_big<EPI>(epi_width<EPI>(g.M), g.N) ? lin_run<LinBig, EPI, TA, TB>(g, st)
                                                : lin_run<LinSmall, EPI, TA, TB>(g, st);
}

#define FORGE_LIN_FORMS(X)                                                                                  \
  X(L_LINEAR, false, false) X(L_GATED, false, false) X(L_LSE, false, false) X(L_DLOGIT, false, false)       \
  X(L_DGATE, true, false) X(L_ACC, true, false) X(L_ACC, true, true)

}  // namespace forge
