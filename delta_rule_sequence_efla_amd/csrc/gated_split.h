// gated_split.h -- the sequential chunk pass of the gated delta rule for bf16
// inputs, each chunk's work spread over fourteen wavefronts, with the state good
// to 16 significant bits or more.
//
// Per chunk (start state S, X and a from gated_ut.h; e = e^G, w = e^{G_C - G}):
//     U = X a (V - diag(e) K S),   S <- e^{G_C} S + K^T diag(w) U,
//     O = diag(e) Q S + (Gam * tril(Q K^T)) U
// q, k and v are bf16, so their products are exact in float32 sums; what would
// be lost is the rounding of S, of D = a (V - diag(e) K S), of X and of U where
// they are operands (2^-8 each).  On the way to the state they therefore go in
// as two bf16 parts (hi + lo, 2^-16): K S and K^T U twice, X D three times
// (lo lo dropped).  On the way to o, which is rounded to bf16 anyway, the high
// parts alone go in.
//
// A workgroup owns 32 value columns (two 16-column tiles) of one (sequence,
// head).  A wavefront's time is close to the sum of its matrix instructions (16
// cycles), vector instructions (4) and LDS round trips, so the chain S -> D -> U
// -> S is cut into as many wavefronts as the registers allow:
//   Y wave per tile and   D = a (V - diag(e) K S) for its 32 tokens; after barrier
//   half of the tokens    M U = X D for them (the later half reads the earlier
//                         half's D); publishes U (for O) and diag(w) U in two
//                         parts (for S)
//   S wave per 32 key     S <- e^{G_C} S + K^T (diag(w) U) in fp32 registers;
//   dims                  publishes S in two parts
//   O wave per half of    Z^T = S^T Q^T, then O^T = diag(e) Z^T + U^T P^T, staged
//   the tokens            in LDS and stored a chunk later
//   three P waves         Gam * tril(Q K^T), half of the key dimension a phase
//   DMA wave              Q, K, V and the chunk's gates into a three-slot ring
// X does not pass the LDS: it comes in fragment order, 12 KiB a chunk, and the
// Y waves load it into registers half a chunk ahead; the S waves, idle then,
// touch a later chunk's X so that those loads are served by the L2.
// Three barriers a chunk, every exchange buffer written in one phase and read in
// another:
//   A (chunk n in LDS, S_n published)
//     Y: K S, D -> publish | S: read K^T | O: Z^T | P: finish P_n | DMA: half of chunk n+2
//   M (D published)
//     Y: X D -> publish U | P: gates -> publish
//   B (U and P published, chunk n+1 in LDS)
//     Y: load K, V, X of n+1 | S: update -> publish | O: O^T | P: start n+1 | DMA
// Bound by that chain: 4 x 4096 tokens of 16 heads, d 128, take 111 us, 1.7 us a chunk
// on every compute unit: 222 MB counted (2 TB/s), 332 TFLOP/s of products.  Eight
// wavefronts took 117 us where these took 107, eleven 109; without P and O (outputs
// wrong) 100; wave priorities, sleeps before contended reads and interleave hints
// were no faster.  The backward's instance, states only, took 49 us for 8 x 2048
// tokens of 8 heads as a launch of its own (gated_reverse.h has both chains' time).
// It keeps this kernel's LDS layout, of which it leaves 63 of 154 KiB (d_k 128)
// unused: Q's third of the ring, bU, P and O_st.
#pragma once

#include <type_traits>

#include "gated_ut.h"

namespace efla {

template <int DK>
struct GatedSplitShape {
  static_assert(DK == 64 || DK == 128, "shapes of the gated recurrence");
  static constexpr int C = 64, BV = 32;
  static constexpr int NT = BV / 16, NRT = C / 16, NKU_D = DK / 32, NKU_C = C / 32, KH = NKU_D / 2;
  static constexpr int QOFF = 0, KOFF = C * DK, VOFF = 2 * C * DK, GOFF = 2 * C * DK + C * BV;
  static constexpr int SLOT = GOFF + kGatedG * 2;  // in bf16 elements
  static constexpr int NPF = 6, OP = BV + 8;
  using TQ = DmaTile<C, DK, 1, true>;
  using TV = DmaTile<C, BV, 1>;
  static constexpr int PQ = TQ::PER_WAVE, PV = TV::PER_WAVE, COUNT = 2 * PQ + PV + 1;
  // wavefronts by index (SIMD = index % 4)
  static constexpr int NSW = NKU_D;  // S waves, 32 key dims each
  static constexpr int kY = 0, kS = 4, kDma = kS + NSW, kP = kDma + 1, kO = kP + 3;
  static constexpr int THREADS = (kO + 2) * kWave, STATE_THREADS = (kDma + 1) * kWave;
};

template <int DK>
struct GatedSplitLds {
  using S = GatedSplitShape<DK>;
  alignas(1024) uint16_t ring[3 * S::SLOT];
  alignas(16) bf16x8 bS_buf[2][S::NT][S::NKU_D][kWave];  // S_n, high and low parts
  alignas(16) bf16x8 bU_buf[S::NT][S::NKU_C][kWave];     // U_n, high parts
  alignas(16) bf16x8 bW_buf[2][S::NT][S::NKU_C][kWave];  // diag(w) U_n, high and low parts
  alignas(16) bf16x8 bD_buf[2][S::NT][kWave];            // D_n of tokens 0-31, high and low parts
  alignas(16) bf16x8 P_buf[S::NPF][kWave];
  alignas(16) uint16_t O_st[S::C][S::OP];
};
template <int DK>
struct GatedSplitRefs {
  using L = GatedSplitLds<DK>;
  uint16_t* ring;
  decltype(L::bS_buf)& bS_buf;
  decltype(L::bU_buf)& bU_buf;
  decltype(L::bW_buf)& bW_buf;
  decltype(L::bD_buf)& bD_buf;
  decltype(L::P_buf)& P_buf;
  decltype(L::O_st)& O_st;
};

// OUT: writes o and the final state.  Else (the backward's recomputation) the
// state at the start of every chunk instead, as the high operand parts,
// transposed, [slots][DV][DK] (the layout of recurrence_split.h), without the O
// and P waves and Q.
template <int DK, bool OUT, typename Lds>
__device__ __forceinline__ void gated_split_run(Lds& lds, const GatedFwd& a, const int x,
                                                const uint16_t* __restrict__ xfr, const float* __restrict__ gws,
                                                const int32_t* __restrict__ order, int NC, int NVB, int remap,
                                                uint16_t* __restrict__ statesT) {
  using S = GatedSplitShape<DK>;
  constexpr int C = S::C, BV = S::BV, NT = S::NT, NRT = S::NRT, NKU_D = S::NKU_D, NKU_C = S::NKU_C, KH = S::KH;
  uint16_t* const ring = lds.ring;
  uint16_t* const slot0 = ring;
  uint16_t* const slot1 = ring + S::SLOT;
  uint16_t* const slot2 = ring + 2 * S::SLOT;
  auto& bS_buf = lds.bS_buf;
  auto& bW_buf = lds.bW_buf;
  auto &bU_buf = lds.bU_buf;
  auto& bD_buf = lds.bD_buf;
  auto& P_buf = lds.P_buf;
  auto& O_st = lds.O_st;

  const int H = a.H, DV = a.DV;
  int bh, vb;
  if (remap) {  // all value blocks of one (b, h) on one XCD (same blockIdx % 8)
    const int slot = x >> 3;
    vb = slot % NVB;
    bh = (slot / NVB) * 8 + (x & 7);
  } else {
    bh = x / NVB;
    vb = x % NVB;
  }
  int seq = bh / H;
  const int h = bh % H, hk = h / (H / a.Hk);
  if (order != nullptr) seq = seq_of_rank(order, seq, a.N);  // packed: longest first
  const SeqSpan sp = seq_span<C>(a.cu, seq, h, H, a.L, NC);
  const int64_t srow = state_row(a.slots, seq, a.P);
  const int nc = sp.nc;
  const int v0 = vb * BV;
  const int lane = threadIdx.x & 63, role = wave_id(), li = lane & 15, g = lane >> 4;
  const auto* q = static_cast<const uint16_t*>(a.q);
  const auto* k = static_cast<const uint16_t*>(a.k);
  const auto* v = static_cast<const uint16_t*>(a.v);
  auto* o = static_cast<uint16_t*>(a.o);
  auto chunk_valid = [&](int n) { return int(sp.len - int64_t(n) * C < C ? sp.len - int64_t(n) * C : C); };
  auto tok_of = [&](int n) { return sp.bos + int64_t(n) * C; };
  auto gates = [&](const uint16_t* cur) { return reinterpret_cast<const float*>(cur + S::GOFF); };  // G2, e, w, a
  auto sync = [&]() {
    wait_lgkm0();
    barrier_nowait();
  };
  auto store_staged = [&](int n, int half) {
    const int valid = chunk_valid(n);
    const int64_t row0 = tok_of(n) * H + h;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 32 * half + 16 * i + (lane >> 2), piece = lane & 3;
      const u32x4 val = *reinterpret_cast<const u32x4*>(&O_st[r][8 * piece]);
      if (r < valid)
        __builtin_nontemporal_store(val, reinterpret_cast<u32x4*>(o + (row0 + int64_t(r) * H) * DV + v0 + 8 * piece));
    }
  };
  auto run = [&](auto&& step) {  // steps of three keep the ring slots compile-time addresses
    for (int n = 0; n < nc; n += 3) {
      step(slot0, slot1, n);
      if (n + 1 < nc) step(slot1, slot2, n + 1);
      if (n + 2 < nc) step(slot2, slot0, n + 2);
    }
  };

  if (role == S::kDma) {
    // ---------------------------------------------------------------- DMA
    // The schedule of recurrence_split.h: chunk n+3 goes into chunk n's slot
    // half after barrier B of step n and half after barrier A of step n+1; a
    // wait is for all but one chunk's transfers.
    constexpr int D = OUT ? S::COUNT : S::COUNT - S::PQ;  // Q comes last
    static_assert(D < 64, "one chunk's transfers fit the vmcnt counter");
    typename S::TQ tq;
    typename S::TV tv;
    tq.init(int64_t(a.Hk) * DK, lane, 0);
    tv.init(int64_t(H) * DV, lane, 0);
    auto issue = [&](int m, int part, int parts) {
      using U = const uint16_t*;
      const int64_t kr = (tok_of(m) * a.Hk + hk) * DK;
      const U ks = (U)uniform_ptr(k + kr), qs = (U)uniform_ptr(q + kr);
      const U vs = (U)uniform_ptr(v + (tok_of(m) * H + h) * DV + v0);
      const void* gsrc = uniform_ptr(gws + (sp.slot0 + m) * kGatedG);
      const int valid = chunk_valid(m);
      const uint32_t addr = lds_addr_of(ring + (m % 3) * S::SLOT);
      auto body = [&](auto ragged) {
        constexpr bool R = decltype(ragged)::value;
#pragma unroll
        for (int j = 0; j < D; ++j) {
          if (j < part * D / parts || j >= (part + 1) * D / parts) continue;
          if (j < S::PQ) tq.template issue<R>(j, addr + 2 * S::KOFF, ks, valid);
          else if (j < S::PQ + S::PV) tv.template issue<R>(j - S::PQ, addr + 2 * S::VOFF, vs, valid);
          else if (j == S::PQ + S::PV) dma16(gsrc, uint32_t(lane) * 16u, addr + 2 * S::GOFF);
          else tq.template issue<R>(j - S::PQ - S::PV - 1, addr + 2 * S::QOFF, qs, valid);
        }
      };
      if (valid == C) body(std::false_type{});
      else body(std::true_type{});
    };
    if (nc > 0) issue(0, 0, 1);
    if (nc > 1) {
      issue(1, 0, 1);
      wait_vmcnt<D>();  // chunk 0 complete
    } else {
      wait_vmcnt<0>();
    }
    if (nc > 2) issue(2, 0, 2);
    for (int n = 0; n < nc; ++n) {
      barrier_nowait();  // A
      if (n + 2 < nc) {
        issue(n + 2, 1, 2);
        barrier_nowait();  // M
        wait_vmcnt<D>();   // chunk n+1 complete: only chunk n+2's transfers remain
      } else {
        barrier_nowait();  // M
        wait_vmcnt<0>();
      }
      barrier_nowait();  // B
      if (n + 3 < nc) issue(n + 3, 0, 2);
    }
    wait_vmcnt<0>();
  } else if (role < S::kS) {
    // ----------------------------------------------------------------- Y
    const int ct = role & 1;  // the later half's waves, with twice the products after M, on SIMDs 2 and 3
    auto y_role = [&](auto halfc) {
      constexpr int Y = decltype(halfc)::value, RT0 = 2 * Y;
      Frag<uint16_t> Kf[2][NKU_D], Xh[2][Y + 1], Xl[2][Y + 1];
      f32x4 aV[2];  // diag(a) V
      auto load_x = [&](int m) {
        const bf16x8* src = reinterpret_cast<const bf16x8*>(xfr + (sp.slot0 + (m < nc ? m : nc - 1)) * kGatedX) + lane;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int kk = 0; kk <= Y; ++kk) {
            Xh[r][kk].v = src[pf_index(RT0 + r, kk) * 64];
            Xl[r][kk].v = src[(6 + pf_index(RT0 + r, kk)) * 64];
          }
      };
      auto load = [&](const uint16_t* __restrict__ cur) {  // this chunk's K and this tile's V
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const bf16x4 v = lds_read_tr(cur + S::VOFF + swz_off<BV>(16 * (RT0 + r) + 4 * g + (li >> 2), 16 * ct + 4 * (li & 3)));
          const f32x4 ag = *reinterpret_cast<const f32x4*>(gates(cur) + 192 + 16 * (RT0 + r) + 4 * g);
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) aV[r][qq] = ag[qq] * static_cast<float>(v[qq]);
        }
#pragma unroll
        for (int ku = 0; ku < NKU_D; ++ku)
#pragma unroll
          for (int r = 0; r < 2; ++r) Kf[r][ku] = wide_frag<DK>(cur + S::KOFF, 16 * (RT0 + r) + li, ku, g);
      };
      auto step = [&](int n) {
        sync();  // A
        if (n == 0) load(ring);
        const float* gt = gates(ring + (n % 3) * S::SLOT) + 16 * RT0 + 4 * g;
        Frag<uint16_t> sh[NKU_D], sl[NKU_D];
#pragma unroll
        for (int ku = 0; ku < NKU_D; ++ku) {
          sh[ku].v = bS_buf[0][ct][ku][lane];
          sl[ku].v = bS_buf[1][ct][ku][lane];
        }
        f32x4 D[2], lo[2], eg[2], wg[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          D[r] = lo[r] = zero4();
          eg[r] = -*reinterpret_cast<const f32x4*>(gt + 64 + 16 * r) * *reinterpret_cast<const f32x4*>(gt + 192 + 16 * r);
          wg[r] = *reinterpret_cast<const f32x4*>(gt + 128 + 16 * r);
        }
#pragma unroll
        for (int ku = 0; ku < NKU_D; ++ku) {  // high and low parts in sums of their own: four chains
#pragma unroll
          for (int r = 0; r < 2; ++r) mma(D[r], Kf[r][ku], sh[ku]);
#pragma unroll
          for (int r = 0; r < 2; ++r) mma(lo[r], Kf[r][ku], sl[ku]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int qq = 0; qq < 4; ++qq)
            D[r][qq] = fmaf(eg[r][qq], D[r][qq] + lo[r][qq], aV[r][qq]);
        Frag<uint16_t> dh[Y + 1], dl[Y + 1];
        split_frag(D[0], D[1], dh[Y], dl[Y]);
        if constexpr (Y == 0) {
          bD_buf[0][ct][lane] = dh[0].v;
          bD_buf[1][ct][lane] = dl[0].v;
        }
        sync();  // M
        if constexpr (Y == 1) {
          dh[0].v = bD_buf[0][ct][lane];
          dl[0].v = bD_buf[1][ct][lane];
        }
        f32x4 U[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) U[r] = zero4();
#pragma unroll
        for (int kk = Y; kk >= 0; --kk) {  // this wave's own D first, while the other half's arrives
#pragma unroll
          for (int r = 0; r < 2; ++r) mma(U[r], Xl[r][kk], dh[kk]);
#pragma unroll
          for (int r = 0; r < 2; ++r) mma(U[r], Xh[r][kk], dl[kk]);
#pragma unroll
          for (int r = 0; r < 2; ++r) mma(U[r], Xh[r][kk], dh[kk]);
        }
        if constexpr (OUT) bU_buf[ct][Y][lane] = acc_frag<uint16_t>(U[0], U[1]).v;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) U[r][qq] *= wg[r][qq];
        Frag<uint16_t> wh, wl;
        split_frag(U[0], U[1], wh, wl);
        bW_buf[0][ct][Y][lane] = wh.v;
        bW_buf[1][ct][Y][lane] = wl.v;
        sync();  // B
        // Past the last chunk the loads go on, from the last chunk's slot and
        // whatever the ring holds, and nothing reads what they bring: behind a
        // branch, the loaded registers would be merged with the old ones, with
        // a wait there.
        load_x(n + 1);
        load(ring + ((n + 1) % 3) * S::SLOT);
      };
      if (nc > 0) load_x(0);
      for (int n = 0; n < nc; ++n) step(n);
    };
    if (role < 2) y_role(std::integral_constant<int, 0>{});
    else y_role(std::integral_constant<int, 1>{});
  } else if (role < S::kDma) {
    // ----------------------------------------------------------------- S
    // rows: logical key dims 32 sw .. 32 sw + 31 (one k-unit)
    const int sw = role - S::kS;
    f32x4 St[2][NT];  // St[d][c][qq] = S[key_phys(16 (2 sw + d) + 4 g + qq)][v0 + 16 c + li]
    const float* s0 = a.s0 == nullptr || srow < 0 ? nullptr : a.s0 + (srow * H + h) * DK * DV + v0 + li;
#pragma unroll
    for (int d = 0; d < 2; ++d)
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int qq = 0; qq < 4; ++qq)
          St[d][c][qq] = s0 != nullptr ? s0[int64_t(key_phys(16 * (2 * sw + d) + 4 * g + qq)) * DV + 16 * c] : 0.0f;
    auto publish = [&]() {
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        Frag<uint16_t> sh, sl;
        split_frag(St[0][c], St[1][c], sh, sl);
        bS_buf[0][c][sw][lane] = sh.v;
        bS_buf[1][c][sw][lane] = sl.v;
      }
    };
    auto save = [&](int n) {  // chunk n's start state, whole rows of S^T (recurrence_split.h)
      constexpr int PR = DK / 8, RW = BV / NKU_D;  // 16-byte pieces per row, rows per S wave
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = RW * sw + 8 * (PR == 16 ? 0 : j) + (lane & 7);
        const int p = 8 * (PR == 16 ? j : 0) + 2 * (lane >> 4) + ((lane >> 3) & 1);
        const bf16x8 f = bS_buf[0][r >> 4][p >> 2][16 * (p & 3) + (r & 15)];
        __builtin_nontemporal_store(
            f, reinterpret_cast<bf16x8*>(statesT + ((sp.slot0 + n) * DV + v0 + r) * DK + 8 * p));
      }
    };
    publish();
    // X of a later chunk touched line by line, a share by each S wave in its idle
    // phase, so that the Y waves' loads half a chunk ahead find it in L2
    uint32_t warm = 0, seen = 0;
    run([&](const uint16_t* __restrict__ cur, const uint16_t*, int n) {
      sync();  // A
      seen |= warm;
      {
        constexpr int LINES = kGatedX * 2 / 128 / S::NSW;
        const int m = n + 3 < nc ? n + 3 : nc - 1;
        const auto* line = reinterpret_cast<const uint32_t*>(xfr + (sp.slot0 + m) * kGatedX) + 32 * (LINES * sw + (lane < LINES ? lane : LINES - 1));
        warm = *line;
      }
      Frag<uint16_t> KT[2][NKU_C];
      const float end = gates(cur)[64 + 63];
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int kt = 0; kt < NKU_C; ++kt) KT[d][kt] = wide_frag_tr<DK>(cur + S::KOFF, 2 * sw + d, kt, lane);
      if constexpr (!OUT) save(n);
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) {
            St[d][c][qq] *= end;
            asm volatile("" : "+v"(St[d][c][qq]));  // here, not past the barrier, where S is the chunk's critical work
          }
      sync();  // M
      sync();  // B
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int kt = 0; kt < NKU_C; ++kt) {
          Frag<uint16_t> wh, wl;
          wh.v = bW_buf[0][c][kt][lane];
          wl.v = bW_buf[1][c][kt][lane];
#pragma unroll
          for (int d = 0; d < 2; ++d) mma(St[d][c], KT[d][kt], wl);
#pragma unroll
          for (int d = 0; d < 2; ++d) mma(St[d][c], KT[d][kt], wh);
        }
      publish();
    });
    if (seen == 0x7fc1a5e3u && lane == 64) ring[0] = 1;  // never: keeps the loads above
    if (OUT && a.sfin != nullptr && srow >= 0) {
      float* sf = a.sfin + (srow * H + h) * DK * DV + v0 + li;
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int qq = 0; qq < 4; ++qq)
            sf[int64_t(key_phys(16 * (2 * sw + d) + 4 * g + qq)) * DV + 16 * c] = St[d][c][qq];
    }
  } else if (role >= S::kO) {
    // ------------------------------------------------------------- output
    const int o_rh = role - S::kO, rt0 = 2 * o_rh;
    Frag<uint16_t> Qf[2][NKU_D];
    float eg[2];
    auto load = [&](const uint16_t* __restrict__ cur) {
#pragma unroll
      for (int r = 0; r < 2; ++r) eg[r] = gates(cur)[64 + 16 * (rt0 + r) + li];
#pragma unroll
      for (int ku = 0; ku < NKU_D; ++ku)
#pragma unroll
        for (int r = 0; r < 2; ++r) Qf[r][ku] = wide_frag<DK>(cur + S::QOFF, 16 * (rt0 + r) + li, ku, g);
    };
    run([&](const uint16_t* __restrict__ cur, const uint16_t*, int n) {
      sync();  // A
      load(cur);
      if (n > 0) store_staged(n - 1, o_rh);
      f32x4 Zt[NT][2];  // Zt[c][r][qq] = Z[16 (rt0 + r) + li][16 c + 4 g + qq]
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r) Zt[c][r] = zero4();
#pragma unroll
      for (int ku = 0; ku < NKU_D; ++ku)
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          Frag<uint16_t> bSo;
          bSo.v = bS_buf[0][c][ku][lane];
#pragma unroll
          for (int r = 0; r < 2; ++r) mma(Zt[c][r], bSo, Qf[r][ku]);
        }
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) Zt[c][r][qq] *= eg[r];
      sync();  // M
      sync();  // B
      Frag<uint16_t> bUo[NT][NKU_C];
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int ku = 0; ku < NKU_C; ++ku) bUo[c][ku].v = bU_buf[c][ku][lane];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int rt = rt0 + r;
        Frag<uint16_t> pf[NKU_C];
#pragma unroll
        for (int ku = 0; ku < NKU_C; ++ku)
          if (32 * ku <= 16 * rt + 15) pf[ku].v = P_buf[pf_index(rt, ku)][lane];
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          f32x4 acc = Zt[c][r];
#pragma unroll
          for (int ku = 0; ku < NKU_C; ++ku)
            if (32 * ku <= 16 * rt + 15) mma(acc, bUo[c][ku], pf[ku]);
          bf16x4 ov;
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) ov[qq] = static_cast<__bf16>(acc[qq]);
          *reinterpret_cast<bf16x4*>(&O_st[16 * rt + li][16 * c + 4 * g]) = ov;
        }
      }
    });
    // the last chunk's output: staged by both output waves before this barrier
    sync();
    if (nc > 0) store_staged(nc - 1, o_rh);
    return;
  } else {
    // ----------------------------------------------------------------- P
    // row tiles R0 .. R1 - 1 of P: 0-1, 2 and 3
    auto p_role = [&](auto r0c, auto r1c) {
      constexpr int R0 = decltype(r0c)::value, R1 = decltype(r1c)::value;
      f32x4 Pt[R1 - R0][R1];  // Pt[r - R0][c][qq] = P[16 r + li][16 c + 4 g + qq], c <= r
      auto clear = [&]() {
#pragma unroll
        for (int r = R0; r < R1; ++r)
#pragma unroll
          for (int c = 0; c <= r; ++c) Pt[r - R0][c] = zero4();
      };
      auto accumulate = [&](const uint16_t* __restrict__ cur, int k0, int k1) {
#pragma unroll
        for (int ku = 0; ku < NKU_D; ++ku) {
          if (ku < k0 || ku >= k1) continue;
          Frag<uint16_t> Qf[R1 - R0], Kf[R1];
#pragma unroll
          for (int r = R0; r < R1; ++r) Qf[r - R0] = wide_frag<DK>(cur + S::QOFF, 16 * r + li, ku, g);
#pragma unroll
          for (int c = 0; c < R1; ++c) Kf[c] = wide_frag<DK>(cur + S::KOFF, 16 * c + li, ku, g);
#pragma unroll
          for (int r = R0; r < R1; ++r)
#pragma unroll
            for (int c = 0; c <= r; ++c) mma(Pt[r - R0][c], Kf[c], Qf[r - R0]);
        }
      };
      clear();
      run([&](const uint16_t* __restrict__ cur, const uint16_t* __restrict__ nxt, int n) {
        sync();  // A
        if (n == 0) accumulate(cur, 0, KH);
        accumulate(cur, KH, NKU_D);
        sync();  // M
        const float* gt = gates(cur);
        f32x4 gc[R1];
#pragma unroll
        for (int c = 0; c < R1; ++c) gc[c] = *reinterpret_cast<const f32x4*>(gt + 16 * c + 4 * g);
#pragma unroll
        for (int r = R0; r < R1; ++r) {
          const float gr = gt[16 * r + li];
#pragma unroll
          for (int c = 0; c <= r; ++c)
#pragma unroll
            for (int qq = 0; qq < 4; ++qq)
              Pt[r - R0][c][qq] =
                  (c < r || 4 * g + qq <= li) ? Pt[r - R0][c][qq] * exp2_gate(gr - gc[c][qq]) : 0.0f;
#pragma unroll
          for (int ku = 0; ku < NKU_C; ++ku)
            if (32 * ku <= 16 * r + 15) {
              const f32x4 phi = (2 * ku + 1 <= r) ? Pt[r - R0][2 * ku + 1] : zero4();
              P_buf[pf_index(r, ku)][lane] = acc_frag<uint16_t>(Pt[r - R0][2 * ku], phi).v;
            }
        }
        sync();  // B
        clear();
        if (n + 1 < nc) accumulate(nxt, 0, KH);
      });
    };
    using std::integral_constant;
    if (role == S::kP) p_role(integral_constant<int, 0>{}, integral_constant<int, 2>{});
    else if (role == S::kP + 1) p_role(integral_constant<int, 2>{}, integral_constant<int, 3>{});
    else p_role(integral_constant<int, 3>{}, integral_constant<int, 4>{});
  }
  sync();  // with the output waves' last barrier
}

template <int DK>
__global__ __launch_bounds__((GatedSplitShape<DK>::THREADS)) void gated_split_kernel(
    GatedFwd a, const uint16_t* __restrict__ xfr, const float* __restrict__ gws, const int32_t* __restrict__ order,
    int NC, int NVB, int remap) {
  // arrays of their own: in one struct, where an exchange buffer's writes may be
  // writes to the ring for all the compiler knows, the forward is 2 us longer
  using S = GatedSplitShape<DK>;
  __shared__ __align__(1024) uint16_t ring[3 * S::SLOT];
  __shared__ __align__(16) bf16x8 bS_buf[2][S::NT][S::NKU_D][kWave];
  __shared__ __align__(16) bf16x8 bU_buf[S::NT][S::NKU_C][kWave];
  __shared__ __align__(16) bf16x8 bW_buf[2][S::NT][S::NKU_C][kWave];
  __shared__ __align__(16) bf16x8 bD_buf[2][S::NT][kWave];
  __shared__ __align__(16) bf16x8 P_buf[S::NPF][kWave];
  __shared__ __align__(16) uint16_t O_st[S::C][S::OP];
  const GatedSplitRefs<DK> lds{ring, bS_buf, bU_buf, bW_buf, bD_buf, P_buf, O_st};
  gated_split_run<DK, true>(lds, a, blockIdx.x, xfr, gws, order, NC, NVB, remap, nullptr);
}

}  // namespace efla
