// gated_split.h -- the sequential chunk pass of the gated delta rule for bf16
// inputs, each chunk's work spread over eight wavefronts, with the state good
// to 16 significant bits or more.
//
// Per chunk (start state S, T from gated_ut.h; e = e^G, w = e^{G_C - G}):
//     U = T (V - diag(e) K S),   S <- e^{G_C} S + K^T diag(w) U,
//     O = diag(e) Q S + (Gam * tril(Q K^T)) U
// q, k and v are bf16, so their products are exact in float32 sums; what would
// be lost is the rounding of S, of D = V - diag(e) K S, of T and of U where
// they are operands (2^-8 each).  On the way to the state they therefore go in
// as two bf16 parts (hi + lo, 2^-16): K S and K^T U twice, T D three times
// (lo lo dropped).  On the way to o, which is rounded to bf16 anyway, the high
// parts alone go in.
//
// A workgroup owns 32 value columns (two 16-column tiles) of one (sequence,
// head).  The roles are those of recurrence_split.h:
//   Y wave per tile      Y = K S, D, U = T D; publishes U (for O) and
//                        diag(w) U in two parts (for S)
//   S wave per half of   S <- e^{G_C} S + K^T (diag(w) U) in fp32 registers;
//   the key dimension    publishes S in two parts
//   O wave per half of   Z^T = S^T Q^T, then O^T = diag(e) Z^T + U^T P^T, staged
//   the chunk's rows     in LDS and stored a chunk later
//   P wave               Gam * tril(Q K^T), half of the key dimension a phase
//   DMA wave             Q, K, V and the chunk's gates into a three-slot ring
// T does not pass the LDS: it comes in fragment order, 12 KiB a chunk, and the
// Y waves load it into registers two chunks ahead.  That is what makes eight
// wavefronts (two a SIMD, 256 VGPRs) the right number here: the Y waves hold
// two chunks' T besides the chunk's K.
// Two barriers a chunk, every exchange buffer written in one phase and read in
// the other:
//   A (chunk n in LDS, S_n published)
//     Y: products -> publish U | S: read K^T | O: Z^T | P: finish -> publish | DMA: half of chunk n+2
//   B (U and P published, chunk n+1 in LDS)
//     Y: read K, V of n+1, load T of n+2 | S: update -> publish | O: O^T, read Q of n+1 | P: start n+1 | DMA
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
  // by wavefront index (SIMD = index % 4): the chain's four on a SIMD each
  static constexpr int kS0 = 0, kY0 = 1, kY1 = 2, kS1 = 3, kP = 4, kO0 = 5, kO1 = 6, kDma = 7;
  static constexpr int THREADS = 8 * kWave;
};

// OUT: writes o and the final state.  Else (the backward's recomputation) the
// state at the start of every chunk instead, as the high operand parts,
// transposed, [slots][DV][DK] (the layout of recurrence_split.h); the O and P
// waves idle and Q is not brought in.
template <int DK, bool OUT>
__global__ __launch_bounds__(512) void gated_split_kernel(GatedFwd a, const uint16_t* __restrict__ tfr,
                                                          const float* __restrict__ gws,
                                                          const int32_t* __restrict__ order, int NC, int NVB, int remap,
                                                          uint16_t* __restrict__ statesT) {
  using S = GatedSplitShape<DK>;
  constexpr int C = S::C, BV = S::BV, NT = S::NT, NRT = S::NRT, NKU_D = S::NKU_D, NKU_C = S::NKU_C, KH = S::KH;
  __shared__ __align__(1024) uint16_t ring[3 * S::SLOT];
  uint16_t* const slot0 = ring;
  uint16_t* const slot1 = ring + S::SLOT;
  uint16_t* const slot2 = ring + 2 * S::SLOT;
  __shared__ __align__(16) bf16x8 bS_buf[2][NT][NKU_D][kWave];  // S_n, high and low parts
  __shared__ __align__(16) bf16x8 bU_buf[NT][NKU_C][kWave];     // U_n, high parts
  __shared__ __align__(16) bf16x8 bW_buf[2][NT][NKU_C][kWave];  // diag(w) U_n, high and low parts
  __shared__ __align__(16) bf16x8 P_buf[S::NPF][kWave];
  __shared__ __align__(16) uint16_t O_st[C][S::OP];

  const int H = a.H, DV = a.DV;
  const int x = blockIdx.x;
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
        wait_vmcnt<D>();  // chunk n+1 complete: only chunk n+2's transfers remain
      } else {
        wait_vmcnt<0>();
      }
      barrier_nowait();  // B
      if (n + 3 < nc) issue(n + 3, 0, 2);
    }
    wait_vmcnt<0>();
  } else if (role == S::kY0 || role == S::kY1) {
    // ----------------------------------------------------------------- Y
    const int ct = role == S::kY1 ? 1 : 0;
    Frag<uint16_t> Kf[NRT][NKU_D];
    bf16x4 Vt[NRT];
    f32x4 eg[NRT];
    struct TFrag {
      Frag<uint16_t> h[6], l[6];
    } T;
    auto load_t = [&](int m) {
      const bf16x8* src = reinterpret_cast<const bf16x8*>(tfr + (sp.slot0 + (m < nc ? m : nc - 1)) * kGatedT) + lane;
#pragma unroll
      for (int f = 0; f < 6; ++f) {
        T.h[f].v = src[f * 64];
        T.l[f].v = src[(6 + f) * 64];
      }
    };
    auto load = [&](const uint16_t* __restrict__ cur) {  // this chunk's K, gates and this tile's V
      const uint16_t* Ks = cur + S::KOFF;
      const uint16_t* Vs = cur + S::VOFF;
      const float* gt = gates(cur);
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt) {
        Vt[rt] = lds_read_tr(Vs + swz_off<BV>(16 * rt + 4 * g + (li >> 2), 16 * ct + 4 * (li & 3)));
        eg[rt] = *reinterpret_cast<const f32x4*>(gt + 64 + 16 * rt + 4 * g);
      }
#pragma unroll
      for (int ku = 0; ku < NKU_D; ++ku)
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt) Kf[rt][ku] = wide_frag<DK>(Ks, 16 * rt + li, ku, g);
    };
    auto step = [&](int n) {
      sync();  // A
      if (n == 0) load(ring);
      Frag<uint16_t> sh[NKU_D], sl[NKU_D];
#pragma unroll
      for (int ku = 0; ku < NKU_D; ++ku) {
        sh[ku].v = bS_buf[0][ct][ku][lane];
        sl[ku].v = bS_buf[1][ct][ku][lane];
      }
      f32x4 Y[NRT];
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt) Y[rt] = zero4();
#pragma unroll
      for (int ku = 0; ku < NKU_D; ++ku) {
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt) mma(Y[rt], Kf[rt][ku], sh[ku]);
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt) mma(Y[rt], Kf[rt][ku], sl[ku]);
      }
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) Y[rt][qq] = fmaf(-eg[rt][qq], Y[rt][qq], static_cast<float>(Vt[rt][qq]));
      Frag<uint16_t> dh[NKU_C], dl[NKU_C];
#pragma unroll
      for (int ku = 0; ku < NKU_C; ++ku) split_frag(Y[2 * ku], Y[2 * ku + 1], dh[ku], dl[ku]);
      f32x4 U[NRT], wg[NRT];  // w read here: held from load() on, the registers would spill
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt) {
        U[rt] = zero4();
        wg[rt] = *reinterpret_cast<const f32x4*>(gates(ring + (n % 3) * S::SLOT) + 128 + 16 * rt + 4 * g);
      }
#pragma unroll
      for (int kk = 0; kk < NKU_C; ++kk) {
#pragma unroll
        for (int rt = 2 * kk; rt < NRT; ++rt) mma(U[rt], T.l[pf_index(rt, kk)], dh[kk]);
#pragma unroll
        for (int rt = 2 * kk; rt < NRT; ++rt) mma(U[rt], T.h[pf_index(rt, kk)], dl[kk]);
#pragma unroll
        for (int rt = 2 * kk; rt < NRT; ++rt) mma(U[rt], T.h[pf_index(rt, kk)], dh[kk]);
      }
#pragma unroll
      for (int ku = 0; ku < NKU_C; ++ku) {
        if constexpr (OUT) bU_buf[ct][ku][lane] = acc_frag<uint16_t>(U[2 * ku], U[2 * ku + 1]).v;
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {
          U[2 * ku][qq] *= wg[2 * ku][qq];
          U[2 * ku + 1][qq] *= wg[2 * ku + 1][qq];
        }
        Frag<uint16_t> wh, wl;
        split_frag(U[2 * ku], U[2 * ku + 1], wh, wl);
        bW_buf[0][ct][ku][lane] = wh.v;
        bW_buf[1][ct][ku][lane] = wl.v;
      }
      sync();  // B
      // Past the last chunk the loads go on, from the last chunk's slot and
      // whatever the ring holds, and nothing reads what they bring: behind a
      // branch, the loaded registers would be merged with the old ones, with a
      // wait there.
      load_t(n + 1);
      load(ring + ((n + 1) % 3) * S::SLOT);
    };
    if (nc > 0) load_t(0);
    for (int n = 0; n < nc; ++n) step(n);
  } else if (role == S::kS0 || role == S::kS1) {
    // ----------------------------------------------------------------- S
    // rows: logical key dims 64 hh .. (k-units KH hh .. KH hh + KH - 1)
    const int hh = role == S::kS1 ? 1 : 0, dt0 = 2 * KH * hh, ku0 = KH * hh;
    f32x4 St[2 * KH][NT];  // St[d][c][qq] = S[key_phys(16 (dt0 + d) + 4 g + qq)][v0 + 16 c + li]
    const float* s0 = a.s0 == nullptr || srow < 0 ? nullptr : a.s0 + (srow * H + h) * DK * DV + v0 + li;
#pragma unroll
    for (int d = 0; d < 2 * KH; ++d)
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int qq = 0; qq < 4; ++qq)
          St[d][c][qq] = s0 != nullptr ? s0[int64_t(key_phys(16 * (dt0 + d) + 4 * g + qq)) * DV + 16 * c] : 0.0f;
    auto publish = [&]() {
#pragma unroll
      for (int u = 0; u < KH; ++u)
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          Frag<uint16_t> sh, sl;
          split_frag(St[2 * u][c], St[2 * u + 1][c], sh, sl);
          bS_buf[0][c][ku0 + u][lane] = sh.v;
          bS_buf[1][c][ku0 + u][lane] = sl.v;
        }
    };
    auto save = [&](int n) {  // chunk n's start state, whole rows of S^T (recurrence_split.h)
      constexpr int PR = DK / 8;
#pragma unroll
      for (int j = 0; j < PR / 4; ++j) {
        const int rr = 8 * (j / (PR / 8)) + (lane & 7);
        const int p = 8 * (j % (PR / 8)) + 2 * (lane >> 4) + ((lane >> 3) & 1);
        const bf16x8 f = bS_buf[0][hh][p >> 2][16 * (p & 3) + rr];
        __builtin_nontemporal_store(
            f, reinterpret_cast<bf16x8*>(statesT + ((sp.slot0 + n) * DV + v0 + 16 * hh + rr) * DK + 8 * p));
      }
    };
    publish();
    // T of a later chunk touched line by line, 6 KiB by each S wave in its idle
    // phase, so that the Y waves' loads half a chunk ahead find it in L2
    uint32_t warm = 0, seen = 0;
    run([&](const uint16_t* __restrict__ cur, const uint16_t*, int n) {
      sync();  // A
      seen |= warm;
      {
        const int m = n + 3 < nc ? n + 3 : nc - 1;
        const auto* line = reinterpret_cast<const uint32_t*>(tfr + (sp.slot0 + m) * kGatedT) + 32 * (48 * hh + (lane < 48 ? lane : 47));
        warm = *line;
      }
      Frag<uint16_t> KT[2 * KH][NKU_C];
      const float end = gates(cur)[64 + 63];
#pragma unroll
      for (int d = 0; d < 2 * KH; ++d)
#pragma unroll
        for (int kt = 0; kt < NKU_C; ++kt) KT[d][kt] = wide_frag_tr<DK>(cur + S::KOFF, dt0 + d, kt, lane);
      if constexpr (!OUT) save(n);
#pragma unroll
      for (int d = 0; d < 2 * KH; ++d)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) {
            St[d][c][qq] *= end;
            asm volatile("" : "+v"(St[d][c][qq]));  // here, not past the barrier, where S is the chunk's critical work
          }
      sync();  // B
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int kt = 0; kt < NKU_C; ++kt) {
          Frag<uint16_t> wh, wl;
          wh.v = bW_buf[0][c][kt][lane];
          wl.v = bW_buf[1][c][kt][lane];
#pragma unroll
          for (int d = 0; d < 2 * KH; ++d) mma(St[d][c], KT[d][kt], wl);
#pragma unroll
          for (int d = 0; d < 2 * KH; ++d) mma(St[d][c], KT[d][kt], wh);
        }
      publish();
    });
    if (seen == 0x7fc1a5e3u && lane == 64) ring[0] = 1;  // never: keeps the loads above
    if (OUT && a.sfin != nullptr && srow >= 0) {
      float* sf = a.sfin + (srow * H + h) * DK * DV + v0 + li;
#pragma unroll
      for (int d = 0; d < 2 * KH; ++d)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int qq = 0; qq < 4; ++qq)
            sf[int64_t(key_phys(16 * (dt0 + d) + 4 * g + qq)) * DV + 16 * c] = St[d][c][qq];
    }
  } else if (!OUT) {
    for (int n = 0; n < nc; ++n) {
      barrier_nowait();
      barrier_nowait();
    }
  } else if (role == S::kO0 || role == S::kO1) {
    // ------------------------------------------------------------- output
    const int o_rh = role == S::kO1 ? 1 : 0, rt0 = 2 * o_rh;
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
    run([&](const uint16_t* __restrict__ cur, const uint16_t* __restrict__ nxt, int n) {
      sync();  // A
      if (n == 0) load(cur);
      else store_staged(n - 1, o_rh);
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
      if (n + 1 < nc) load(nxt);
    });
    // the last chunk's output: staged by both output waves before this barrier
    sync();
    if (nc > 0) store_staged(nc - 1, o_rh);
    return;
  } else {
    // ----------------------------------------------------------------- P
    f32x4 Pt[NRT][NRT];  // Pt[r][c][qq] = P[16 r + li][16 c + 4 g + qq], c <= r
    auto clear = [&]() {
#pragma unroll
      for (int r = 0; r < NRT; ++r)
#pragma unroll
        for (int c = 0; c <= r; ++c) Pt[r][c] = zero4();
    };
    auto accumulate = [&](const uint16_t* __restrict__ cur, int ku0, int ku1) {
#pragma unroll
      for (int ku = 0; ku < NKU_D; ++ku) {
        if (ku < ku0 || ku >= ku1) continue;
        Frag<uint16_t> Qf[NRT], Kf[NRT];
#pragma unroll
        for (int r = 0; r < NRT; ++r) {
          Qf[r] = wide_frag<DK>(cur + S::QOFF, 16 * r + li, ku, g);
          Kf[r] = wide_frag<DK>(cur + S::KOFF, 16 * r + li, ku, g);
        }
#pragma unroll
        for (int r = 0; r < NRT; ++r)
#pragma unroll
          for (int c = 0; c <= r; ++c) mma(Pt[r][c], Kf[c], Qf[r]);
      }
    };
    clear();
    run([&](const uint16_t* __restrict__ cur, const uint16_t* __restrict__ nxt, int n) {
      sync();  // A
      if (n == 0) accumulate(cur, 0, KH);
      accumulate(cur, KH, NKU_D);
      const float* gt = gates(cur);
      f32x4 gc[NRT];
#pragma unroll
      for (int c = 0; c < NRT; ++c) gc[c] = *reinterpret_cast<const f32x4*>(gt + 16 * c + 4 * g);
#pragma unroll
      for (int r = 0; r < NRT; ++r) {
        const float gr = gt[16 * r + li];
#pragma unroll
        for (int c = 0; c <= r; ++c)
#pragma unroll
          for (int qq = 0; qq < 4; ++qq)
            Pt[r][c][qq] = (c < r || 4 * g + qq <= li) ? Pt[r][c][qq] * exp2_gate(gr - gc[c][qq]) : 0.0f;
#pragma unroll
        for (int ku = 0; ku < NKU_C; ++ku)
          if (32 * ku <= 16 * r + 15) {
            const f32x4 phi = (2 * ku + 1 <= r) ? Pt[r][2 * ku + 1] : zero4();
            P_buf[pf_index(r, ku)][lane] = acc_frag<uint16_t>(Pt[r][2 * ku], phi).v;
          }
      }
      sync();  // B
      clear();
      if (n + 1 < nc) accumulate(nxt, 0, KH);
    });
  }
  sync();  // with the output waves' last barrier
}

}  // namespace efla
