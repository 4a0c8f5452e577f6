// gated_reverse.h -- the reverse pass over the chunks of the gated backward for
// bf16 inputs, in the form of recurrence_reverse.h.
//
// Per chunk, last to first, with dS' the loss gradient at the chunk's end, e =
// e^G, w = e^{G_C - G} and Qe = diag(e) Q - P T diag(e) K (gated_ut.h):
//     dstates[n] = dS'
//     E = diag(w) K dS',   F = diag(e) T^T E = diag(e a) X^T E
//     dS = e^{G_C} dS' + Qe^T dO - K^T F
// dS is held and summed in float32; as an operand it is rounded to bf16 once (it
// is read by products that end in bf16 gradients), as are E and F.
//
// Roles, barriers, ring schedule and the layout of dstates ([slots][d_v][d_k])
// are those of reverse_states_kernel; a chunk's gates ride in its ring slot (1
// KiB), the Y waves scale their accumulator rows by them, and the S waves scale
// dS by e^{G_C} before they add Qe^T dO.  Query and key heads may be shared.
// Bound like it by the chain dS, E, F, dS and the LDS reads of K and Qe: 51 us for
// 8 x 2048 tokens of 8 heads, d 128 (32 chunks, 1.6 us each), as a launch of its own;
// with the chunks' start states in one launch (below) 91 us.
#pragma once

#include <type_traits>

#include "gated.h"
#include "gated_ut.h"
#include "gated_split.h"
#include "lds_ring.h"

namespace efla {

template <int DK>
struct GatedReverseShape {
  static_assert(DK == 64 || DK == 128, "shapes of the gated reverse pass");
  static constexpr int C = 64, BV = 32;
  static constexpr int NT = BV / 16;  // dS tiles per workgroup
  static constexpr int NRT = C / 16, NKU_D = DK / 32, NKU_C = C / 32;
  static constexpr int NSW = NKU_D;  // S waves, 32 key dims each
  static constexpr int KOFF = 0, QOFF = C * DK, XOFF = 2 * C * DK, OOFF = 2 * C * DK + kGatedX / 2;
  static constexpr int GOFF = OOFF + C * BV;
  static constexpr int SLOT = GOFF + kGatedG * 2;  // in bf16 elements
  using TK = DmaTile<C, DK, 1, true>;  // K and Qe: 16-byte-fragment swizzle
  using TO = DmaTile<C, BV, 1>;
  static constexpr int PK = TK::PER_WAVE, PX = kGatedX / 2 * 2 / 1024, PO = TO::PER_WAVE;
  static constexpr int COUNT = 2 * PK + PX + PO + 1;  // transfers per chunk
  static constexpr int kY0 = 0, kS0 = 2, kDma = 2 + NSW, NWAVES = 3 + NSW, THREADS = NWAVES * kWave;
};

template <int DK>
struct GatedReverseLds {
  using S = GatedReverseShape<DK>;
  alignas(1024) uint16_t ring[3 * S::SLOT];
  alignas(16) bf16x8 bS_buf[S::NT][S::NKU_D][kWave];  // dS' as operand fragments
  alignas(16) bf16x8 bF_buf[S::NT][S::NKU_C][kWave];  // -F as operand fragments
};

// dense batch; workgroup x of NVB = DV / BV per (b, h).
template <int DK>
__device__ __forceinline__ void gated_reverse_run(GatedReverseLds<DK>& lds, const GatedBwd& b, const int x,
                                                  const uint16_t* __restrict__ qe, const uint16_t* __restrict__ xfr,
                                                  const float* __restrict__ gws, uint16_t* __restrict__ dstatesT,
                                                  int NC, int NVB, int remap) {
  using S = GatedReverseShape<DK>;
  constexpr int C = S::C, BV = S::BV, NT = S::NT, NRT = S::NRT, NKU_D = S::NKU_D, NKU_C = S::NKU_C;
  uint16_t* const ring = lds.ring;
  uint16_t* const slot0 = ring;
  uint16_t* const slot1 = ring + S::SLOT;
  uint16_t* const slot2 = ring + 2 * S::SLOT;
  auto& bS_buf = lds.bS_buf;
  auto& bF_buf = lds.bF_buf;

  const auto* k = static_cast<const uint16_t*>(b.k);
  const auto* dout = static_cast<const uint16_t*>(b.d_o);
  int bh, vb;
  if (remap) {  // all value blocks of one (b, h) on one XCD (same blockIdx % 8)
    const int slot = x >> 3;
    vb = slot % NVB;
    bh = (slot / NVB) * 8 + (x & 7);
  } else {
    bh = x / NVB;
    vb = x % NVB;
  }
  const int H = b.H, DV = b.DV;
  const int64_t h = bh % H, hk = h / (H / b.Hk);
  const SeqSpan sp = seq_span<C>(nullptr, bh / H, h, H, b.L, NC);
  const int nc = sp.nc;
  const int v0 = vb * BV;
  const int lane = threadIdx.x & 63, role = wave_id(), li = lane & 15, g = lane >> 4;
  // step n processes chunk nc - 1 - n
  auto chunk_of = [&](int n) { return nc - 1 - n; };
  auto chunk_valid = [&](int m) { return int(sp.len - int64_t(m) * C < C ? sp.len - int64_t(m) * C : C); };
  auto tok_of = [&](int m) { return sp.bos + int64_t(m) * C; };
  auto gates = [&](const uint16_t* cur) { return reinterpret_cast<const float*>(cur + S::GOFF); };
  auto sync = [&]() {
    wait_lgkm0();
    barrier_nowait();
  };
  auto run = [&](auto&& step) {  // steps of three keep the ring slots compile-time addresses
    for (int n = 0; n < nc; n += 3) {
      step(slot0, n);
      if (n + 1 < nc) step(slot1, n + 1);
      if (n + 2 < nc) step(slot2, n + 2);
    }
  };

  if (role == S::kDma) {
    // ---------------------------------------------------------------- DMA
    // The forward pass's schedule (recurrence_split.h): step n+3's chunk goes
    // into step n's slot half after barrier B of step n and half after
    // barrier A of step n+1; before barrier B of step n only step n+2's
    // transfers may remain (waits counted against one chunk's transfers).
    constexpr int D = S::COUNT;
    static_assert(D < 64, "one chunk's transfers fit the vmcnt counter");
    typename S::TK tk, tq;
      typename S::TO to;
    tk.init(int64_t(b.Hk) * DK, lane, 0);
    tq.init(DK, lane, 0);
      to.init(int64_t(H) * DV, lane, 0);
    auto issue = [&](int n, int part, int parts) {
      const int m = chunk_of(n);
      const auto* ks = static_cast<const uint16_t*>(uniform_ptr(k + (tok_of(m) * b.Hk + hk) * DK));
      const auto* qs = static_cast<const uint16_t*>(uniform_ptr(qe + (sp.slot0 + m) * C * DK));
      const void* xs = uniform_ptr(xfr + (sp.slot0 + m) * kGatedX);  // the high parts
      const auto* os = static_cast<const uint16_t*>(uniform_ptr(dout + (tok_of(m) * H + h) * DV + v0));
      const void* gsrc = uniform_ptr(gws + (sp.slot0 + m) * kGatedG);
      const int valid = chunk_valid(m);
      const uint32_t addr = lds_addr_of(ring + (n % 3) * S::SLOT);
      auto body = [&](auto ragged) {
        constexpr bool R = decltype(ragged)::value;
#pragma unroll
        for (int j = 0; j < D; ++j) {
          if (j < part * D / parts || j >= (part + 1) * D / parts) continue;
          if (j < S::PK) tk.template issue<R>(j, addr + 2 * S::KOFF, ks, valid);
          else if (j < 2 * S::PK) tq.template issue<false>(j - S::PK, addr + 2 * S::QOFF, qs, C);
          else if (j < 2 * S::PK + S::PX) dma16(xs, uint32_t(j - 2 * S::PK) * 1024u + uint32_t(lane) * 16u, addr + 2 * S::XOFF + 1024 * (j - 2 * S::PK));
          else if (j < D - 1) to.template issue<R>(j - 2 * S::PK - S::PX, addr + 2 * S::OOFF, os, valid);
          else dma16(gsrc, uint32_t(lane) * 16u, addr + 2 * S::GOFF);
        }
      };
      if (valid == C) body(std::false_type{});
      else body(std::true_type{});
    };
    if (nc > 0) issue(0, 0, 1);
    if (nc > 1) {
      issue(1, 0, 1);
      wait_vmcnt<D>();  // step 0's chunk complete
    } else {
      wait_vmcnt<0>();
    }
    if (nc > 2) issue(2, 0, 2);
    for (int n = 0; n < nc; ++n) {
      barrier_nowait();  // A
      if (n + 2 < nc) issue(n + 2, 1, 2);
      if (n + 2 < nc) wait_vmcnt<D>();  // step n+1's chunk complete
      else wait_vmcnt<0>();
      barrier_nowait();  // B
      if (n + 3 < nc) issue(n + 3, 0, 2);
    }
    wait_vmcnt<0>();
  } else if (role < S::kS0) {
    // ----------------------------------------------------------------- Y
    const int ct = role - S::kY0;
    Frag<uint16_t> Kf[NRT][NKU_D];
    Frag<uint16_t> Xf[NRT][NKU_C];  // X^T: row tile rt, k-unit ku (X^T is upper triangular: ku >= rt / 2)
    f32x4 eg[NRT], wg[NRT];
    auto load = [&](const uint16_t* __restrict__ cur) {
      const uint16_t* Ks = cur + S::KOFF;
      const uint16_t* Xs = cur + S::XOFF;
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt) {
        eg[rt] = *reinterpret_cast<const f32x4*>(gates(cur) + 64 + 16 * rt + 4 * g) *
                 *reinterpret_cast<const f32x4*>(gates(cur) + 192 + 16 * rt + 4 * g);
        wg[rt] = *reinterpret_cast<const f32x4*>(gates(cur) + 128 + 16 * rt + 4 * g);
      }
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
        for (int ku = 0; ku < NKU_C; ++ku)
          if (32 * ku + 31 >= 16 * rt) Xf[rt][ku] = tri_frag_tr(Xs, rt, ku, lane);
#pragma unroll
      for (int ku = 0; ku < NKU_D; ++ku)
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt) Kf[rt][ku] = wide_frag<DK>(Ks, 16 * rt + li, ku, g);
    };
    for (int n = 0; n < nc; ++n) {
      const int sn = n % 3;
      sync();  // A
      if (n == 0) load(ring);
      Frag<uint16_t> bS[NKU_D];
#pragma unroll
      for (int ku = 0; ku < NKU_D; ++ku) bS[ku].v = bS_buf[ct][ku][lane];
      f32x4 E[NRT];
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt) E[rt] = zero4();
#pragma unroll
      for (int ku = 0; ku < NKU_D; ++ku)
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt) mma(E[rt], Kf[rt][ku], bS[ku]);
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) E[rt][qq] *= wg[rt][qq];
      Frag<uint16_t> bE[NKU_C];
#pragma unroll
      for (int ku = 0; ku < NKU_C; ++ku) bE[ku] = acc_frag<uint16_t>(E[2 * ku], E[2 * ku + 1]);
#pragma unroll
      for (int ku = 0; ku < NKU_C; ++ku) {
        f32x4 F0 = zero4(), F1 = zero4();
#pragma unroll
        for (int kk = ku; kk < NKU_C; ++kk) {
          mma(F0, Xf[2 * ku][kk], bE[kk]);
          mma(F1, Xf[2 * ku + 1][kk], bE[kk]);
        }
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {
          F0[qq] *= -eg[2 * ku][qq];
          F1[qq] *= -eg[2 * ku + 1][qq];
        }
        bF_buf[ct][ku][lane] = acc_frag<uint16_t>(F0, F1).v;
      }
      sync();  // B
      if (n + 1 < nc) load(ring + (sn == 2 ? 0 : (sn + 1) * S::SLOT));
    }
  } else {
    // ----------------------------------------------------------------- S
    // rows: logical key dims 32 s .. 32 s + 31 of dS
    const int sw = role - S::kS0, col0 = v0;
    // St[d][c][qq] = dS[key_phys(16 (2 sw + d) + 4 g + qq)][col0 + 16 c + li]
    f32x4 St[2][NT];
#pragma unroll
    for (int d = 0; d < 2; ++d)
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {
          const int key = key_phys(16 * (2 * sw + d) + 4 * g + qq);
          St[d][c][qq] = b.dsf != nullptr ? b.dsf[(int64_t(bh) * DK + key) * DV + col0 + 16 * c + li] : 0.0f;
        }
    // dS' as operand fragments: fragment c holds key dims 32 sw + 8 g .. + 7
    // of column col0 + 16 c + li
    auto publish = [&]() {
#pragma unroll
      for (int c = 0; c < NT; ++c) bS_buf[c][sw][lane] = acc_frag<uint16_t>(St[0][c], St[1][c]).v;
    };
    // dstates[m] (m: the chunk of this step, whose end-gradient the buffer
    // holds), from the fragments every S wavefront published: this wavefront
    // stores its share of the rows of dS'^T (8 with d_k 128, 16 with d_k 64),
    // each instruction 8 rows x 128 contiguous bytes (two lanes per bank in
    // each 16-lane read group), nontemporal; every row is written whole
    // (from the registers, 64-byte pieces from several wavefronts wrote 1.16x
    // the bytes)
    auto save = [&](int m) {
      constexpr int PR = DK / 8, RW = BV / NKU_D;  // 16-byte pieces per row, rows per S wavefront
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = RW * sw + 8 * (PR == 16 ? 0 : j) + (lane & 7);
        const int p = 8 * (PR == 16 ? j : 0) + 2 * (lane >> 4) + ((lane >> 3) & 1);
        const bf16x8 f = bS_buf[r >> 4][p >> 2][16 * (p & 3) + (r & 15)];
        __builtin_nontemporal_store(
            f, reinterpret_cast<bf16x8*>(dstatesT + ((sp.slot0 + m) * DV + col0 + r) * DK + 8 * p));
      }
    };
    publish();
    run([&](const uint16_t* __restrict__ cur, int n) {
      sync();  // A
      save(chunk_of(n));
      const float end = gates(cur)[64 + 63];
      Frag<uint16_t> KT[2][NKU_C], QT[2][NKU_C], dOf[NT][NKU_C];
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int kt = 0; kt < NKU_C; ++kt) {
          KT[d][kt] = wide_frag_tr<DK>(cur + S::KOFF, 2 * sw + d, kt, lane);
          QT[d][kt] = wide_frag_tr<DK>(cur + S::QOFF, 2 * sw + d, kt, lane);
        }
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int kt = 0; kt < NKU_C; ++kt) dOf[c][kt] = sw_frag_tr<BV>(cur + S::OOFF, 16 * c, kt, lane);
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int c = 0; c < NT; ++c) {
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) St[d][c][qq] *= end;
#pragma unroll
          for (int kt = 0; kt < NKU_C; ++kt) mma(St[d][c], QT[d][kt], dOf[c][kt]);
        }
      sync();  // B
      Frag<uint16_t> bF[NT][NKU_C];
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int kt = 0; kt < NKU_C; ++kt) bF[c][kt].v = bF_buf[c][kt][lane];
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int kt = 0; kt < NKU_C; ++kt) mma(St[d][c], KT[d][kt], bF[c][kt]);
      publish();
    });
    if (b.ds0 != nullptr) {
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int qq = 0; qq < 4; ++qq)
            b.ds0[(int64_t(bh) * DK + key_phys(16 * (2 * sw + d) + 4 * g + qq)) * DV + col0 + 16 * c + li] =
                St[d][c][qq];
    }
  }
}

// The reverse pass and the chunks' start states (gated_split.h), which do not need
// each other, in one launch: the first half of the workgroups runs the one, the
// second the other.  Where neither fills the GPU they run side by side (8 heads
// of 515 tokens, d 64: two launches took 11.0 and 8.7 us); where both do (256
// workgroups each at the 340M layer) they follow each other as before.
template <int DK>
union GatedChainsLds {
  GatedSplitLds<DK> states;
  GatedReverseLds<DK> reverse;
};
template <int DK>
__global__ __launch_bounds__((GatedSplitShape<DK>::STATE_THREADS)) void gated_chains_kernel(
    GatedFwd a, GatedBwd b, const uint16_t* __restrict__ qe, const uint16_t* __restrict__ xfr,
    const float* __restrict__ gws, uint16_t* __restrict__ statesT, uint16_t* __restrict__ dstatesT, int NC, int NVB,
    int remap) {
  static_assert(GatedReverseShape<DK>::THREADS <= GatedSplitShape<DK>::STATE_THREADS, "one shape for both");
  __shared__ GatedChainsLds<DK> lds;
  const int half = int(gridDim.x >> 1), x = int(blockIdx.x);
  if (x >= half) {
    gated_split_run<DK, false>(lds.states, a, x - half, xfr, gws, nullptr, NC, NVB, remap, statesT);
  } else if (wave_id() < GatedReverseShape<DK>::NWAVES) {  // the others end here and leave its barriers
    gated_reverse_run<DK>(lds.reverse, b, x, qe, xfr, gws, dstatesT, NC, NVB, remap);
  }
}

}  // namespace efla
