// gated_bwd_chunk.h -- the per-chunk gradients of the gated backward for bf16
// inputs, two workgroups per compute unit, in the form of bwd_chunk_tr.h (every
// operand held once as a swizzled bf16 tile, read as rows or by transposing
// reads; value blocks of 32 columns by direct transfers; eight wavefronts at
// 128 VGPRs).
//
// The formulas are gated_bwd.h's.  What the gates add, and where it fits:
//   * D = V - diag(e) K S and dU = P^T dO + diag(w) K dS' scale accumulator rows.
//   * dK = diag(w) U dS'^T - diag(e) dD S^T: U and dD are needed unscaled too (for
//     dP and dv), so the scaled operands are tiles of their own, rounded from the
//     accumulators like the unscaled ones; diag(w) U takes V's place, which is
//     read in the block's first phase alone, and V of the next block is fetched
//     with the block's other operands.
//   * Row sums for dg.  k_i . Y3_i = sum_c dD_ic (e K S)_ic and k_j . Y2_j = sum_c
//     U_jc (w K dS')_jc: both factors sit in the same wavefront's accumulators
//     one phase apart, so no product is added; q_i . Y1_i comes from dQ's
//     accumulators before dP K is added.  <dS', S> is summed from the tiles.
//   * M = dP0 * P + diag(a) N of gated_bwd.h: Q K^T is formed once more in fp32
//     at the end (P itself was rounded to bf16), on the tiles that hold dP.
//   * Gam is formed from G as one float (gated_ut.h), not two: behind 48 resets in a
//     chunk its entries are off by up to 7e-4, below the 2^-8 of the roundings to
//     bf16 around it.  Measured behind 0 / 48 resets: dq 3.3e-3 / 3.5e-3, dk 3.4e-3 /
//     3.5e-3, dv 3.0e-3 / 2.8e-3, dbeta 2.7e-3 / 3.3e-3, dg 2.5e-3 / 1.6e-3.
// Every product is formed transposed: an accumulator tile then holds, in one lane,
// four consecutive columns of one row (token), so tiles are written to the LDS
// and rows of K and Q read beside them as 8-byte pieces (4 elements) instead of
// one by one, a row's gate is one value a lane, and a row sum is three adds and
// two lane exchanges.
// Shared key heads (SHARED): dq and dk of every value head leave in fp32, and
// gated_head_sum_kernel adds them up.
// X and P stay in fragment order in the LDS (gated_ut.h); T is not held: a scales
// D's and dV's rows instead, so the sum over D and dU is dX itself, and da needs
// the row sums of (X^T dU) D alone, both in registers.
// 80 KiB of LDS.  8 x 2048 tokens of 8 heads, d 128: 121 us (133 to 160 in a process's
// first launches), four rounds of 30 us at two workgroups to a compute unit.  Bound
// by latency: between its 18 barriers four wavefronts a SIMD keep the vector unit
// busy 0.55, the LDS 0.57 (a third of it conflicts of transposing reads) and the matrix unit 0.14
// of the time; an accumulator tile spills in the loop (24 bytes a lane; 2 registers
// of it where key heads are shared).  In LDS places without those conflicts X and P
// cost more address arithmetic than they save (267 us of the whole backward for 260).
#pragma once

#include <type_traits>

#include "bwd_chunk_tr.h"
#include "gated.h"
#include "gated_ut.h"

namespace efla {

template <int DK>
struct GatedTrShape : BwdTrShape<DK, 64> {
  using B = BwdTrShape<DK, 64>;
  static constexpr int C = 64;
  static constexpr int EDT = B::LOOP_END;               // diag(e) dD (negated) [C][BV]
  static constexpr int LOOP_END = EDT + C * B::BV * 2;
  // tail: Q, later W, over X and P; dX, later Gam dA, behind Q and dP
  static constexpr int WH = B::TT, WL = WH + C * C * 2, DXH = B::A0, DXL = DXH + C * C * 2, DAF = B::A0;
  // row and column sums of M: behind dA in the region that held Q and dX, or
  // (d_k 64) behind the tail's arrays
  static constexpr int MSUM_BYTES = 2 * B::NRT * C * 4;
  static constexpr bool MSUM_IN = B::TT + C * B::CPF * 4 + MSUM_BYTES <= B::A0;
  static constexpr int MSUM = MSUM_IN ? B::TT + C * B::CPF * 4 : B::TAIL_END;
  static constexpr int TAIL_END = MSUM_IN ? B::TAIL_END : B::TAIL_END + MSUM_BYTES;
  static constexpr int BYTES = LOOP_END > TAIL_END ? LOOP_END : TAIL_END;
};

template <int DK, bool SHARED>
__global__ __launch_bounds__((GatedTrShape<DK>::NTH)) __attribute__((amdgpu_waves_per_eu(4, 4))) void gated_bwd_tr_kernel(
    GatedBwd b, const uint16_t* __restrict__ xfr, const uint16_t* __restrict__ pfr, const float* __restrict__ gws, const uint16_t* __restrict__ states, const uint16_t* __restrict__ dstates,
    float* __restrict__ dqh, float* __restrict__ dkh, int NC) {
  using S = GatedTrShape<DK>;
  constexpr int C = 64, BV = S::BV, NRT = S::NRT, NDT = S::NDT, NKU_D = S::NKU_D, NKU_C = S::NKU_C, NWV = S::NWV;
  constexpr int NTH = S::NTH, NQ = S::NQ, NP = S::NP, CPF = S::CPF;
  __shared__ __align__(1024) unsigned char lds[S::BYTES];
  __shared__ __align__(16) float as[C], dls[C], lam[C];
  __shared__ __align__(16) float gs[C], es[C], ws[C], ys[C];
  // row sums: dD.(e K S), U.(w K dS') and (X^T dU).D, by tile column of the block
  __shared__ __align__(16) float xw[6][C];
  __shared__ float c0s[NWV];
  auto b16 = [&](int off) { return reinterpret_cast<uint16_t*>(lds + off); };
  auto f32p = [&](int off) { return reinterpret_cast<float*>(lds + off); };
  uint16_t *Kt = b16(S::KT), *Xt = b16(S::TT), *Pt = b16(S::PT), *St = b16(S::ST), *dSt = b16(S::DST);
  uint16_t *Vt = b16(S::VT), *dOt = b16(S::DOT), *Dt = b16(S::DT), *dUt = b16(S::DUT), *Ut = b16(S::UT);
  uint16_t *dDt = b16(S::DDT), *eDt = b16(S::EDT), *Wt = Vt;

  const int H = b.H, Hk = b.Hk, DV = b.DV;
  const int64_t slot = blockIdx.x;
  const uint32_t bh = blockIdx.x / uint32_t(NC), batch = bh / uint32_t(H);
  const int n = int(blockIdx.x - bh * uint32_t(NC)), h32 = int(bh - batch * uint32_t(H));
  const int64_t h = h32, hk = h32 / (H / Hk);
  const int64_t left = b.L - int64_t(n) * C;
  const int valid = int(left < C ? left : C);
  const int64_t tok0 = batch * b.L + int64_t(n) * C;
  const int64_t row0 = tok0 * H + h, krow0 = tok0 * Hk + hk;
  const int tid = threadIdx.x, lane0 = tid & 63, w = wave_id(), li0 = lane0 & 15, g0 = lane0 >> 4;
  const int64_t k_stride = int64_t(Hk) * DK, v_stride = int64_t(H) * DV;
  const auto* q = static_cast<const uint16_t*>(b.q);
  const auto* k = static_cast<const uint16_t*>(b.k);
  const auto* v = static_cast<const uint16_t*>(b.v);
  const auto* dout = static_cast<const uint16_t*>(b.d_o);
  auto* dv = static_cast<uint16_t*>(b.dv);
  auto st16 = [](uint16_t* p, const u32x4& x) { *reinterpret_cast<u32x4*>(p) = x; };
  constexpr u32x4 Z{0u, 0u, 0u, 0u};

  // the chunk's K, X (high parts) and P: direct transfers (rows of K past the end re-read row 0
  // and are cleared with the first block's)
  constexpr int UK = C * DK / 8;
  static_assert(UK % NTH == 0, "whole units per thread");
  typename S::TK dma_k;
  dma_k.init(k_stride, lane0, w);
  {
    const auto* ks = static_cast<const uint16_t*>(uniform_ptr(k + krow0 * DK));
#pragma unroll
    for (int i = 0; i < S::TK::PER_WAVE; ++i) {
      if (valid == C) dma_k.template issue<false>(i, lds_addr_of(Kt), ks, C);
      else dma_k.template issue<true>(i, lds_addr_of(Kt), ks, valid);
    }
    if (w < 6) {  // 6 KiB each, in fragment order
      const uint32_t at = 1024u * uint32_t(w);
      dma16(uniform_ptr(xfr + slot * kGatedX), at + 16u * uint32_t(lane0), lds_addr_of(Xt) + at);
      dma16(uniform_ptr(pfr + slot * kGatedP), at + 16u * uint32_t(lane0), lds_addr_of(Pt) + at);
    }
  }
  if (tid < 4 * C) {
    const float x = gws[slot * kGatedG + tid];
    float* const to = tid < C ? gs : tid < 2 * C ? es : tid < 3 * C ? ws : as;
    to[tid & (C - 1)] = x;
  }
  if (tid < 6 * C) xw[tid >> 6][tid & 63] = 0.0f;

  typename S::TS dma_s;
  typename S::TV dma_v;
  dma_s.init(DK, lane0, w);
  dma_v.init(v_stride, lane0, w);
  auto dma_rows = [&](uint16_t* dst, const uint16_t* src, int v0) {
    const auto* sp_ = static_cast<const uint16_t*>(uniform_ptr(src + row0 * DV + v0));
#pragma unroll
    for (int i = 0; i < S::TV::PER_WAVE; ++i) {
      if (valid == C) dma_v.template issue<false>(i, lds_addr_of(dst), sp_, C);
      else dma_v.template issue<true>(i, lds_addr_of(dst), sp_, valid);
    }
  };
  auto dma_block = [&](int v0) {
    const auto* sb = static_cast<const uint16_t*>(uniform_ptr(states + (slot * DV + v0) * DK));
    const auto* db = static_cast<const uint16_t*>(uniform_ptr(dstates + (slot * DV + v0) * DK));
    dma_rows(Vt, v, v0);
#pragma unroll
    for (int i = 0; i < S::TS::PER_WAVE; ++i) {
      dma_s.template issue<false>(i, lds_addr_of(St), sb, BV);
      dma_s.template issue<false>(i, lds_addr_of(dSt), db, BV);
    }
    dma_rows(dOt, dout, v0);
  };
  // tile (rt, c) of a [C][BV] array: lane (li, g) holds row 16 rt + li, columns 16 c + 4 g ..
  auto put = [&](uint16_t* X, const f32x4& a, int rt, int c, int li, int g) {
    st4(X + swz_off<BV>(16 * rt + li, 16 * c + 4 * g), a);
  };
  auto sum4 = [](const f32x4& a, const f32x4& b_) {
    return fmaf(a[0], b_[0], fmaf(a[1], b_[1], fmaf(a[2], b_[2], a[3] * b_[3])));
  };

  // The [C][DK] tiles of a wavefront: two rows by two (d_k 64: one) columns, so
  // that fragments serve two products; reading them is what the LDS is busiest with.
  auto q_row = [&](int i) { return 2 * (w >> 2) + (i & 1); };
  auto q_col = [&](int i) { return NQ / 2 * (w & 3) + (i >> 1); };
  f32x4 dQa[NQ], dKa[NQ], dPa[NP], dXa[NP];
#pragma unroll
  for (int i = 0; i < NQ; ++i) dQa[i] = dKa[i] = zero4();
#pragma unroll
  for (int i = 0; i < NP; ++i) dPa[i] = dXa[i] = zero4();
  float c0 = 0.0f;  // this thread's part of <dS', S>

  constexpr int UX = kGatedX / 8;  // 16-byte units of X, both parts
  u32x4 rx[cdiv(UX, NTH)];

  dma_block(0);
  auto block = [&](const int v0, auto lastc) {
    constexpr bool LAST = decltype(lastc)::value;
    // lane indices the compiler cannot see through, so that fragment addresses
    // are formed here rather than held across the loop
    int li = li0, g = g0, lane = lane0, tidv = tid;
    asm volatile("" : "+v"(li), "+v"(g), "+v"(lane), "+v"(tidv));
    wait_vmcnt<0>();  // this wavefront's transfers of the block
    if (valid < C) {
      __syncthreads();  // every wavefront's transfers landed
      for (int i = tidv; i < 2 * (C - valid) * (BV / 8); i += NTH) {
        const int r = valid + (i >> 1) / (BV / 8), ch = (i >> 1) % (BV / 8);
        st16(((i & 1) ? dOt : Vt) + swz_off<BV>(r, 8 * ch), Z);
      }
      if (v0 == 0)
        for (int i = tidv; i < (C - valid) * (DK / 8); i += NTH)
          st16(Kt + swzw_off<DK>(valid + i / (DK / 8), 8 * (i % (DK / 8))), Z);
    }
    __syncthreads();  // the block's operands in place (and the chunk's K, T, P, gates)
    const int rt = w >> 1, c = w & 1;  // this wavefront's tile of the [C][BV] products
    // D = V - diag(e) K S and dU = P^T dO + diag(w) K dS'
    f32x4 d = zero4(), du = zero4(), eks, wkd;
    const float ar = as[16 * rt + li];
    {
#pragma unroll
      for (int ku = 0; ku < NKU_D; ++ku) {
        const Frag<uint16_t> a = wide_frag<DK>(Kt, 16 * rt + li, ku, g);
        mma(d, wide_frag<DK>(St, 16 * c + li, ku, g), a);
        mma(du, wide_frag<DK>(dSt, 16 * c + li, ku, g), a);
      }
      eks = es[16 * rt + li] * d;
      wkd = ws[16 * rt + li] * du;
      du = wkd;
#pragma unroll
      for (int ku = 0; ku < NKU_C; ++ku)
        if (32 * ku + 31 >= 16 * rt) mma(du, sw_frag_tr<BV>(dOt, 16 * c, ku, lane), tri_frag_tr(Pt, rt, ku, lane));
      const bf16x4 vv = *reinterpret_cast<const bf16x4*>(Vt + swz_off<BV>(16 * rt + li, 16 * c + 4 * g));
#pragma unroll
      for (int qq = 0; qq < 4; ++qq) d[qq] = static_cast<float>(vv[qq]) - eks[qq];
      put(Dt, ar * d, rt, c, li, g);
      put(dUt, du, rt, c, li, g);
      // <dS', S>: both tiles have one layout, eight elements a thread
      if (tidv < BV * DK / 8) {
        const bf16x8 sv = *reinterpret_cast<const bf16x8*>(St + 8 * tidv), dsv = *reinterpret_cast<const bf16x8*>(dSt + 8 * tidv);
#pragma unroll
        for (int e = 0; e < 8; ++e) c0 = fmaf(static_cast<float>(sv[e]), static_cast<float>(dsv[e]), c0);
      }
    }
    __syncthreads();
    if constexpr (LAST) {
#pragma unroll
      for (int i = 0; i < cdiv(UX, NTH); ++i)
        if (tidv + NTH * i < UX) rx[i] = *reinterpret_cast<const u32x4*>(xfr + slot * kGatedX + 8 * (tidv + NTH * i));
    }
    // U = X (a D) and dD = a X^T dU (= dV), and both scaled for dK
    {
      f32x4 u = zero4(), dd = zero4();
#pragma unroll
      for (int ku = 0; ku < NKU_C; ++ku) {
        if (32 * ku <= 16 * rt + 15) mma(u, sw_frag_tr<BV>(Dt, 16 * c, ku, lane), tri_frag(Xt, rt, ku, lane));
        if (32 * ku + 31 >= 16 * rt)
          mma(dd, sw_frag_tr<BV>(dUt, 16 * c, ku, lane), tri_frag_tr(Xt, rt, ku, lane));
      }
      const float da = row_sum4(sum4(dd, d));
      dd *= ar;
      put(Ut, u, rt, c, li, g);
      put(dDt, dd, rt, c, li, g);
      const float xs = row_sum4(sum4(dd, eks)), wk = row_sum4(sum4(u, wkd));
      put(Wt, ws[16 * rt + li] * u, rt, c, li, g);
      put(eDt, -es[16 * rt + li] * dd, rt, c, li, g);
      if (g == 0) {  // one lane per row and tile column: its own place
        xw[c][16 * rt + li] += xs;
        xw[2 + c][16 * rt + li] += wk;
        xw[4 + c][16 * rt + li] += da;
      }
    }
    __syncthreads();
    // dv = dD from its staged tile, as whole 64-byte row pieces
    if (tidv < 4 * C) {
      const int r = tidv >> 2, p = tidv & 3;
      if (r < valid) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(dDt + r * BV + 8 * (p ^ swz_row<BV / 8>(r)));
        __builtin_nontemporal_store(x, reinterpret_cast<u32x4*>(dv + row0 * DV + r * v_stride + v0 + 8 * p));
      }
    }
    if (v0 + BV >= DV) {  // the tail's Q, during the last block (over X and P, done with)
      const auto* qs = static_cast<const uint16_t*>(uniform_ptr(q + krow0 * DK));
#pragma unroll
      for (int i = 0; i < S::TK::PER_WAVE; ++i) {
        if (valid == C) dma_k.template issue<false>(i, lds_addr_of(b16(S::QT)), qs, C);
        else dma_k.template issue<true>(i, lds_addr_of(b16(S::QT)), qs, valid);
      }
    }
    // dQ += dO S^T (unscaled);  dK += (w U) dS'^T + (-e dD) S^T;  dP0 += dO U^T;  dX += dU (a D)^T
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int rr = q_row(i), dt = q_col(i);
      const Frag<uint16_t> bS = wide_frag_tr<DK>(St, dt, 0, lane);
      mma(dQa[i], bS, sw_frag<BV>(dOt, 16 * rr + li, 0, g));
      mma(dKa[i], wide_frag_tr<DK>(dSt, dt, 0, lane), sw_frag<BV>(Wt, 16 * rr + li, 0, g));
      mma(dKa[i], bS, sw_frag<BV>(eDt, 16 * rr + li, 0, g));
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int t = w + NWV * i, rr = t / NRT, jt = t % NRT;
      if (jt <= rr) {
        mma(dPa[i], sw_frag<BV>(Ut, 16 * jt + li, 0, g), sw_frag<BV>(dOt, 16 * rr + li, 0, g));
        mma(dXa[i], sw_frag<BV>(Dt, 16 * jt + li, 0, g), sw_frag<BV>(dUt, 16 * rr + li, 0, g));
      }
    }
    if (v0 + BV < DV) {
      __syncthreads();  // every read of this block's operands done
      dma_block(v0 + BV);
    }
  };
  for (int v0 = 0; v0 + BV < DV; v0 += BV) block(v0, std::false_type{});
  block(DV - BV, std::true_type{});
  wait_vmcnt<0>();  // Q's transfers and X
  __syncthreads();  // done with the loop's arrays (K stays); Q in place

  // ---- the UT-transform part (bwd_chunk_tr.h), with the gates -----------------
  int li = li0, g = g0, lane = lane0;
  // As in a value block: between the stages the compiler may not carry addresses
  // over (it kept a dozen for the last stage in scratch, whose reloads one by one
  // took 10,000 of a chunk's 95,000 cycles)
  auto fresh = [&]() { asm volatile("" : "+v"(li), "+v"(g), "+v"(lane)); };
  uint16_t *Qt = b16(S::QT), *dPt = b16(S::DPT), *dXh = b16(S::DXH), *dXl = b16(S::DXL);
  uint16_t *Wh = b16(S::WH), *Wl = b16(S::WL), *Xh = b16(S::XF), *Xl = Xh + kGatedX / 2, *Eb = b16(S::EB);
  uint16_t *dQs = b16(S::DQS), *dKs = b16(S::DKS);
  float *dAf = f32p(S::DAF), *red = f32p(S::RED), *msum = f32p(S::MSUM);
  constexpr int CPG = S::CPG;
  auto split = [](float x, uint16_t& hi, uint16_t& lo) {
    hi = from_f32<uint16_t>(x);
    lo = from_f32<uint16_t>(x - to_f32(hi));
  };
  auto split4 = [&](const f32x4& x, uint16_t* hi, uint16_t* lo) {  // four values, 8 bytes of each part
    uint16_t h4[4], l4[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split(x[e], h4[e], l4[e]);
    *reinterpret_cast<uint2*>(hi) = *reinterpret_cast<const uint2*>(h4);
    *reinterpret_cast<uint2*>(lo) = *reinterpret_cast<const uint2*>(l4);
  };
  // key columns of the four values a lane holds of tile column dt, as stored
  auto key4 = [&](int dt) { return key_phys(16 * dt + 4 * g); };
  auto mma3 = [](f32x4& acc, const Frag<uint16_t>& ah, const Frag<uint16_t>& al, const Frag<uint16_t>& bh_,
                 const Frag<uint16_t>& bl) {
    mma(acc, ah, bh_);
    mma(acc, ah, bl);
    mma(acc, al, bh_);
  };
  c0 = row_sum4(row_sum16(c0));
  if (lane == 0) c0s[w] = c0;
  // rows of Q past the end re-read row 0: cleared before they are read
  if (valid < C) {
    for (int i = tid; i < (C - valid) * (DK / 8); i += NTH)
      st16(Qt + swzw_off<DK>(valid + i / (DK / 8), 8 * (i % (DK / 8))), Z);
    __syncthreads();
  }
  // Y1 = diag(e) dO S^T, and q . Y1 row by row (partial sums by dt)
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int rr = q_row(i), dt = q_col(i);
    const int r = 16 * rr + li;
    dQa[i] *= es[r];
    const bf16x4 qv = *reinterpret_cast<const bf16x4*>(Qt + swzw_off<DK>(r, key4(dt)));
    f32x4 qf;
#pragma unroll
    for (int qq = 0; qq < 4; ++qq) qf[qq] = static_cast<float>(qv[qq]);
    const float s = row_sum4(sum4(dQa[i], qf));
    if (g == 0) red[dt * C + r] = s;
  }
  fresh();
  // dP = Gam * dP0 as bf16, dX and X as high and low parts; the first part of
  // M (strictly lower), dP * Q K^T, stays in registers
  f32x4 M[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = w + NWV * i, rr = t / NRT, jt = t % NRT;
    const int r = 16 * rr + li, c = 16 * jt + 4 * g;
    f32x4 qk = zero4();
    if (jt <= rr) {
#pragma unroll
      for (int ku = 0; ku < NKU_D; ++ku)
        mma(qk, wide_frag<DK>(Kt, 16 * jt + li, ku, g), wide_frag<DK>(Qt, 16 * rr + li, ku, g));
    }
    const float gr = gs[r];
    const f32x4 gj = *reinterpret_cast<const f32x4*>(gs + c);
    f32x4 p, dx;
#pragma unroll
    for (int qq = 0; qq < 4; ++qq) {
      p[qq] = c + qq <= r ? dPa[i][qq] * exp2_gate(gr - gj[qq]) : 0.0f;
      M[i][qq] = c + qq < r ? p[qq] * qk[qq] : 0.0f;
      dx[qq] = c + qq <= r ? dXa[i][qq] : 0.0f;
    }
    st4(dPt + swz_off<C>(r, c), p);
    split4(dx, dXh + swz_off<C>(r, c), dXl + swz_off<C>(r, c));
  }
#pragma unroll
  for (int i = 0; i < cdiv(UX, NTH); ++i)
    if (tid + NTH * i < UX) st16(Xh + 8 * (tid + NTH * i), rx[i]);
  __syncthreads();
  if (tid < C) {  // y_i so far
    float s = -(xw[0][tid] + xw[1][tid]);
#pragma unroll
    for (int j = 0; j < NDT; ++j) s += red[j * C + tid];
    ys[tid] = s;
  }
  fresh();
  // dQ += dP K;  dK += dP^T Q
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int rr = q_row(i), dt = q_col(i);
#pragma unroll
    for (int ku = 0; ku < NKU_C; ++ku) {
      if (32 * ku <= 16 * rr + 15)
        mma(dQa[i], wide_frag_tr<DK>(Kt, dt, ku, lane), sw_frag<C>(dPt, 16 * rr + li, ku, g));
      if (32 * ku + 31 >= 16 * rr)
        mma(dKa[i], wide_frag_tr<DK>(Qt, dt, ku, lane), sw_frag_tr<C>(dPt, 16 * rr, ku, lane));
    }
  }
  // dQ is complete: it waits for its place in the LDS as packed bf16 (half the
  // registers), or, of a shared head, leaves in fp32
  uint2 dQp[NQ];
  auto leave = [&](const f32x4& x, float* dst, int rr, int dt) {
    const int r = 16 * rr + li;
    if (r < valid) *reinterpret_cast<f32x4*>(dst + (row0 + int64_t(r) * H) * DK + key4(dt)) = x;
  };
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    if constexpr (SHARED) leave(dQa[i], dqh, q_row(i), q_col(i));
    else {
      bf16x4 x;
#pragma unroll
      for (int qq = 0; qq < 4; ++qq) x[qq] = static_cast<__bf16>(dQa[i][qq]);
      dQp[i] = __builtin_bit_cast(uint2, x);
    }
  }
  __syncthreads();  // red is read, Q and dP are done with
  // W = X^T dX, as high and low parts (over Q)
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = w + NWV * i, rr = t / NRT, jt = t % NRT;
    f32x4 acc = zero4();
#pragma unroll
    for (int ku = 0; ku < NKU_C; ++ku)
      if (32 * ku + 31 >= 16 * rr && 32 * ku + 31 >= 16 * jt)  // X and dT are lower triangular
        mma3(acc, sw_frag_tr<C>(dXh, 16 * jt, ku, lane), sw_frag_tr<C>(dXl, 16 * jt, ku, lane),
             tri_frag_tr(Xh, rr, ku, lane), tri_frag_tr(Xl, rr, ku, lane));
    const int at = swz_off<C>(16 * rr + li, 16 * jt + 4 * g);
    split4(acc, Wh + at, Wl + at);
  }
  __syncthreads();
  fresh();
  // Gam dA = -Gam * (W X^T) (strictly lower, fp32, over dX);  K K^T on the lower
  // tiles: lambda, N = Gam dA * K K^T and M += diag(a) N, with their sums
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = w + NWV * i, rr = t / NRT, jt = t % NRT;
    f32x4 acc = zero4(), gg = zero4();
    if (jt <= rr) {
#pragma unroll
      for (int ku = 0; ku < NKU_C; ++ku)
        if (32 * ku <= 16 * jt + 15)  // X^T's rows of this tile are zero past column 16 jt + 15
          mma3(acc, tri_frag(Xh, jt, ku, lane), tri_frag(Xl, jt, ku, lane),
               sw_frag<C>(Wh, 16 * rr + li, ku, g), sw_frag<C>(Wl, 16 * rr + li, ku, g));
#pragma unroll
      for (int ku = 0; ku < NKU_D; ++ku)
        mma(gg, wide_frag<DK>(Kt, 16 * jt + li, ku, g), wide_frag<DK>(Kt, 16 * rr + li, ku, g));
    }
    const int r = 16 * rr + li, c = 16 * jt + 4 * g;
    const float gr = gs[r], ar = as[r];
    const f32x4 gj = *reinterpret_cast<const f32x4*>(gs + c);
    f32x4 da;
    float s = 0.0f, sm = 0.0f;
#pragma unroll
    for (int qq = 0; qq < 4; ++qq) {
      da[qq] = c + qq < r ? -acc[qq] * exp2_gate(gr - gj[qq]) : 0.0f;
      if (c + qq == r) lam[r] = gg[qq];
      const float nn = da[qq] * gg[qq], m = fmaf(ar, nn, M[i][qq]);
      s += nn;
      sm += m;
      const float cs = row_sum16(m);  // over the tile's rows
      if (li == 0) msum[(NRT + rr) * C + c + qq] = cs;
    }
    *reinterpret_cast<f32x4*>(dAf + r * CPF + c) = da;
    s = row_sum4(s);
    sm = row_sum4(sm);
    if (g == 0) {
      red[jt * C + r] = s;
      msum[jt * C + r] = sm;
    }
  }
  __syncthreads();
  // da_i += sum_j N_ij, then dbeta and dlambda, by one wavefront;  dg by another;
  // dG + dG^T as bf16 (over X)
  if (tid < C) {
    float s = xw[4][tid] + xw[5][tid];
#pragma unroll
    for (int jt = 0; jt < NRT; ++jt) s += red[jt * C + tid];
    float dl = 0.0f;
    if (tid < valid) {
      const float bt = to_f32(static_cast<const uint16_t*>(b.beta)[row0 + int64_t(tid) * H]);
      float da_db, da_dl;
      efla_alpha_grad(bt, lam[tid], b.rule, da_db, da_dl);
      dl = s * da_dl;
      static_cast<uint16_t*>(b.dbeta)[row0 + int64_t(tid) * H] = from_f32<uint16_t>(s * da_db);
    }
    dls[tid] = dl;
  } else if (tid < 2 * C) {
    // dg_t = e^{G_C} <dS', S> + sum_{j<t} k_j . Y2_j + sum_{i>=t} y_i: sums of the
    // tokens before, and, with the tokens in reverse order, from here on
    const int t = lane, rev = C - 1 - lane;
    float y = ys[rev];
#pragma unroll
    for (int jt = 0; jt < NRT; ++jt) y += msum[jt * C + rev] - msum[(NRT + jt) * C + rev];
    const float wj = xw[2][t] + xw[3][t];
    const float before = wave_scan_dpp(wj), from = wave_scan_dpp(y);
    float all = 0.0f;
#pragma unroll
    for (int j = 0; j < NWV; ++j) all += c0s[j];
    const float after = __shfl(from, rev);
    if (t < valid)
      store_gate_grad<uint16_t>(b.dg, row0 + int64_t(t) * H, fmaf(es[C - 1], all, before - wj + after), b.dg32);
  }
#pragma unroll
  for (int i = 0; i < C * C / 4 / NTH; ++i) {
    const int u = tid + NTH * i, r = u / (C / 4), c = 4 * (u % (C / 4));
    f32x4 x = as[r] * *reinterpret_cast<const f32x4*>(dAf + r * CPF + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = fmaf(as[c + e], dAf[(c + e) * CPF + r], x[e]);
    st4(Eb + swz_off<C>(r, c), x);
  }
  __syncthreads();
  fresh();
  // dK += (dG + dG^T) K + 2 diag(dlambda) K
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int rr = q_row(i), dt = q_col(i);
#pragma unroll
    for (int ku = 0; ku < NKU_C; ++ku)
      mma(dKa[i], wide_frag_tr<DK>(Kt, dt, ku, lane), sw_frag<C>(Eb, 16 * rr + li, ku, g));
    const int r = 16 * rr + li, cp = key4(dt);
    const float dl = 2.0f * dls[r];
    const bf16x4 kv = *reinterpret_cast<const bf16x4*>(Kt + swzw_off<DK>(r, cp));
#pragma unroll
    for (int qq = 0; qq < 4; ++qq) dKa[i][qq] = fmaf(dl, static_cast<float>(kv[qq]), dKa[i][qq]);
    if constexpr (!SHARED) {  // dQ and dK staged as bf16 rows over W and dA
      *reinterpret_cast<uint2*>(dQs + r * CPG + cp) = dQp[i];
      st4(dKs + r * CPG + cp, dKa[i]);
    }
  }
  if constexpr (SHARED) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) leave(dKa[i], dkh, q_row(i), q_col(i));
  } else {
    __syncthreads();
    auto* dq = static_cast<uint16_t*>(b.dq);
    auto* dk = static_cast<uint16_t*>(b.dk);
#pragma unroll
    for (int i = 0; i < UK / NTH; ++i) {
      const int u = tid + NTH * i, r = u / (DK / 8), ch = u % (DK / 8);
      if (r < valid) {
        __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(dQs + r * CPG + 8 * ch),
                                    reinterpret_cast<u32x4*>(dq + krow0 * DK + r * k_stride + 8 * ch));
        __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(dKs + r * CPG + 8 * ch),
                                    reinterpret_cast<u32x4*>(dk + krow0 * DK + r * k_stride + 8 * ch));
      }
    }
  }
}

}  // namespace efla
