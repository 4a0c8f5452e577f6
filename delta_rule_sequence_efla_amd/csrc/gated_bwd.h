// gated_bwd.h -- the chunked backward pass of the gated delta rule (gated.h) in
// fp32 on fp32 matrix cores, for every type and size.
//
// Per chunk with start state S, end-state gradient dS', e = e^G, w = e^{G_C - G}
// (one value a token), Gam_ij = e^{G_i - G_j} and
//     A = tril(diag(a) (Gam * K K^T), -1),  X = (I + A)^{-1},  T = X diag(a),
//     D = V - diag(e) K S,  U = T D,  P = Gam * tril(Q K^T),
//     O = diag(e) Q S + P U,  S' = e^{G_C} S + K^T diag(w) U,
// calculus gives
//     dU = P^T dO + diag(w) K dS'       dD = T^T dU = dV       dT = tril(dU D^T)
//     dP0 = tril(dO U^T),  dP = Gam * dP0
//     dQ = Y1 + dP K                    Y1 = diag(e) dO S^T
//     dK = dP^T Q + Y2 - Y3 + (dG + dG^T) K + 2 diag(dlambda) K
//                                       Y2 = diag(w) U dS'^T,  Y3 = diag(e) dD S^T
//     da_j = sum_i dT_ij X_ij,  dA = -X^T dT diag(a) X^T (strictly lower),
//     N = dA * Gam * K K^T,     da_i += sum_j N_ij,   dG = diag(a) (Gam * dA)
//     dS = e^{G_C} dS' + Q^T diag(e) dO - K^T diag(e) dD
// and dbeta, dlambda from da (bwd_kernels.h).  The gates: every factor e^{G_i -
// G_j} is crossed by the gates j < t <= i, so with M = dP0 * P + diag(a) N
// (strictly lower)
//     dg_t = e^{G_C} <dS', S> + sum_{j<t} (k_j . Y2_j)
//          + sum_{i>=t} (q_i . Y1_i - k_i . Y3_i + sum_j M_ij - sum_j M_ji):
// pairs with both ends at or past t cancel term by term, out of one fp32
// array, so no large sums are subtracted.
// Shared key heads: dq and dk are formed per value head (fp32, in the
// workspace) and summed in head order by a last kernel, so results do not
// depend on timing.
#pragma once

#include "bwd_kernels.h"
#include "gated.h"
#include "launchers.h"

namespace efla {

struct GatedBwdLayout {
  size_t t, x, p, a, gc, s, ds, dqh, dkh, xfr, qe, total;
};

// Inclusive sum over the 64 lanes of a wavefront.
__device__ __forceinline__ float wave_scan_f32(float x, int lane) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const float y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// ---------------------------------------------------------------------------
// T, X, P, a and G of every chunk, fp32, one workgroup per chunk.  X by blocks of
// 16 rows: the rows above contribute by matrix products, spread over the
// wavefronts, then a thread per column solves the diagonal block out of
// registers (row by row over the whole chunk, one wavefront took 35 us of a
// chunk's 40).
// ---------------------------------------------------------------------------
template <typename T, int DK, int C>
__global__ __launch_bounds__(kThreads) void gated_ut_kernel(GatedBwd b, float* __restrict__ tws,
                                                            float* __restrict__ xws, float* __restrict__ pws,
                                                            float* __restrict__ aws, double* __restrict__ gws, int NC) {
  constexpr int DKP = round_up(DK, 32), CP = round_up(C, 32), QP = DKP + 4, CPP = CP + 4, NCP = CP / 16;
  __shared__ __align__(16) float Qs[CP * QP];
  __shared__ __align__(16) float Ks[CP * QP];
  __shared__ __align__(16) float Am[CP * CPP];
  __shared__ __align__(16) float Xm[CP * CPP];
  __shared__ __align__(16) float Rm[16 * CPP];
  __shared__ float as[CP];
  __shared__ double gs[CP];
  const int64_t slot = blockIdx.x;
  const uint32_t bh = blockIdx.x / uint32_t(NC);
  const int n = int(blockIdx.x - bh * uint32_t(NC));
  const int h = int(bh % uint32_t(b.H)), hk = h / (b.H / b.Hk);
  const int64_t t0 = bh / uint32_t(b.H) * b.L + int64_t(n) * C;
  const int valid = int(b.L - int64_t(n) * C < C ? b.L - int64_t(n) * C : C);
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), li = lane & 15, g = lane >> 4;
  {
    F32Stager<T, C, DK> sq, sk;
    sq.load(static_cast<const T*>(b.q) + (t0 * b.Hk + hk) * DK, int64_t(b.Hk) * DK, valid, tid);
    sk.load(static_cast<const T*>(b.k) + (t0 * b.Hk + hk) * DK, int64_t(b.Hk) * DK, valid, tid);
    if constexpr (C < CP || DK < DKP) {
      for (int i = tid; i < CP * QP; i += kThreads) Qs[i] = Ks[i] = 0.0f;
      __syncthreads();
    }
    sq.store(Qs, QP, tid);
    sk.store(Ks, QP, tid);
  }
  if (w == 0) {
    const float gg = lane < valid ? gate_floor(b.g[(t0 + lane) * b.H + h]) : 0.0f;
    const double G = wave_scan_gate(gg, lane);
    if (lane < CP) gs[lane] = G;
    if (lane < C) gws[slot * C + lane] = G;
  }
  __syncthreads();
  for (int t = w; t < NCP * NCP; t += 4) {
    const int r0 = 16 * (t / NCP), c0 = 16 * (t % NCP);
    f32x4 acc = zero4(), pp = zero4();
    if (c0 <= r0) {
      tile_mma16<false, true>(acc, Ks, QP, Ks, QP, r0, c0, DKP, li, g);
      tile_mma16<false, true>(pp, Qs, QP, Ks, QP, r0, c0, DKP, li, g);
    }
#pragma unroll
    for (int qq = 0; qq < 4; ++qq) {
      const int r = r0 + 4 * g + qq, c = c0 + li;
      const float gam = c <= r ? expf(float(gs[r] - gs[c])) : 0.0f;
      if (r == c) as[r] = acc[qq];
      Am[r * CPP + c] = c < r ? gam * acc[qq] : 0.0f;
      if (r < C && c < C) pws[slot * C * C + r * C + c] = c <= r ? gam * pp[qq] : 0.0f;
    }
  }
  __syncthreads();
  if (tid < CP) {
    const float a =
        tid < valid ? efla_alpha_rule(to_f32(static_cast<const T*>(b.beta)[(t0 + tid) * b.H + h]), as[tid], b.rule) : 0.0f;
    as[tid] = a;
    if (tid < C) aws[slot * C + tid] = a;
  }
  __syncthreads();
  // x_r = delta_rc - a_r sum_{m<r} (Gam * G)_rm x_m
  for (int b0 = 0; b0 < CP; b0 += 16) {
    for (int jt = w; 16 * jt < b0; jt += 4) {
      f32x4 acc = zero4();
      tile_mma16<false, false>(acc, Am, CPP, Xm, CPP, b0, 16 * jt, b0, li, g);
#pragma unroll
      for (int qq = 0; qq < 4; ++qq) Rm[(4 * g + qq) * CPP + 16 * jt + li] = acc[qq];
    }
    __syncthreads();
    if (tid < CP) {
      float x[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float s = tid < b0 ? Rm[r * CPP + tid] : 0.0f;
#pragma unroll
        for (int m = 0; m < r; ++m) s = fmaf(Am[(b0 + r) * CPP + b0 + m], x[m], s);
        x[r] = (b0 + r == tid ? 1.0f : 0.0f) - as[b0 + r] * s;
        Xm[(b0 + r) * CPP + tid] = x[r];
      }
    }
    __syncthreads();
  }
  for (int i = tid; i < C * C; i += kThreads) {
    const int r = i / C, c = i % C;
    const float x = Xm[r * CPP + c];
    xws[slot * C * C + i] = x;
    tws[slot * C * C + i] = x * as[c];
  }
}

// ---------------------------------------------------------------------------
// Reverse pass over the chunks: one workgroup per (b, h, 16 value columns), dS
// (d_k x 16, fp32) in LDS, as bwd_state_kernel:
//   dstates[n] = dS';  E = P^T dO + diag(w) K dS',  F = T^T E,
//   dS = e^{G_C} dS' + Q^T diag(e) dO - K^T diag(e) F
// ---------------------------------------------------------------------------
template <typename T, int DK, int C>
__global__ __launch_bounds__(kThreads) void gated_bwd_state_kernel(GatedBwd b, const float* __restrict__ tws,
                                                                   const float* __restrict__ pws,
                                                                   const double* __restrict__ gws,
                                                                   float* __restrict__ dstates, int NC, int NVB) {
  constexpr int DKP = round_up(DK, 32), CP = round_up(C, 32);
  constexpr int QP = DKP + 4, CPP = CP + 4, VP = 16 + 4;
  __shared__ __align__(16) float Qs[CP * QP];
  __shared__ __align__(16) float Ks[CP * QP];
  __shared__ __align__(16) float Ts[CP * CPP];
  __shared__ __align__(16) float Ps[CP * CPP];
  __shared__ __align__(16) float dOs[CP * VP];
  __shared__ __align__(16) float Es[CP * VP];
  __shared__ __align__(16) float Fs[CP * VP];
  __shared__ __align__(16) float dSs[DKP * VP];
  __shared__ float es[CP], ws[CP];

  const int x = blockIdx.x, bh = x / NVB, vb = x % NVB, DV = b.DV;
  const int h = bh % b.H, hk = h / (b.H / b.Hk);
  const int64_t bos = int64_t(bh / b.H) * b.L, slot0 = int64_t(bh) * NC;
  const int v0 = 16 * vb;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), li = lane & 15, g = lane >> 4;

  for (int i = tid; i < CP * QP; i += kThreads) Qs[i] = Ks[i] = 0.0f;
  for (int i = tid; i < CP * CPP; i += kThreads) Ts[i] = Ps[i] = 0.0f;
  for (int i = tid; i < CP * VP; i += kThreads) dOs[i] = 0.0f;
  for (int i = tid; i < DKP * 16; i += kThreads) {
    const int d = i / 16, c = i % 16;
    dSs[d * VP + c] = (b.dsf != nullptr && d < DK) ? b.dsf[(int64_t(bh) * DK + d) * DV + v0 + c] : 0.0f;
  }
  F32Stager<T, C, DK> sq, sk;
  F32Stager<float, C, C> st, spp;
  F32Stager<T, C, 16> sdo;
  double G = 0.0, GC = 0.0;
  auto load = [&](int n) {
    const int64_t t0 = bos + int64_t(n) * C;
    const int64_t left = b.L - int64_t(n) * C;
    const int valid = int(left < C ? left : C);
    sq.load(static_cast<const T*>(b.q) + (t0 * b.Hk + hk) * DK, int64_t(b.Hk) * DK, valid, tid);
    sk.load(static_cast<const T*>(b.k) + (t0 * b.Hk + hk) * DK, int64_t(b.Hk) * DK, valid, tid);
    sdo.load(static_cast<const T*>(b.d_o) + (t0 * b.H + h) * DV + v0, int64_t(b.H) * DV, valid, tid);
    st.load(tws + (slot0 + n) * C * C, C, C, tid);
    spp.load(pws + (slot0 + n) * C * C, C, C, tid);
    if (tid < CP) G = tid < C ? gws[(slot0 + n) * C + tid] : 0.0;
    GC = gws[(slot0 + n) * C + C - 1];
  };
  if (NC > 0) load(NC - 1);
  __syncthreads();
  for (int n = NC - 1; n >= 0; --n) {
    float* dst = dstates + (slot0 + n) * DK * DV;
    for (int i = tid; i < DK * 16; i += kThreads) {
      const int d = i / 16, c = i % 16;
      dst[int64_t(d) * DV + v0 + c] = dSs[d * VP + c];
    }
    sq.store(Qs, QP, tid);
    sk.store(Ks, QP, tid);
    sdo.store(dOs, VP, tid);
    st.store(Ts, CPP, tid);
    spp.store(Ps, CPP, tid);
    if (tid < CP) {
      es[tid] = expf(float(G));
      ws[tid] = expf(float(GC - G));
    }
    const float end = expf(float(GC));
    if (n > 0) load(n - 1);  // in flight during this chunk
    __syncthreads();
    for (int rt = w; rt < CP / 16; rt += 4) {
      f32x4 acc = zero4(), kd = zero4();
      tile_mma16<true, false>(acc, Ps, CPP, dOs, VP, 16 * rt, 0, CP, li, g);
      tile_mma16<false, false>(kd, Ks, QP, dSs, VP, 16 * rt, 0, DKP, li, g);
#pragma unroll
      for (int qq = 0; qq < 4; ++qq) {
        const int r = 16 * rt + 4 * g + qq;
        Es[r * VP + li] = fmaf(ws[r], kd[qq], acc[qq]);
      }
    }
    __syncthreads();
    for (int rt = w; rt < CP / 16; rt += 4) {
      f32x4 acc = zero4();
      tile_mma16<true, false>(acc, Ts, CPP, Es, VP, 16 * rt, 0, CP, li, g);
#pragma unroll
      for (int qq = 0; qq < 4; ++qq) {
        const int r = 16 * rt + 4 * g + qq;
        Fs[r * VP + li] = es[r] * acc[qq];
        dOs[r * VP + li] *= es[r];  // read above by every wavefront
      }
    }
    __syncthreads();
    for (int dt = w; dt < DKP / 16; dt += 4) {
      f32x4 plus = zero4(), minus = zero4();
      tile_mma16<true, false>(plus, Qs, QP, dOs, VP, 16 * dt, 0, CP, li, g);
      tile_mma16<true, false>(minus, Ks, QP, Fs, VP, 16 * dt, 0, CP, li, g);
#pragma unroll
      for (int qq = 0; qq < 4; ++qq) {
        float* p = dSs + (16 * dt + 4 * g + qq) * VP + li;
        *p = fmaf(end, *p, plus[qq] - minus[qq]);
      }
    }
    __syncthreads();
  }
  if (b.ds0 != nullptr) {
    for (int i = tid; i < DK * 16; i += kThreads) {
      const int d = i / 16, c = i % 16;
      b.ds0[(int64_t(bh) * DK + d) * DV + v0 + c] = dSs[d * VP + c];
    }
  }
}

// ---------------------------------------------------------------------------
// Every chunk's gradients in parallel: one workgroup per chunk and head, value
// columns 16 at a time (as bwd_chunk_kernel), then the UT-transform part and
// the gates.  dqh, dkh: fp32 [B L][H][d_k] where key heads are shared, else null.
// ---------------------------------------------------------------------------
template <typename T, int DK, int C>
__global__ __launch_bounds__(kThreads) void gated_bwd_chunk_kernel(
    GatedBwd b, const float* __restrict__ tws, const float* __restrict__ xws, const float* __restrict__ pws,
    const float* __restrict__ aws, const double* __restrict__ gws, const float* __restrict__ states,
    const float* __restrict__ dstates, float* __restrict__ dqh, float* __restrict__ dkh, int NC) {
  using S = BwdChunkShape<T, DK, C>;
  constexpr int DKP = S::DKP, CP = S::CP, QP = S::QP, CPP = S::CPP, VP = S::VP, NQ = S::NQ, NP = S::NP;
  constexpr int NCQ = DKP / 16, NCP = CP / 16;
  __shared__ __align__(16) float Qs[CP * QP];
  __shared__ __align__(16) float Ks[CP * QP];
  __shared__ __align__(16) float M0[CP * CPP];  // T, then dT
  __shared__ __align__(16) float M1[CP * CPP];  // P, then dP, then X^T dX
  __shared__ __align__(16) float R[S::RBUF];
  __shared__ float rx[NCQ * CP], rw[NCQ * CP];  // row sums by tile column
  __shared__ float as[CP], das[CP], dls[CP], es[CP], ws[CP], ys[CP], c0s[kThreads / kWave];
  __shared__ double gs[CP];

  const int64_t slot = blockIdx.x;
  const uint32_t bh = blockIdx.x / uint32_t(NC);
  const int n = int(blockIdx.x - bh * uint32_t(NC)), H = b.H, Hk = b.Hk, DV = b.DV;
  const int h = int(bh % uint32_t(H)), hk = h / (H / Hk);
  const int64_t left = b.L - int64_t(n) * C;
  const int valid = int(left < C ? left : C);
  const int64_t t0 = bh / uint32_t(H) * b.L + int64_t(n) * C, row0 = t0 * H + h, krow0 = t0 * Hk + hk;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), li = lane & 15, g = lane >> 4;
  const int64_t k_stride = int64_t(Hk) * DK, v_stride = int64_t(H) * DV;
  const T* v = static_cast<const T*>(b.v);
  const T* dout = static_cast<const T*>(b.d_o);
  T* dv = static_cast<T*>(b.dv);
  {
    F32Stager<T, C, DK> sq, sk;
    F32Stager<float, C, C> st, spp;
    sq.load(static_cast<const T*>(b.q) + krow0 * DK, k_stride, valid, tid);
    sk.load(static_cast<const T*>(b.k) + krow0 * DK, k_stride, valid, tid);
    st.load(tws + slot * C * C, C, C, tid);
    spp.load(pws + slot * C * C, C, C, tid);
    if constexpr (C < CP || DK < DKP) {
      for (int i = tid; i < CP * QP; i += kThreads) Qs[i] = Ks[i] = 0.0f;
      for (int i = tid; i < CP * CPP; i += kThreads) M0[i] = M1[i] = 0.0f;
      __syncthreads();
    }
    sq.store(Qs, QP, tid);
    sk.store(Ks, QP, tid);
    st.store(M0, CPP, tid);
    spp.store(M1, CPP, tid);
  }
  const double GC = gws[slot * C + C - 1];
  const float end = expf(float(GC));
  if (tid < CP) {
    const double G = tid < C ? gws[slot * C + tid] : GC;
    as[tid] = tid < C ? aws[slot * C + tid] : 0.0f;
    gs[tid] = G;
    es[tid] = expf(float(G));
    ws[tid] = expf(float(GC - G));
  }
  float* Sv = R;               // S[:, block]      DKP x 16
  float* dSv = Sv + DKP * VP;  // dS'[:, block]
  float* Vv = dSv + DKP * VP;  // V rows, block    CP x 16
  float* dOv = Vv + CP * VP;
  float* Dv = dOv + CP * VP;
  float* Uv = Dv + CP * VP;
  float* dUv = Uv + CP * VP;
  float* dDv = dUv + CP * VP;

  f32x4 y1[NQ], y2[NQ], y3[NQ], dPa[NP], dTa[NP];
#pragma unroll
  for (int i = 0; i < NQ; ++i) y1[i] = y2[i] = y3[i] = zero4();
#pragma unroll
  for (int i = 0; i < NP; ++i) dPa[i] = dTa[i] = zero4();
  float c0 = 0.0f;  // this thread's part of <dS', S>

  const float* st = states + slot * DK * DV;
  const float* dst = dstates + slot * DK * DV;
  F32Stager<float, DK, 16> ss, sds;
  F32Stager<T, C, 16> sv, sdo;
  auto load_block = [&](int v0) {
    ss.load(st + v0, DV, DK, tid);
    sds.load(dst + v0, DV, DK, tid);
    sv.load(v + row0 * DV + v0, v_stride, valid, tid);
    sdo.load(dout + row0 * DV + v0, v_stride, valid, tid);
  };
  load_block(0);
  if constexpr (C < CP || DK < DKP) {  // padding rows of the block buffers stay zero
    __syncthreads();
    for (int i = tid; i < S::VBUF; i += kThreads) R[i] = 0.0f;
  }
  for (int v0 = 0; v0 < DV; v0 += 16) {
    __syncthreads();
    ss.store(Sv, VP, tid);
    sds.store(dSv, VP, tid);
    sv.store(Vv, VP, tid);
    sdo.store(dOv, VP, tid);
    if (v0 + 16 < DV) load_block(v0 + 16);
    __syncthreads();
    for (int i = tid; i < DK * 16; i += kThreads) c0 = fmaf(Sv[(i / 16) * VP + i % 16], dSv[(i / 16) * VP + i % 16], c0);
    for (int t = w; t < 2 * NCP; t += 4) {
      const int rt = t % NCP;
      f32x4 acc = zero4();
      if (t < NCP) {
        tile_mma16<false, false>(acc, Ks, QP, Sv, VP, 16 * rt, 0, DKP, li, g);
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {
          const int r = 16 * rt + 4 * g + qq;
          Dv[r * VP + li] = fmaf(-es[r], acc[qq], Vv[r * VP + li]);
        }
      } else {
        f32x4 kd = zero4();
        tile_mma16<true, false>(acc, M1, CPP, dOv, VP, 16 * rt, 0, CP, li, g);
        tile_mma16<false, false>(kd, Ks, QP, dSv, VP, 16 * rt, 0, DKP, li, g);
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {
          const int r = 16 * rt + 4 * g + qq;
          dUv[r * VP + li] = fmaf(ws[r], kd[qq], acc[qq]);
        }
      }
    }
    __syncthreads();
    for (int t = w; t < 2 * NCP; t += 4) {
      const int rt = t % NCP;
      f32x4 acc = zero4();
      if (t < NCP) {
        tile_mma16<false, false>(acc, M0, CPP, Dv, VP, 16 * rt, 0, CP, li, g);
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) Uv[(16 * rt + 4 * g + qq) * VP + li] = acc[qq];
      } else {
        tile_mma16<true, false>(acc, M0, CPP, dUv, VP, 16 * rt, 0, CP, li, g);
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {
          const int r = 16 * rt + 4 * g + qq;
          dDv[r * VP + li] = acc[qq];
          if (r < valid) dv[row0 * DV + r * v_stride + v0 + li] = from_f32<T>(acc[qq]);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int t = w + 4 * i, r0 = 16 * (t / NCQ), cc = 16 * (t % NCQ);
      tile_mma16<false, true>(y1[i], dOv, VP, Sv, VP, r0, cc, 16, li, g);
      tile_mma16<false, true>(y2[i], Uv, VP, dSv, VP, r0, cc, 16, li, g);
      tile_mma16<false, true>(y3[i], dDv, VP, Sv, VP, r0, cc, 16, li, g);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int t = w + 4 * i, r0 = 16 * (t / NCP), cc = 16 * (t % NCP);
      tile_mma16<false, true>(dPa[i], dOv, VP, Uv, VP, r0, cc, 16, li, g);
      tile_mma16<false, true>(dTa[i], dUv, VP, Dv, VP, r0, cc, 16, li, g);
    }
  }
  __syncthreads();  // done with T and the value-block buffers

  // row sums q . Y1 - k . Y3 and k . Y2 by tile column; y2 becomes Y2 - Y3
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int t = w + 4 * i, ct = t % NCQ, r0 = 16 * (t / NCQ);
#pragma unroll
    for (int qq = 0; qq < 4; ++qq) {
      const int r = r0 + 4 * g + qq, c = 16 * ct + li;
      const float e = es[r];
      y1[i][qq] *= e;
      y2[i][qq] *= ws[r];
      y3[i][qq] *= e;
      const float xs = row_sum16(Qs[r * QP + c] * y1[i][qq] - Ks[r * QP + c] * y3[i][qq]);
      const float wk = row_sum16(Ks[r * QP + c] * y2[i][qq]);
      if (li == 0) {
        rx[ct * CP + r] = xs;
        rw[ct * CP + r] = wk;
      }
      y2[i][qq] -= y3[i][qq];
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) c0 += __shfl_xor(c0, d);
  if (lane == 0) c0s[w] = c0;
  float* X = R;
  float* R1 = R + CP * CPP;
  float* R2 = R1 + CP * CPP;
  // dP0 * P (strictly lower) -> R2;  dP (lower, diagonal included) -> M1;  dT -> M0;  X -> R0
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = w + 4 * i, r0 = 16 * (t / NCP), cc = 16 * (t % NCP);
#pragma unroll
    for (int qq = 0; qq < 4; ++qq) {
      const int r = r0 + 4 * g + qq, c = cc + li;
      R2[r * CPP + c] = c < r ? dPa[i][qq] * M1[r * CPP + c] : 0.0f;
      M1[r * CPP + c] = c <= r ? expf(float(gs[r] - gs[c])) * dPa[i][qq] : 0.0f;
      M0[r * CPP + c] = c <= r ? dTa[i][qq] : 0.0f;
    }
  }
  {
    F32Stager<float, C, C> sx;
    sx.load(xws + slot * C * C, C, C, tid);
    if constexpr (C < CP) {
      for (int i = tid; i < CP * CPP; i += kThreads) X[i] = 0.0f;
      __syncthreads();
    }
    sx.store(X, CPP, tid);
  }
  __syncthreads();
  // dQ = Y1 + dP K;  dK = Y2 - Y3 + dP^T Q;  dX = dT diag(a);  da_j = sum_i dT_ij X_ij
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int t = w + 4 * i, r0 = 16 * (t / NCQ), cc = 16 * (t % NCQ);
    tile_mma16<false, false>(y1[i], M1, CPP, Ks, QP, r0, cc, CP, li, g);
    tile_mma16<true, false>(y2[i], M1, CPP, Qs, QP, r0, cc, CP, li, g);
  }
  for (int i = tid; i < CP * CP; i += kThreads) {
    const int r = i / CP, c = i % CP;
    R1[r * CPP + c] = M0[r * CPP + c] * as[c];
  }
  if (tid < CP) {
    float s = 0.0f, y = 0.0f;
    for (int r = 0; r < CP; ++r) {
      s = fmaf(M0[r * CPP + tid], X[r * CPP + tid], s);
      y += R2[tid * CPP + r] - R2[r * CPP + tid];
    }
    for (int j = 0; j < NCQ; ++j) y += rx[j * CP + tid];
    das[tid] = s;
    ys[tid] = y;
  }
  __syncthreads();
  // W = X^T dX -> M1
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = w + 4 * i, r0 = 16 * (t / NCP), cc = 16 * (t % NCP);
    f32x4 acc = zero4();
    tile_mma16<true, false>(acc, X, CPP, R1, CPP, r0, cc, CP, li, g);
#pragma unroll
    for (int qq = 0; qq < 4; ++qq) M1[(r0 + 4 * g + qq) * CPP + cc + li] = acc[qq];
  }
  __syncthreads();
  // Gam dA = -Gam * (W X^T) (strictly lower) -> R2;  G = K K^T -> R1
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = w + 4 * i, r0 = 16 * (t / NCP), cc = 16 * (t % NCP);
    f32x4 acc = zero4(), gg = zero4();
    tile_mma16<false, true>(acc, M1, CPP, X, CPP, r0, cc, CP, li, g);
    tile_mma16<false, true>(gg, Ks, QP, Ks, QP, r0, cc, DKP, li, g);
#pragma unroll
    for (int qq = 0; qq < 4; ++qq) {
      const int r = r0 + 4 * g + qq, c = cc + li;
      R2[r * CPP + c] = c < r ? -expf(float(gs[r] - gs[c])) * acc[qq] : 0.0f;
      R1[r * CPP + c] = gg[qq];
    }
  }
  __syncthreads();
  // N = R2 * R1: da_i += sum_j N_ij, its part of the gates;  dG = diag(a) Gam dA -> R0 (X is done)
  if (tid < CP) {
    float s = 0.0f, cs = 0.0f;
    for (int c = 0; c < tid; ++c) s = fmaf(R2[tid * CPP + c], R1[tid * CPP + c], s);
    for (int r = tid + 1; r < CP; ++r) cs = fmaf(as[r] * R2[r * CPP + tid], R1[r * CPP + tid], cs);
    das[tid] += s;
    ys[tid] += as[tid] * s - cs;
  }
  for (int i = tid; i < CP * CP; i += kThreads) {
    const int r = i / CP, c = i % CP;
    X[r * CPP + c] = as[r] * R2[r * CPP + c];
  }
  __syncthreads();
  if (tid < CP) {
    float dl = 0.0f;
    if (tid < valid) {
      const float bt = to_f32(static_cast<const T*>(b.beta)[row0 + int64_t(tid) * H]);
      float da_db, da_dl;
      efla_alpha_grad(bt, R1[tid * CPP + tid], b.rule, da_db, da_dl);
      dl = das[tid] * da_dl;
      static_cast<T*>(b.dbeta)[row0 + int64_t(tid) * H] = from_f32<T>(das[tid] * da_db);
    }
    dls[tid] = dl;
  }
  if (w == 0) {  // dg_t = c0 + sum_{j<t} k_j . Y2_j + sum_{i>=t} y_i
    float wj = 0.0f;
    const float y = lane < CP ? ys[lane] : 0.0f;
    if (lane < CP)
      for (int j = 0; j < NCQ; ++j) wj += rw[j * CP + lane];
    const float before = wave_scan_f32(wj, lane) - wj;
    float after = y;  // suffix sums
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const float z = __shfl_down(after, d);
      if (lane + d < kWave) after += z;
    }
    const float cc = end * (c0s[0] + c0s[1] + c0s[2] + c0s[3]);
    if (lane < valid) store_gate_grad<T>(b.dg, row0 + int64_t(lane) * H, cc + before + after, b.dg32);
  }
  __syncthreads();
  // dK += (dG + dG^T) K + 2 diag(dlambda) K;  write dq, dk
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int t = w + 4 * i, r0 = 16 * (t / NCQ), cc = 16 * (t % NCQ);
    tile_mma16<false, false>(y2[i], X, CPP, Ks, QP, r0, cc, CP, li, g);
    tile_mma16<true, false>(y2[i], X, CPP, Ks, QP, r0, cc, CP, li, g);
#pragma unroll
    for (int qq = 0; qq < 4; ++qq) {
      const int r = r0 + 4 * g + qq, c = cc + li;
      if (r < valid && c < DK) {
        const float gq = y1[i][qq], gk = fmaf(2.0f * dls[r], Ks[r * QP + c], y2[i][qq]);
        if (dqh != nullptr) {
          dqh[(row0 + int64_t(r) * H) * DK + c] = gq;
          dkh[(row0 + int64_t(r) * H) * DK + c] = gk;
        } else {
          static_cast<T*>(b.dq)[krow0 * DK + r * k_stride + c] = from_f32<T>(gq);
          static_cast<T*>(b.dk)[krow0 * DK + r * k_stride + c] = from_f32<T>(gk);
        }
      }
    }
  }
}

// dq, dk of a shared key head: the sums over its H / Hk value heads, in order.
// One thread per four values.
template <typename T>
__global__ __launch_bounds__(kThreads) void gated_head_sum_kernel(const float* __restrict__ dqh,
                                                                  const float* __restrict__ dkh, T* __restrict__ dq,
                                                                  T* __restrict__ dk, int64_t rows, int R, int DK) {
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;  // (token, key head), four values
  const int shift = __builtin_ctz(unsigned(DK)) - 2;  // d_k / 4 threads a row, a power of two
  const int64_t row = i >> shift;
  if (row >= rows) return;
  const int c = int(i & ((1 << shift) - 1)) * 4;
  f32x4 x = zero4(), y = zero4();
  for (int r = 0; r < R; ++r) {
    x += *reinterpret_cast<const f32x4*>(dqh + (row * R + r) * DK + c);
    y += *reinterpret_cast<const f32x4*>(dkh + (row * R + r) * DK + c);
  }
  st4(dq + row * DK + c, x);
  st4(dk + row * DK + c, y);
}

}  // namespace efla
