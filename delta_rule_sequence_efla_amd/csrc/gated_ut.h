// gated_ut.h -- the UT transform of the gated delta rule (gated.h) for bf16
// inputs, one wavefront per chunk of 64 tokens.
//
// For a chunk with key rows K, coefficients a and gate sums G_i:
//     A = tril(diag(a) (Gam * K K^T), -1),  Gam_ij = e^{G_i - G_j},
//     X = (I + A)^{-1},  T = X diag(a).
// The work is laid out as in ut_wave.h (K as row fragments straight from
// memory, the four diagonal 16x16 blocks of X by forward substitution, the
// blocks below by fp32 16x16x4 products out of registers), with the tiles of
// K K^T scaled by Gam before they are used; Gam_ii = 1, so lambda still is
// their diagonal.  Gates are kept as base-2 logarithms: e^{G_i - G_j} is one
// v_exp_f32.
//
// Written per chunk slot:
//   xfr  X as the recurrence's operand fragments, in two bf16 parts (X = hi +
//        lo to 2^-16): [12][64 lanes][8], fragments (rt, ku) of the lower
//        triangle as pf_index numbers them, high parts first.  A lane's tile
//        of X_ij^T is half a fragment of row tile i, so X leaves the registers
//        in that order, 1 KiB coalesced, and is loaded the same way.  T itself
//        is not stored: where it is a factor, the other operand's rows are
//        scaled by a (T D = X (a D), T^T dU = a (X^T dU)).
//   gws  [4][64] fp32: G log2(e), e^{G_i}, e^{G_C - G_i}, a.  Tokens past the
//        end have a = 0 and G = G_C.
//   BWD: also what the backward's passes read: P = Gam * tril(Q K^T) as six
//        bf16 fragments in the same order, and the effective queries Qe =
//        diag(e^G) Q - P T diag(e^G) K, bf16 [64][d_k], through which the output
//        reads the chunk's start state (O = Qe S + P T V), formed from registers
//        as in ut_wave.h.
// Bound by HBM like ut_wave_kernel: 16 KiB of K read and 13 KiB written a chunk
// at d_k 128, 28 us for 4 x 4096 tokens of 16 heads (4.3 TB/s); the backward's
// instance reads 32 and writes 35 KiB, 36 us for 8 x 2048 tokens of 8 heads (3.9
// TB/s; 47 us when it wrote T and X in float32 as well).  A few chunks alone take
// 10 us, a launch and 6 us of one wavefront's chain.
#pragma once

#include "gated.h"
#include "launchers.h"
#include "lds_ring.h"
#include "ut_wave.h"

namespace efla {

// What the backward instance reads and writes besides (null otherwise).
struct GatedUtBwd {
  const uint16_t* q;
  uint16_t *p, *qe;
};

constexpr double kLog2e = 1.4426950408889634;
constexpr int kGatedX = 12 * 64 * 8;  // bf16 values of X per chunk slot
constexpr int kGatedP = 6 * 64 * 8;   // and of P
constexpr int kGatedG = 4 * 64;       // floats of the gate block per chunk slot

// e^{x} for x in base-2 logarithms
__device__ __forceinline__ float exp2_gate(float x) { return __builtin_amdgcn_exp2f(x); }

// High and low bf16 parts of eight fp32 values (two accumulator tiles), x = hi +
// lo to 2^-16, two values at a time: one packed conversion, the high parts back
// as floats by a shift and a mask, and one packed conversion of what is left
// (element by element the compiler converts every high part twice).
__device__ __forceinline__ void split_frag(const f32x4& lo4, const f32x4& hi4, Frag<uint16_t>& h, Frag<uint16_t>& l) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  u32x4 hp, lp;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const f32x4& src = e < 2 ? lo4 : hi4;
    const f32x2 x{src[2 * (e & 1)], src[2 * (e & 1) + 1]};
    const uint32_t p = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
    const f32x2 rest{x[0] - __uint_as_float(p << 16), x[1] - __uint_as_float(p & 0xffff0000u)};
    hp[e] = p;
    lp[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, bf16x2));
  }
  h.v = __builtin_bit_cast(bf16x8, hp);
  l.v = __builtin_bit_cast(bf16x8, lp);
}

// Fragments of a lower-triangular [64][64] array held in fragment order in the
// LDS: of rows 16 rt .., one 16-byte read, ...
__device__ __forceinline__ Frag<uint16_t> tri_frag(const uint16_t* X, int rt, int ku, int lane) {
  Frag<uint16_t> f;
  f.v = *reinterpret_cast<const bf16x8*>(X + (pf_index(rt, ku) * 64 + lane) * 8);
  return f;
}
// ... and of its transpose, rows 16 ct .. of X^T (ku >= ct / 2), as sw_frag_tr
__device__ __forceinline__ Frag<uint16_t> tri_frag_tr(const uint16_t* X, int ct, int ku, int lane) {
  const int j = lane & 15, g = lane >> 4;
  const int at = ((j & 3) * 16 + 4 * g + (j >> 2)) * 8 + 4 * (ct & 1);
  const bf16x4 lo = lds_read_tr(X + pf_index(2 * ku, ct >> 1) * 512 + at);
  const bf16x4 hi = lds_read_tr(X + pf_index(2 * ku + 1, ct >> 1) * 512 + at);
  Frag<uint16_t> f;
  f.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return f;
}

template <int DK, bool BWD = false>
__global__ __launch_bounds__(256, BWD ? 2 : 4) void gated_ut_wave_kernel(const uint16_t* __restrict__ k,
                                                            const uint16_t* __restrict__ beta,
                                                            const float* __restrict__ gate, uint16_t* __restrict__ xfr,
                                                            float* __restrict__ gws, int H, int Hk, int64_t L, int NC,
                                                            int64_t nchunks, int rule, const int32_t* __restrict__ cu,
                                                            int N, int64_t nwg_ut, int32_t* __restrict__ order,
                                                            GatedUtBwd b) {
  constexpr int C = 64;
  using S = UtWaveShape<DK, C>;
  constexpr int NRT = S::NRT, NKU = S::NKU, GBLK = S::GBLK, XP = S::XP, XBLK = S::XBLK;
  __shared__ __align__(16) unsigned char scratch_all[S::WAVES][S::SCRATCH];
  __shared__ __align__(16) float a_all[S::WAVES][64];
  __shared__ __align__(16) float g_all[S::WAVES][64];

  if (order != nullptr && int64_t(blockIdx.x) >= nwg_ut) {  // packed batch: the workgroups after the chunks rank the sequences
    rank_sequences<C>(cu, N, L, int(blockIdx.x - nwg_ut), order, reinterpret_cast<int*>(scratch_all));
    return;
  }
  const int lane = threadIdx.x & 63, w = wave_id(), li = lane & 15, g = lane >> 4;
  const int64_t id = int64_t(blockIdx.x) * S::WAVES + w;
  if (id >= nchunks) return;  // no workgroup barriers below
  SeqSpan sp;
  int chunk;
  const uint32_t unit = uint32_t(id) / uint32_t(NC), at = uint32_t(id) - unit * uint32_t(NC);
  const uint32_t batch = cu == nullptr ? unit / uint32_t(H) : 0u;
  const int64_t h = unit - batch * uint32_t(H);
  if (cu == nullptr) {
    chunk = int(at);
    sp = seq_span<C>(nullptr, int(batch), h, H, L, NC);
  } else if (!gated_slot_chunk<C>(cu, N, at, h, H, L, NC, lane, sp, chunk)) {
    return;  // a slot no chunk of the packed batch uses
  }
  const int64_t t0 = int64_t(chunk) * C;
  const int valid = int(sp.len - t0 < C ? sp.len - t0 : C);
  const int64_t tok0 = sp.bos + t0, row0 = tok0 * H + h;
  const int64_t hk = h / (H / Hk);
  float* Gs = reinterpret_cast<float*>(scratch_all[w]);  // [4][GBLK] diagonal blocks of Gam * K K^T, row-major
  float* Xs = Gs + 4 * GBLK;                             // [4][XBLK] diagonal X blocks, column-major
  float* as = a_all[w];
  float* gs = g_all[w];
  float* gl = a_all[w];  // the sums' second floats, until a takes their place

  Frag<uint16_t> Kf[NRT][NKU];
#pragma unroll
  for (int rt = 0; rt < NRT; ++rt) {
    const int t = 16 * rt + li;
    const uint16_t* src = k + ((tok0 + t) * Hk + hk) * DK + 8 * g;
#pragma unroll
    for (int ku = 0; ku < NKU; ++ku) {
      if (t < valid) Kf[rt][ku].v = *reinterpret_cast<const bf16x8*>(src + 32 * ku);
      else Kf[rt][ku].v = bf16x8{};
    }
  }
  float bt = 0.0f, gt = 0.0f;
  if (lane < valid) {
    bt = to_f32(beta[row0 + int64_t(lane) * H]);
    gt = gate_floor(gate[row0 + int64_t(lane) * H]);
  }
  // G in two floats, so that differences behind a reset are as good as before
  // it.  The block in gws holds the first: it serves P, which is rounded to bf16
  // (behind 48 resets in a chunk o is off by 3.0e-3, without any by 2.9e-3), and
  // the backward's Gam (gated_bwd_chunk.h).
  // Against float sums: 0.3 us of a 135 us forward (4 x 4096 tokens, 16 heads, d 128).
  const double Gd64 = wave_scan_gate(gt, lane) * kLog2e;
  const float G = float(Gd64);
  gs[lane] = G;
  gl[lane] = float(Gd64 - double(G));
  float* gdst = gws + id * kGatedG;
  gdst[lane] = G;
  gdst[64 + lane] = exp2_gate(G);
  gdst[128 + lane] = exp2_gate(float(__shfl(Gd64, 63) - Gd64));
  wave_lds_order();

  // Gam * K K^T: Gd[b] holds rows li, columns 4g.. of diagonal block b (K K^T
  // is symmetric), Gu[i][m] the tile of block (i, m) transposed, m < i
  f32x4 Gd[NRT];
  f32x4 Gu[NRT][NRT];
  float gr[NRT];
  f32x4 gc[NRT];
#pragma unroll
  for (int b = 0; b < NRT; ++b) {
    gr[b] = gs[16 * b + li];
    gc[b] = *reinterpret_cast<const f32x4*>(gs + 16 * b + 4 * g);
  }
  auto gam = [&](int r, int c, int qq) {
    return exp2_gate((gr[r] - gc[c][qq]) + (gl[16 * r + li] - gl[16 * c + 4 * g + qq]));
  };
#pragma unroll
  for (int bb = 0; bb < NRT; ++bb) {
    Gd[bb] = zero4();
#pragma unroll
    for (int ku = 0; ku < NKU; ++ku) mma(Gd[bb], Kf[bb][ku], Kf[bb][ku]);
#pragma unroll
    for (int qq = 0; qq < 4; ++qq) Gd[bb][qq] = 4 * g + qq <= li ? Gd[bb][qq] * gam(bb, bb, qq) : 0.0f;
  }
#pragma unroll
  for (int i = 1; i < NRT; ++i)
#pragma unroll
    for (int m = 0; m < i; ++m) {
      Gu[i][m] = zero4();
#pragma unroll
      for (int ku = 0; ku < NKU; ++ku) mma(Gu[i][m], Kf[m][ku], Kf[i][ku]);
#pragma unroll
      for (int qq = 0; qq < 4; ++qq) Gu[i][m][qq] *= gam(i, m, qq);
    }
#pragma unroll
  for (int bb = 0; bb < NRT; ++bb) *reinterpret_cast<f32x4*>(Gs + bb * GBLK + li * 16 + 4 * g) = Gd[bb];
  wave_lds_order();
  {
    const float lam = Gs[(lane >> 4) * GBLK + (lane & 15) * 17];
    const float a = (lane < valid) ? efla_alpha_rule(bt, lam, rule) : 0.0f;
    as[lane] = a;
    gdst[192 + lane] = a;
  }
  wave_lds_order();

  // diagonal blocks of X by forward substitution, lane = (block, column)
  {
    const int bb = lane >> 4, c = lane & 15;
    const float* Gb = Gs + bb * GBLK;
    f32x4 ab[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) ab[j] = *reinterpret_cast<const f32x4*>(as + 16 * bb + 4 * j);
    float x[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
      for (int j = 0; 4 * j < r; ++j) {
        const f32x4 grow = *reinterpret_cast<const f32x4*>(Gb + r * 16 + 4 * j);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int m = 4 * j + e;
          if (m < r) {
            if (e & 1) s1 = fmaf(grow[e], x[m], s1);
            else s0 = fmaf(grow[e], x[m], s0);
          }
        }
      }
      x[r] = (r == c ? 1.0f : 0.0f) - ab[r / 4][r % 4] * (s0 + s1);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<f32x4*>(Xs + bb * XBLK + c * XP + 4 * j) = f32x4{x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]};
  }
  wave_lds_order();
  // XTo[i][j] is the tile of X_ij^T (element qq of lane (li, g) = X[16 i + li][16 j + 4 g + qq])
  f32x4 X[NRT][NRT], XTo[NRT][NRT];
#pragma unroll
  for (int bb = 0; bb < NRT; ++bb) {
    X[bb][bb] = *reinterpret_cast<const f32x4*>(Xs + bb * XBLK + li * XP + 4 * g);
#pragma unroll
    for (int qq = 0; qq < 4; ++qq) XTo[bb][bb][qq] = Xs[bb * XBLK + (4 * g + qq) * XP + li];
  }
  f32x4 arow[NRT];
#pragma unroll
  for (int i = 0; i < NRT; ++i) arow[i] = *reinterpret_cast<const f32x4*>(as + 16 * i + 4 * g);
  wave_lds_order();
#pragma unroll
  for (int i = 1; i < NRT; ++i)
#pragma unroll
    for (int j = 0; j < i; ++j) {
      f32x4 R = zero4();
#pragma unroll
      for (int m = j; m < i; ++m) mma16_f32(R, Gu[i][m], X[m][j]);
#pragma unroll
      for (int qq = 0; qq < 4; ++qq) R[qq] *= arow[i][qq];
      f32x4 Y = zero4(), YT = zero4();
      mma16_f32(Y, XTo[i][i], R);
      mma16_f32(YT, R, XTo[i][i]);
#pragma unroll
      for (int qq = 0; qq < 4; ++qq) {
        X[i][j][qq] = -Y[qq];
        XTo[i][j][qq] = -YT[qq];
      }
    }
  bf16x8* xdst = reinterpret_cast<bf16x8*>(xfr + id * kGatedX) + lane;
#pragma unroll
  for (int i = 0; i < NRT; ++i)
#pragma unroll
    for (int ku = 0; 32 * ku <= 16 * i + 15; ++ku) {
      f32x4 t[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int j = 2 * ku + p;
#pragma unroll
        for (int qq = 0; qq < 4; ++qq)
          t[p][qq] = (j < i || (j == i && 4 * g + qq <= li)) ? XTo[i][j < i ? j : i][qq] : 0.0f;
      }
      Frag<uint16_t> hi, lo;
      split_frag(t[0], t[1], hi, lo);
      xdst[pf_index(i, ku) * 64] = hi.v;
      xdst[(6 + pf_index(i, ku)) * 64] = lo.v;
    }
  if constexpr (BWD) {
    constexpr int TP = S::TP, NKC = C / 32;
    uint16_t* Ts = reinterpret_cast<uint16_t*>(scratch_all[w]);  // [C][TP] staging
    float e_row[NRT];
#pragma unroll
    for (int i = 0; i < NRT; ++i) e_row[i] = exp2_gate(gr[i]);
    Frag<uint16_t> Qr[NRT][NKU];
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt) {
      const int t = 16 * rt + li;
#pragma unroll
      for (int ku = 0; ku < NKU; ++ku) {
        Qr[rt][ku].v = bf16x8{};
        if (t < valid)
          Qr[rt][ku].v = *reinterpret_cast<const bf16x8*>(b.q + ((tok0 + t) * Hk + hk) * DK + 32 * ku + 8 * g);
      }
    }
#pragma unroll
    for (int r = 0; r < NRT; ++r)
#pragma unroll
      for (int c = 0; c < NRT; ++c) {
        f32x4 acc = zero4();
        if (c <= r) {
#pragma unroll
          for (int ku = 0; ku < NKU; ++ku) mma(acc, Qr[r][ku], Kf[c][ku]);
        }
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {
          const int ii = 16 * r + 4 * g + qq, jj = 16 * c + li;
          Ts[ii * TP + jj] = from_f32<uint16_t>(jj <= ii ? acc[qq] * exp2_gate(gc[r][qq] - gr[c]) : 0.0f);
        }
      }
    wave_lds_order();
    // P^T as B operand fragments, ku <= rt / 2 (P is lower triangular), stored as such
    bf16x8* pdst = reinterpret_cast<bf16x8*>(b.p + id * kGatedP) + lane;
    Frag<uint16_t> PtB[NRT][NKC];
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
      for (int ku = 0; ku < NKC; ++ku)
        if (2 * ku <= rt) {
          const bf16x4 lo = *reinterpret_cast<const bf16x4*>(Ts + (16 * rt + li) * TP + 32 * ku + 4 * g);
          const bf16x4 hi = *reinterpret_cast<const bf16x4*>(Ts + (16 * rt + li) * TP + 32 * ku + 16 + 4 * g);
          PtB[rt][ku].v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
          __builtin_nontemporal_store(PtB[rt][ku].v, pdst + pf_index(rt, ku) * 64);
        }
    float acol[NRT];
#pragma unroll
    for (int j = 0; j < NRT; ++j) acol[j] = as[16 * j + li];
    f32x4 PTt[NRT][NRT];  // [j][rt]: (P T)^T[16 j + 4 g + qq][16 rt + li]
#pragma unroll
    for (int j = 0; j < NRT; ++j)
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt) {
        PTt[j][rt] = zero4();
        if (j > rt) continue;
#pragma unroll
        for (int ku = j / 2; ku <= rt / 2; ++ku) {
          f32x4 lo = zero4(), hi = zero4();
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) {
            if (j <= 2 * ku) lo[qq] = X[2 * ku][j][qq] * acol[j];
            if (j <= 2 * ku + 1) hi[qq] = X[2 * ku + 1][j][qq] * acol[j];
          }
          mma(PTt[j][rt], acc_frag<uint16_t>(lo, hi), PtB[rt][ku]);
        }
      }
    // rows (tokens) scaled by e^G: (P T diag(e^G))^T
#pragma unroll
    for (int j = 0; j < NRT; ++j) {
      f32x4 ej;
#pragma unroll
      for (int qq = 0; qq < 4; ++qq) ej[qq] = exp2_gate(gc[j][qq]);
#pragma unroll
      for (int rt = j; rt < NRT; ++rt)
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) PTt[j][rt][qq] *= ej[qq];
    }
    Frag<uint16_t> PTB[NKC][NRT];
#pragma unroll
    for (int ku = 0; ku < NKC; ++ku)
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt)
        if (2 * ku <= rt) PTB[ku][rt] = acc_frag<uint16_t>(PTt[2 * ku][rt], PTt[2 * ku + 1][rt]);
    uint16_t* qdst = b.qe + id * int64_t(C) * DK;
#pragma unroll
    for (int ku2 = 0; ku2 < NKU; ++ku2) {
      f32x4 Cq[2][NRT];  // [h][rt]: (P T diag(e^G) K)[16 rt + li][32 ku2 + 8 g + 4 h + qq]
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        Frag<uint16_t> sel;  // picks dim 32 ku2 + 8 (li / 4) + 4 hh + li % 4 for column li
#pragma unroll
        for (int e = 0; e < 8; ++e)
          sel.v[e] = static_cast<__bf16>((g == (li >> 2) && e == 4 * hh + (li & 3)) ? 1.0f : 0.0f);
        f32x4 ZK[NRT];
#pragma unroll
        for (int tb = 0; tb < NRT; ++tb) {
          ZK[tb] = zero4();
          mma(ZK[tb], Kf[tb][ku2], sel);
        }
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt) {
          Cq[hh][rt] = zero4();
#pragma unroll
          for (int ku = 0; 2 * ku <= rt; ++ku)
            mma(Cq[hh][rt], acc_frag<uint16_t>(ZK[2 * ku], ZK[2 * ku + 1]), PTB[ku][rt]);
        }
      }
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt) {
        const bf16x8 qv = Qr[rt][ku2].v;
        bf16x8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          o[e] = static_cast<__bf16>(fmaf(e_row[rt], static_cast<float>(qv[e]), -Cq[e / 4][rt][e % 4]));
        __builtin_nontemporal_store(o, reinterpret_cast<bf16x8*>(qdst + (16 * rt + li) * DK + 32 * ku2 + 8 * g));
      }
    }
  }
}

}  // namespace efla
